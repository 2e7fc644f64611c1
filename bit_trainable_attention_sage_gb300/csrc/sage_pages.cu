// sage_pages.cu -- who has which page of a pool: sequences that grow, end (sage_kv_resize), go on as others'
// (sage_kv_fork), and the pool compacted (sage_kv_compact).
//
// refs[p] counts the table entries that name page p; 0: it is free.  held[b] of row b's entries are pages.
// Free pages are given in ascending order to the sequences in ascending order, so that a call's result
// depends on nothing but its inputs.  Counting is integer, by atomics whose order does not matter.
//
// One cluster of kCluster CTAs plans a call: sequences and pages are cut over its threads in order, and a
// place in the order is a prefix sum over the cluster through distributed shared memory.  Bound by latency:
// a handful of cluster barriers.  What a plan copies is copied by a second kernel over all SMs, bound by
// memory bandwidth.
#include "sage_kv.cuh"
#include "sage_decode.h"
#include "sage_pages.h"

namespace sage {

__device__ unsigned int g_pages_err = 0;    // 1: a page, length or sequence was out of range; 2: the pool had no free page left

namespace pages {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kAll = kCluster * kThreads;
constexpr int kCopyThreads = 256;
constexpr int kSmall = 2048;                 // sequences whose children a CTA counts in its shared memory

struct Args {
    KvView c;
    int *table;              // c.table, which these calls write
    int *refs, *held;        // (pages), (B)
    const int *want;         // resize: (B) slots that are wanted
    const int *parent, *lens;   // fork: (B)
    int *out;                // resize: (B) slots held; fork: (B) lengths; compact: (1) pages used
    // workspace
    int *list;               // (pages): resize, fork: free pages in order; compact: free pages below the used number
    int *from;               // (pages): compact: pages that move, at their places in the order of the used ones
    int *map;                // (pages): compact: new page of a page that moves
    PageSum *first;          // (B): resize: first place in the list
    int *need;               // (B): fork: place in the list (-1: none)
    int *children, *heir;    // (B): fork
    int *held0;              // (B): fork: held as it was
    int *copy;               // (B, 3): fork: source page, destination page (-1: none), rows
    int *old;                // (B, max_pages): fork: the table as it was
    int *count;              // (2): compact: used pages, moves
};

__device__ __forceinline__ int cluster_rank() { return blockIdx.x; }     // the grid is one cluster

// The sums of x and y over the cluster's threads before this one, and over all of them.  x: pages that sequences
// want, which together can be more than 32 bits hold; y: things of the pool or sequences.  (Read by other CTAs until
// the next barrier of the cluster.)
struct Totals {
    PageSum x;
    int y;
};
struct Prefix {
    Totals before, total;
};
struct WarpTotals {
    PageSum x[kWarps];
    int y[kWarps];
};
__device__ __forceinline__ Prefix prefix(PageSum x, int y, Totals &s_total, WarpTotals &s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Prefix p{};
    PageSum ix = x;
    int iy = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const PageSum ux = __shfl_up_sync(0xffffffffu, ix, o);
        const int uy = __shfl_up_sync(0xffffffffu, iy, o);
        if (lane >= o) {
            ix += ux;
            iy += uy;
        }
    }
    if (lane == 31) {
        s_warp.x[warp] = ix;
        s_warp.y[warp] = iy;
    }
    p.before = Totals{ix - x, iy - y};
    __syncthreads();
    if (warp == 0) {
        PageSum sum = lane < kWarps ? s_warp.x[lane] : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s_total.x = sum;
    } else if (warp == 1) {
        const int sum = __reduce_add_sync(0xffffffffu, lane < kWarps ? s_warp.y[lane] : 0);
        if (lane == 0) s_total.y = sum;
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        p.before.x += w < warp ? s_warp.x[w] : 0;
        p.before.y += w < warp ? s_warp.y[w] : 0;
    }
    cluster_sync();
#pragma unroll
    for (int r = 0; r < kCluster; ++r) {
        const Totals n{cluster_long(&s_total.x, r), cluster_word(&s_total.y, r)};
        if (r < cluster_rank()) {
            p.before.x += n.x;
            p.before.y += n.y;
        }
        p.total.x += n.x;
        p.total.y += n.y;
    }
    return p;
}

// This thread's part of n things in order.
__device__ __forceinline__ void part_of(int n, int &begin, int &end) {
    const int per = (n + kAll - 1) / kAll, at = cluster_rank() * kThreads + threadIdx.x;
    begin = static_cast<int>(min(static_cast<long long>(n), static_cast<long long>(at) * per));
    end = min(n, begin + per);
}

__device__ __forceinline__ int held_of(const Args &a, int b) {
    const int n = __ldcg(a.held + b);
    if (n >= 0 && n <= a.c.max_pages) return n;
    atomicOr(&g_pages_err, 1u);
    return n < 0 ? 0 : a.c.max_pages;
}
// pages that n slots take, held to what a sequence can have
__device__ __forceinline__ int pages_of(const Args &a, int n) {
    if (n < 0 || n > a.c.cap) {
        atomicOr(&g_pages_err, 1u);
        n = n < 0 ? 0 : a.c.cap;
    }
    const int p = kv_page_of(a.c, n);
    return p + (n > p * a.c.page ? 1 : 0);
}
__device__ __forceinline__ bool is_page(const Args &a, int p) {
    if (static_cast<unsigned>(p) < static_cast<unsigned>(a.c.pages)) return true;
    atomicOr(&g_pages_err, 1u);
    return false;
}

// This thread's pages that are free.
__device__ __forceinline__ int free_pages(const Args &a, int &begin, int &end) {
    part_of(a.c.pages, begin, end);
    int n = 0;
    for (int p = begin; p < end; ++p) n += __ldcg(a.refs + p) == 0;
    return n;
}
// They, n of them, to their places in the list, as far as it is wanted.
__device__ __forceinline__ void list_free(const Args &a, int begin, int end, int n, int at, PageSum wanted) {
    for (int p = begin; p < end && n > 0 && at < wanted; ++p)
        if (__ldcg(a.refs + p) == 0) {
            a.list[at++] = p;
            --n;
        }
}

// ---- resize --------------------------------------------------------------------------------------
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) resize_kernel(const __grid_constant__ Args a) {
    __shared__ Totals s_total[2];
    __shared__ WarpTotals s_warp;
    const int lane = threadIdx.x & 31, warp = cluster_rank() * kWarps + (threadIdx.x >> 5);
    // pages that are no longer wanted go back, a warp a sequence
    for (int b = warp; b < a.c.B; b += kCluster * kWarps) {
        const int m = held_of(a, b), k = pages_of(a, __ldg(a.want + b));
        for (int e = k + lane; e < m; e += 32) {
            int *entry = a.table + static_cast<size_t>(b) * a.c.max_pages + e;
            const int p = *entry;
            if (is_page(a, p)) atomicSub(a.refs + p, 1);
            *entry = -1;
        }
    }
    // the places in the list of free pages of those that grow; in most steps of a decoding loop none does
    int begin, end;
    PageSum n = 0;
    part_of(a.c.B, begin, end);
    for (int b = begin; b < end; ++b) n += pages_more(pages_of(a, __ldg(a.want + b)), held_of(a, b));
    const Prefix grow = prefix(n, 0, s_total[0], s_warp);            // (a barrier of the cluster: the counts are down)
    int free = 0;
    if (grow.total.x > 0) {                                          // the whole cluster alike
        PageSum at = grow.before.x;
        int p0, p1;
        for (int b = begin; b < end; ++b) {
            a.first[b] = at;
            at += pages_more(pages_of(a, __ldg(a.want + b)), held_of(a, b));
        }
        const int mine = free_pages(a, p0, p1);
        __syncthreads();                                             // s_warp has been read
        const Prefix f = prefix(0, mine, s_total[1], s_warp);
        list_free(a, p0, p1, mine, f.before.y, grow.total.x);
        free = f.total.y;
    }
    cluster_sync();                                                  // (in either case: no CTA leaves while its sums are read)
    for (int b = warp; b < a.c.B; b += kCluster * kWarps) {
        const int m = held_of(a, b), k = pages_of(a, __ldg(a.want + b));
        int got = 0;
        if (k > m) {
            const PageSum first = __ldcg(a.first + b);               // below `free`, a count of pages, where got > 0
            got = pages_got(k - m, first, free);
            if (got < k - m && lane == 0) atomicOr(&g_pages_err, 2u);
            for (int i = lane; i < got; i += 32) {
                const int p = __ldcg(a.list + first + i);
                a.table[static_cast<size_t>(b) * a.c.max_pages + m + i] = p;
                a.refs[p] = 1;
            }
        }
        __syncwarp();                                                // every lane has read held[b]
        if (lane == 0) {
            const int now = k > m ? m + got : k;
            a.held[b] = now;
            a.out[b] = now * a.c.page;
        }
    }
}

// ---- fork ----------------------------------------------------------------------------------------
// sequence b's parent: itself where the input is none of -1 .. B - 1
__device__ __forceinline__ int parent_of(const Args &a, int b) {
    const int p = __ldg(a.parent + b);
    if (p >= -1 && p < a.c.B) return p;
    atomicOr(&g_pages_err, 1u);
    return b;
}
// slots of a sequence as it was, held to its pages
__device__ __forceinline__ int slots_of(const Args &a, int q, int held) {
    const int n = __ldg(a.lens + q);
    const long long most = static_cast<long long>(held) * a.c.page;
    if (n >= 0 && n <= most) return n;
    atomicOr(&g_pages_err, 1u);
    return n < 0 ? 0 : static_cast<int>(most);
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) fork_kernel(const __grid_constant__ Args a) {
    __shared__ Totals s_total;
    __shared__ WarpTotals s_warp;
    __shared__ int s_children[kSmall], s_heir[kSmall];
    const int lane = threadIdx.x & 31, warp = cluster_rank() * kWarps + (threadIdx.x >> 5);
    // How many go on from each sequence, and which of them keeps its last pages: itself, or else the first.  Each CTA
    // finds that for itself where the sequences are few: a barrier of the cluster costs more.
    const bool small = a.c.B <= kSmall;
    int *children = small ? s_children : a.children, *heirs = small ? s_heir : a.heir;
    const int first = small ? threadIdx.x : cluster_rank() * kThreads + threadIdx.x, step = small ? kThreads : kAll;
    for (int b = first; b < a.c.B; b += step) {
        children[b] = 0;
        heirs[b] = a.c.B;
    }
    if (small) __syncthreads();
    else cluster_sync();
    for (int b = first; b < a.c.B; b += step) {
        const int p = parent_of(a, b);
        if (p < 0) continue;
        atomicAdd(children + p, 1);
        atomicMin(heirs + p, p == b ? -1 : b);
    }
    if (small) __syncthreads();
    else cluster_sync();
    auto children_of = [&](int q) { return small ? s_children[q] : __ldcg(a.children + q); };
    auto heir_of = [&](int q) { return small ? s_heir[q] : __ldcg(a.heir + q); };
    // counts of the pages, and the rows as they were, a warp a sequence
    for (int q = warp; q < a.c.B; q += kCluster * kWarps) {
        const int h = held_of(a, q), c = children_of(q), full = kv_page_of(a.c, slots_of(a, q, h));
        const bool stays = c == 1 && heir_of(q) == -1;
        if (!stays) {
            for (int e = lane; e < h; e += 32) {
                const size_t i = static_cast<size_t>(q) * a.c.max_pages + e;
                const int p = a.table[i], more = e < full ? c - 1 : c == 0 ? -1 : 0;
                a.old[i] = p;
                if (is_page(a, p) && more) atomicAdd(a.refs + p, more);
            }
        }
        if (lane == 0) a.held0[q] = h;
    }
    cluster_sync();                                                  // the counts are as the new rows will have them
    // places in the list of free pages of those that need a copy of a page in use, and the list
    auto copies = [&](int b) -> bool {
        const int p = parent_of(a, b);
        if (p < 0 || p == b || heir_of(p) == b) return false;
        const int n = slots_of(a, p, __ldcg(a.held0 + p));
        return n > kv_page_of(a.c, n) * a.c.page;
    };
    int begin, end, p0, p1, n = 0;
    part_of(a.c.B, begin, end);
    for (int b = begin; b < end; ++b) n += copies(b);
    const int mine = free_pages(a, p0, p1);
    const Prefix f = prefix(n, mine, s_total, s_warp);
    int place = static_cast<int>(f.before.x);                        // (at most one a sequence)
    for (int b = begin; b < end; ++b) a.need[b] = copies(b) ? place++ : -1;
    list_free(a, p0, p1, mine, f.before.y, f.total.x);
    const int free = f.total.y;
    cluster_sync();
    // the new rows
    for (int b = warp; b < a.c.B; b += kCluster * kWarps) {
        const int p = parent_of(a, b), was = __ldcg(a.held0 + b), want = __ldcg(a.need + b);
        int keep = 0, slots = 0, src = -1, dst = -1, rows = 0;
        if (p >= 0) {
            const int h = __ldcg(a.held0 + p);
            slots = slots_of(a, p, h);
            const int full = kv_page_of(a.c, slots);
            rows = slots - full * a.c.page;
            keep = p == b || heir_of(p) == b ? h : full;
            if (want >= 0) {
                if (want < free) {
                    src = __ldcg(a.old + static_cast<size_t>(p) * a.c.max_pages + full);
                    dst = __ldcg(a.list + want);
                } else {                                             // the pool has none left: full pages only
                    if (lane == 0) atomicOr(&g_pages_err, 2u);
                    slots = full * a.c.page;
                }
            }
            if (p != b) {
                for (int e = lane; e < keep; e += 32)
                    a.table[static_cast<size_t>(b) * a.c.max_pages + e] = __ldcg(a.old + static_cast<size_t>(p) * a.c.max_pages + e);
                if (dst >= 0 && lane == 0) {
                    a.table[static_cast<size_t>(b) * a.c.max_pages + full] = dst;
                    a.refs[dst] = 1;
                }
                if (dst >= 0) keep = full + 1;
            }
        }
        for (int e = keep + lane; e < was; e += 32) a.table[static_cast<size_t>(b) * a.c.max_pages + e] = -1;
        if (lane == 0) {
            a.held[b] = keep;
            a.out[b] = slots;
            a.copy[3 * b] = src;
            a.copy[3 * b + 1] = dst >= 0 && is_page(a, src) ? dst : -1;
            a.copy[3 * b + 2] = rows;
        }
    }
}

// ROW_BYTES / 16 lanes a row, rows [0, n) of a head from one page to another, K and V together.
template <int UNROLL>
__device__ __forceinline__ void copy_rows(const uint4 *k0, uint4 *k1, const uint4 *v0, uint4 *v1, long long chunks, int tid, int threads) {
    for (long long i0 = tid; i0 < chunks; i0 += threads * UNROLL) {
        uint4 k[UNROLL], v[UNROLL];
#pragma unroll
        for (int x = 0; x < UNROLL; ++x)
            if (i0 + x * threads < chunks) {
                k[x] = k0[i0 + x * threads];
                v[x] = v0[i0 + x * threads];
            }
#pragma unroll
        for (int x = 0; x < UNROLL; ++x)
            if (i0 + x * threads < chunks) {
                k1[i0 + x * threads] = k[x];
                v1[i0 + x * threads] = v[x];
            }
    }
}

// grid: B * H: the rows of a page in use to the page that a child got for them
__global__ void __launch_bounds__(kCopyThreads) fork_copy_kernel(const __grid_constant__ Args a, int row_bytes, int page_scales) {
    const int bh = blockIdx.x, b = bh / a.c.H, h = bh - b * a.c.H;
    const int src = a.copy[3 * b], dst = a.copy[3 * b + 1], rows = a.copy[3 * b + 2];
    if (dst < 0) return;
    const size_t from = (static_cast<size_t>(src) * a.c.H + h), to = (static_cast<size_t>(dst) * a.c.H + h);
    const size_t chunks = static_cast<size_t>(a.c.page) * row_bytes / 16;
    copy_rows<4>(static_cast<const uint4 *>(a.c.K) + from * chunks, static_cast<uint4 *>(a.c.K) + to * chunks,
                 static_cast<const uint4 *>(a.c.V) + from * chunks, static_cast<uint4 *>(a.c.V) + to * chunks, static_cast<long long>(rows) * (row_bytes / 16), threadIdx.x, kCopyThreads);
    const int scales = page_scales ? (rows + (1 << a.c.block_shift) - 1) >> a.c.block_shift : 0;
    for (int i = threadIdx.x; i < scales; i += kCopyThreads) {
        a.c.sK[to * page_scales + i] = a.c.sK[from * page_scales + i];
        a.c.sV[to * page_scales + i] = a.c.sV[from * page_scales + i];
    }
}

// ---- compact ---------------------------------------------------------------------------------------
// The i-th of the used pages from place U on (U: how many are used) moves to the i-th free page below U.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) compact_kernel(const __grid_constant__ Args a) {
    __shared__ Totals s_total;
    __shared__ WarpTotals s_warp;
    int begin, end, n = 0;
    part_of(a.c.pages, begin, end);
    for (int p = begin; p < end; ++p) n += __ldcg(a.refs + p) != 0;
    const Prefix used = prefix(0, n, s_total, s_warp);
    const int U = used.total.y;
    // `at` used pages lie before p: a free p below U is free page p - at of them; a used one from U on has
    // place `at` in the order of all, of which the last ones move
    int at = used.before.y;
    for (int p = begin; p < end; ++p) {
        const bool there = __ldcg(a.refs + p) != 0;
        if (p == U) a.count[1] = U - at;                             // moves: free pages below U
        if (p < U && !there) a.list[p - at] = p;
        if (p >= U && there) a.from[at] = p;
        if (p >= U && !there) a.map[p] = -1;
        at += there;
    }
    if (cluster_rank() == 0 && threadIdx.x == 0) {
        a.count[0] = U;
        if (U == a.c.pages) a.count[1] = 0;                          // (no page U)
        a.out[0] = U;
    }
    cluster_sync();
    const int moves = __ldcg(a.count + 1);
    for (int i = cluster_rank() * kThreads + threadIdx.x; i < moves; i += kAll) {
        const int src = __ldcg(a.from + U - moves + i), dst = __ldcg(a.list + i);
        a.map[src] = dst;
        a.refs[dst] = __ldcg(a.refs + src);
        a.refs[src] = 0;
    }
}

// Tables and pages over all SMs: the first `rows` CTAs take the tables' rows in turn, all of them the moves' slices.
constexpr int kSlice = 4 * kCopyThreads;     // 16-byte chunks a CTA copies of K and of V at a time

__global__ void __launch_bounds__(kCopyThreads) compact_copy_kernel(const __grid_constant__ Args a, int row_bytes, int page_scales) {
    const int U = a.count[0], moves = a.count[1];
    if (moves == 0) return;
    for (int b = blockIdx.x; b < a.c.B; b += gridDim.x) {
        const int h = held_of(a, b);
        for (int e = threadIdx.x; e < h; e += kCopyThreads) {
            int *entry = a.table + static_cast<size_t>(b) * a.c.max_pages + e;
            const int p = *entry;
            if (!is_page(a, p) || p < U) continue;
            const int to = a.map[p];
            if (to >= 0) *entry = to;
            else atomicOr(&g_pages_err, 1u);                         // a page that the counts do not know
        }
    }
    const long long chunks = static_cast<long long>(a.c.H) * a.c.page * row_bytes / 16, scales = static_cast<long long>(a.c.H) * page_scales;
    const long long slices = (chunks + kSlice - 1) / kSlice, units = moves * slices;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int i = static_cast<int>(u / slices);
        const long long s = u - i * slices;
        const size_t src = a.from[U - moves + i], dst = a.list[i];
        const long long first = s * kSlice, n = min(static_cast<long long>(kSlice), chunks - first);
        copy_rows<4>(static_cast<const uint4 *>(a.c.K) + src * chunks + first, static_cast<uint4 *>(a.c.K) + dst * chunks + first,
                     static_cast<const uint4 *>(a.c.V) + src * chunks + first, static_cast<uint4 *>(a.c.V) + dst * chunks + first, n, threadIdx.x, kCopyThreads);
        if (s == 0)
            for (long long x = threadIdx.x; x < scales; x += kCopyThreads) {
                a.c.sK[dst * scales + x] = a.c.sK[src * scales + x];
                a.c.sV[dst * scales + x] = a.c.sV[src * scales + x];
            }
    }
}

// ---- host ------------------------------------------------------------------------------------------
// Places in the workspace, in ints; the last is its size.
struct Places {
    size_t list, from, map, first, need, children, heir, held0, copy, old, count, all;
};
static Places places(const sage_kv &c) {
    Places p;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += (n + 3) & ~static_cast<size_t>(3);
        return here;
    };
    p.list = take(c.pages);
    p.from = take(c.pages);
    p.map = take(c.pages);
    p.first = take(2 * static_cast<size_t>(c.B));
    p.need = take(c.B);
    p.children = take(c.B);
    p.heir = take(c.B);
    p.held0 = take(c.B);
    p.copy = take(3 * static_cast<size_t>(c.B));
    p.count = take(2);
    p.old = take(static_cast<size_t>(c.B) * c.max_pages);
    p.all = at;
    return p;
}

static Args args(const sage_kv &c, int *refs, int *held, int *out, void *workspace) {
    const Places p = places(c);
    int *w = static_cast<int *>(workspace);
    Args a{};
    a.c = kv_view(c);
    a.table = const_cast<int *>(c.table);
    a.refs = refs; a.held = held; a.out = out;
    a.list = w + p.list; a.from = w + p.from; a.map = w + p.map; a.first = reinterpret_cast<PageSum *>(w + p.first); a.need = w + p.need; a.children = w + p.children; a.heir = w + p.heir;
    a.held0 = w + p.held0; a.copy = w + p.copy; a.count = w + p.count; a.old = w + p.old;
    return a;
}
static int row_bytes(const sage_kv &c) { return c.d * (kv_format(c) == SAGE_KV_16 ? 2 : 1); }
static int page_scales(const sage_kv &c) { return kv_format(c) == SAGE_KV_16 ? 0 : c.page / (kv_block(c) ? kv_block(c) : 1); }

static int check(const sage_kv *c, const int *refs, const int *held, const void *workspace, size_t workspace_bytes) {
    const int st = check_kv(c, true);
    if (st != SAGE_OK) return st;
    if (!refs || !held) return SAGE_ERR_ARG;
    if (misaligned(refs, 4) || misaligned(held, 4)) return SAGE_ERR_ALIGN;
    if (!workspace || workspace_bytes < places(*c).all * sizeof(int)) return SAGE_ERR_WORKSPACE;
    return misaligned(workspace, 16) ? SAGE_ERR_ALIGN : SAGE_OK;
}
static int status(cudaError_t e) { return e == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA; }

}  // namespace pages

unsigned int take_pages_error(unsigned int which) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_pages_err, sizeof(v));
    if (v & which) {
        const unsigned int left = v & ~which;
        cudaMemcpyToSymbol(g_pages_err, &left, sizeof(left));
    }
    return v & which;
}

}  // namespace sage

using namespace sage;

extern "C" {

size_t sage_pages_workspace_bytes(const sage_kv *c) {
    return check_kv(c, false) == SAGE_OK ? pages::places(*c).all * sizeof(int) : 0;
}

int sage_kv_resize(const sage_kv *c, int *refs, int *held, const int *want, int *slots, void *workspace, size_t workspace_bytes,
                   sage_stream_t stream) {
    const int st = pages::check(c, refs, held, workspace, workspace_bytes);
    if (st != SAGE_OK) return st;
    if (!want || !slots) return SAGE_ERR_ARG;
    const size_t n = static_cast<size_t>(c->B) * sizeof(int);        // one sequence's may be read after another's is written
    if (overlap(slots, n, want, n) || overlap(slots, n, held, n)) return SAGE_ERR_ARG;
    if (misaligned(want, 4) || misaligned(slots, 4)) return SAGE_ERR_ALIGN;
    pages::Args a = pages::args(*c, refs, held, slots, workspace);
    a.want = want;
    pages::resize_kernel<<<pages::kCluster, pages::kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    return pages::status(cudaGetLastError());
}

int sage_kv_fork(const sage_kv *c, int *refs, int *held, const int *parent, const int *lens, int *lens_out, void *workspace,
                 size_t workspace_bytes, sage_stream_t stream) {
    const int st = pages::check(c, refs, held, workspace, workspace_bytes);
    if (st != SAGE_OK) return st;
    if (c->score || c->pos) return SAGE_ERR_UNSUPPORTED;             // what eviction writes may not be shared
    if (!parent || !lens || !lens_out) return SAGE_ERR_ARG;
    const size_t n = static_cast<size_t>(c->B) * sizeof(int);
    if (overlap(lens_out, n, parent, n) || overlap(lens_out, n, lens, n) || overlap(lens_out, n, held, n)) return SAGE_ERR_ARG;
    if (misaligned(parent, 4) || misaligned(lens, 4) || misaligned(lens_out, 4)) return SAGE_ERR_ALIGN;
    pages::Args a = pages::args(*c, refs, held, lens_out, workspace);
    a.parent = parent;
    a.lens = lens;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    pages::fork_kernel<<<pages::kCluster, pages::kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return SAGE_ERR_CUDA;
    pages::fork_copy_kernel<<<static_cast<unsigned>(c->B) * c->H, pages::kCopyThreads, 0, s>>>(a, pages::row_bytes(*c), pages::page_scales(*c));
    return pages::status(cudaGetLastError());
}

int sage_kv_compact(const sage_kv *c, int *refs, const int *held, int *used, void *workspace, size_t workspace_bytes, sage_stream_t stream) {
    const int st = pages::check(c, refs, held, workspace, workspace_bytes);
    if (st != SAGE_OK) return st;
    if (!used) return SAGE_ERR_ARG;
    if (misaligned(used, 4)) return SAGE_ERR_ALIGN;
    pages::Args a = pages::args(*c, refs, const_cast<int *>(held), used, workspace);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    pages::compact_kernel<<<pages::kCluster, pages::kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return SAGE_ERR_CUDA;
    pages::compact_copy_kernel<<<kSMs * 6, pages::kCopyThreads, 0, s>>>(a, pages::row_bytes(*c), pages::page_scales(*c));
    return pages::status(cudaGetLastError());
}

}  // extern "C"
