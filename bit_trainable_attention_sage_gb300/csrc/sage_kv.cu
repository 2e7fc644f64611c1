// sage_kv.cu -- writing the paged key-value cache: new tokens (sage_kv_append) and eviction by
// accumulated attention weight (sage_kv_evict).
#include "sage_kv.cuh"

namespace sage {

__device__ unsigned int g_kv_err = 0;   // 1: a page, length or slot was out of range

// ---------------------------------------------------------------------------------------------
// append
//
// delta = fl32(max|x| / M), code = nearest of fl32(x / delta), M = 127 (INT8) or 448 (E4M3), one
// delta a row of d values, x = fl32(K - mu) or V; a 16-bit pool takes the values as they are.
// Every element is read once and written once: bound by memory bandwidth (prompts) or by latency
// (single tokens).  d / 8 lanes hold a row, 16 bytes each, so the maximum is 3 or 4 shuffles, a
// row's loads and stores are whole sectors, and K and V of a row, and ROWS rows, are in flight
// together.
// ---------------------------------------------------------------------------------------------
constexpr int kAppendThreads = 256;

struct AppendArgs {
    KvView c;
    const void *K, *V;
    const int *start, *count, *pos0;
    const float *mu;
    int T;
};

template <typename T>
__device__ __forceinline__ void unpack16(const uint4 u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f;
        if constexpr (std::is_same<T, __half>::value)
            f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        else
            f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// One row's 8 values of a lane -> 8 codes, and the row's scale.
template <int KIND, int LANES>
__device__ __forceinline__ uint2 kv_codes(const float (&x)[8], float *delta_out) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float delta = __fdiv_rn(m, KIND == SAGE_KV_INT8 ? 127.0f : 448.0f);
    *delta_out = delta;
    if (delta == 0.0f) return make_uint2(0u, 0u);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (KIND == SAGE_KV_INT8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                int q = __float2int_rn(__fdiv_rn(x[4 * i + j], delta));
                q = max(-127, min(127, q));                 // a subnormal delta can round down
                w[i] |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * j);
            }
        } else {
            w[i] = e4m3x2(__fdiv_rn(x[4 * i], delta), __fdiv_rn(x[4 * i + 1], delta)) |
                   static_cast<uint32_t>(e4m3x2(__fdiv_rn(x[4 * i + 2], delta), __fdiv_rn(x[4 * i + 3], delta))) << 16;
        }
    }
    return make_uint2(w[0], w[1]);
}

// grid: (row groups of a head, B * H).  ROWS rows of each lane group are loaded before any is
// written.
template <typename T, int KIND, int D, int ROWS>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs a) {
    constexpr int LANES = D / 8, GROUPS = kAppendThreads / LANES;
    const int bh = blockIdx.y, b = bh / a.c.H, h = bh - b * a.c.H;
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    const int t0 = blockIdx.x * (GROUPS * ROWS);
    int n = a.T;
    if (a.count) {
        n = __ldg(a.count + b);
        if (n < 0 || n > a.T) {
            if (threadIdx.x == 0) atomicOr(&g_kv_err, 1u);
            n = n < 0 ? 0 : a.T;
        }
    }
    if (t0 >= n) return;
    const int start = __ldg(a.start + b);
    const uint4 *K = reinterpret_cast<const uint4 *>(a.K) + static_cast<size_t>(bh) * a.T * LANES + lane;
    const uint4 *V = reinterpret_cast<const uint4 *>(a.V) + static_cast<size_t>(bh) * a.T * LANES + lane;
    uint4 k[ROWS], v[ROWS];
    long long row[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int t = t0 + r * GROUPS + group;
        k[r] = v[r] = make_uint4(0u, 0u, 0u, 0u);
        row[r] = -1;
        if (t < n) {
            k[r] = __ldg(K + static_cast<size_t>(t) * LANES);
            v[r] = __ldg(V + static_cast<size_t>(t) * LANES);
            const long long s = static_cast<long long>(start) + t;
            if (s < 0 || s >= a.c.cap) {
                atomicOr(&g_kv_err, 1u);
            } else {
                const int p = kv_page(a.c, b, static_cast<int>(s), &g_kv_err);
                if (p >= 0) {
                    row[r] = static_cast<long long>(kv_row(a.c, p, h, static_cast<int>(s)));
                    if (lane == 0) {
                        const size_t at = static_cast<size_t>(bh) * a.c.cap + s;
                        if (a.c.score) a.c.score[at] = 0.0f;
                        if (a.c.pos) a.c.pos[at] = a.pos0 ? __ldg(a.pos0 + b) + t : static_cast<int>(s);
                    }
                }
            }
        }
    }
    if constexpr (KIND == SAGE_KV_16) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            if (row[r] >= 0) {
                reinterpret_cast<uint4 *>(a.c.K)[row[r] * LANES + lane] = k[r];
                reinterpret_cast<uint4 *>(a.c.V)[row[r] * LANES + lane] = v[r];
            }
    } else {
        float mu[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (a.mu) {
            const float4 *m = reinterpret_cast<const float4 *>(a.mu + static_cast<size_t>(bh) * D + lane * 8);
            const float4 m0 = __ldg(m), m1 = __ldg(m + 1);
            mu[0] = m0.x; mu[1] = m0.y; mu[2] = m0.z; mu[3] = m0.w;
            mu[4] = m1.x; mu[5] = m1.y; mu[6] = m1.z; mu[7] = m1.w;
        }
        // every lane of a warp takes part in the shuffles, rows or none
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            float x[8], y[8], dk, dv;
            unpack16<T>(k[r], x);
            unpack16<T>(v[r], y);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fsub_rn(x[i], mu[i]);
            const uint2 ck = kv_codes<KIND, LANES>(x, &dk), cv = kv_codes<KIND, LANES>(y, &dv);
            if (row[r] >= 0) {
                reinterpret_cast<uint2 *>(a.c.K)[row[r] * LANES + lane] = ck;
                reinterpret_cast<uint2 *>(a.c.V)[row[r] * LANES + lane] = cv;
                if (lane == 0) {
                    a.c.sK[row[r]] = dk;
                    a.c.sV[row[r]] = dv;
                }
            }
        }
    }
}

template <typename T, int KIND, int D>
static void launch_append_k(const AppendArgs &a, cudaStream_t st) {
    constexpr int GROUPS = kAppendThreads / (D / 8);
    const unsigned bh = static_cast<unsigned>(a.c.B) * a.c.H;
    if (a.T <= GROUPS) {
        kv_append_kernel<T, KIND, D, 1><<<dim3(1, bh), kAppendThreads, 0, st>>>(a);
    } else {
        const unsigned x = (a.T + GROUPS * 4 - 1) / (GROUPS * 4);
        kv_append_kernel<T, KIND, D, 4><<<dim3(x, bh), kAppendThreads, 0, st>>>(a);
    }
}

template <typename T, int KIND>
static void launch_append_d(const AppendArgs &a, int d, cudaStream_t st) {
    if (d == 64) launch_append_k<T, KIND, 64>(a, st);
    else launch_append_k<T, KIND, 128>(a, st);
}

static void launch_append(const sage_kv &c, const AppendArgs &a, cudaStream_t st) {
    // a 16-bit pool is copied: one instance serves both 16-bit types
    if (c.kind == SAGE_KV_16) launch_append_d<__half, SAGE_KV_16>(a, c.d, st);
    else if (c.kind == SAGE_KV_INT8 && c.dtype == SAGE_FP16) launch_append_d<__half, SAGE_KV_INT8>(a, c.d, st);
    else if (c.kind == SAGE_KV_INT8) launch_append_d<__nv_bfloat16, SAGE_KV_INT8>(a, c.d, st);
    else if (c.dtype == SAGE_FP16) launch_append_d<__half, SAGE_KV_FP8>(a, c.d, st);
    else launch_append_d<__nv_bfloat16, SAGE_KV_FP8>(a, c.d, st);
}

// ---------------------------------------------------------------------------------------------
// eviction
//
// Which slots stay is a selection, not a sort: the budget-th largest key of a row of n keys by
// radix selection (four passes of 8 bits), then one pass in slot order that takes what is above it
// and the first of what is equal.  Only stayers in slots >= budget move, into the freed slots
// below: sources and destinations are disjoint, so the moves need no order among them, and a
// cache that is cut back by a few tokens moves a few rows instead of being compacted.
//
// kv_select_kernel: one CTA a (sequence, kv head); reads score and pos, writes the pairs
// (destination, source) to the workspace.  kv_move_kernel: the moves, spread over the GPU.
// ---------------------------------------------------------------------------------------------
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

struct EvictArgs {
    KvView c;
    const int *lens, *seen;
    int *lens_out;
    int *moves;          // (B*H): rows to move
    int *dst, *src;      // (B*H, max_moves)
    int budget, recent, max_moves;
};

// Larger key = stays longer.  Recent tokens above every score; scores in the order of the reals
// (-0 = +0), NaN last.
__device__ __forceinline__ uint32_t evict_key(float s, bool recent) {
    if (recent) return 0xFFFFFFFFu;
    if (s != s) return 0u;
    const uint32_t u = __float_as_uint(s + 0.0f);           // -0 becomes +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);      // at most 0xFF800000 (+inf)
}

struct KeyReader {
    const float *score;
    const int *pos;
    long long newest;    // positions from here on are recent
    __device__ __forceinline__ uint32_t operator()(int s) const {
        return evict_key(__ldg(score + s), __ldg(pos + s) >= newest);
    }
};

__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(const EvictArgs a) {
    __shared__ int hist[256];
    __shared__ int wcount[2][kSelWarps];
    __shared__ int s_digit, s_above;
    const int bh = blockIdx.x, b = bh / a.c.H;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int n = kv_len(a.c, a.lens, b, &g_kv_err);
    if (tid == 0 && bh - b * a.c.H == 0) a.lens_out[b] = min(n, a.budget);
    if (n <= a.budget) {
        if (tid == 0) a.moves[bh] = 0;
        return;
    }
    const size_t base = static_cast<size_t>(bh) * a.c.cap;
    const KeyReader key{a.c.score + base, a.c.pos + base, static_cast<long long>(__ldg(a.seen + b)) - a.recent};
    // the budget-th largest key: `prefix` its leading digits, `need` its rank among the keys that share them
    uint32_t prefix = 0;
    int need = a.budget;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
        for (int s = tid; s < n; s += kSelThreads) {
            const uint32_t k = key(s);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (warp == 0) {
            // lane l holds digits 255 - 8 l .. 248 - 8 l, in descending order
            int c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = hist[255 - 8 * lane - i];
                sum += c[i];
            }
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            int above = incl - sum;
            if (above < need && need <= incl) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (above < need && need <= above + c[i]) {
                        s_digit = 255 - 8 * lane - i;
                        s_above = above;
                    }
                    above += c[i];
                }
            }
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(s_digit) << shift;
        need -= s_above;
        __syncthreads();
    }
    // slot order: warp w owns slots [w * span, (w + 1) * span), span a multiple of 32
    const uint32_t T = prefix;
    const int span = ((n + kSelThreads - 1) / kSelThreads) * 32;
    const int s0 = min(n, warp * span), s1 = min(n, s0 + span);
    int eq = 0;
    for (int s = s0; s < s1; s += 32) {
        const bool in = s + lane < s1;
        eq += __popc(__ballot_sync(0xffffffffu, in && key(s + lane) == T));
    }
    if (lane == 0) wcount[0][warp] = eq;
    __syncthreads();
    int eq0 = 0;                                      // equal keys in the slots before this warp's
    for (int w = 0; w < warp; ++w) eq0 += wcount[0][w];
    __syncthreads();
    // freed slots below the budget and stayers from it on, counted, then numbered
    const uint32_t before = (1u << lane) - 1u;
    int at[2] = {0, 0};
    for (int pass = 0; pass < 2; ++pass) {
        int e = eq0, freed = at[0], moved = at[1];
        for (int s = s0; s < s1; s += 32) {
            const bool in = s + lane < s1;
            const uint32_t k = in ? key(s + lane) : 0u;
            const bool iseq = in && k == T;
            const uint32_t beq = __ballot_sync(0xffffffffu, iseq);
            const bool stays = in && (k > T || (iseq && e + __popc(beq & before) < need));
            e += __popc(beq);
            const bool f = in && !stays && s + lane < a.budget, m = stays && s + lane >= a.budget;
            const uint32_t bf = __ballot_sync(0xffffffffu, f), bm = __ballot_sync(0xffffffffu, m);
            if (pass == 1) {
                const size_t o = static_cast<size_t>(bh) * a.max_moves;
                if (f) a.dst[o + freed + __popc(bf & before)] = s + lane;
                if (m) a.src[o + moved + __popc(bm & before)] = s + lane;
            }
            freed += __popc(bf);
            moved += __popc(bm);
        }
        if (pass == 0) {
            if (lane == 0) {
                wcount[0][warp] = freed;
                wcount[1][warp] = moved;
            }
            __syncthreads();
            for (int w = 0; w < warp; ++w) {
                at[0] += wcount[0][w];
                at[1] += wcount[1][w];
            }
            if (tid == kSelThreads - 1) a.moves[bh] = at[1] + wcount[1][warp];
        }
    }
}

// grid: (blocks a row, B * H); ROW_BYTES / 16 lanes a move.
template <int ROW_BYTES>
__global__ void __launch_bounds__(256) kv_move_kernel(const EvictArgs a) {
    constexpr int CHUNKS = ROW_BYTES / 16;                   // 4, 8 or 16
    constexpr int GROUPS = 256 / CHUNKS;
    const int bh = blockIdx.y, b = bh / a.c.H, h = bh - b * a.c.H;
    const int m = a.moves[bh];
    const int lane = threadIdx.x % CHUNKS;
    for (int i = blockIdx.x * GROUPS + threadIdx.x / CHUNKS; i < m; i += gridDim.x * GROUPS) {
        const size_t o = static_cast<size_t>(bh) * a.max_moves + i;
        const int d = a.dst[o], s = a.src[o];
        const int pd = kv_page(a.c, b, d, &g_kv_err), ps = kv_page(a.c, b, s, &g_kv_err);
        if (pd < 0 || ps < 0) continue;
        const size_t rd = kv_row(a.c, pd, h, d), rs = kv_row(a.c, ps, h, s);
        uint4 *K = static_cast<uint4 *>(a.c.K), *V = static_cast<uint4 *>(a.c.V);
        const uint4 k = K[rs * CHUNKS + lane], v = V[rs * CHUNKS + lane];
        K[rd * CHUNKS + lane] = k;
        V[rd * CHUNKS + lane] = v;
        if (lane == 0) {
            if (a.c.sK) {
                a.c.sK[rd] = a.c.sK[rs];
                a.c.sV[rd] = a.c.sV[rs];
            }
            const size_t base = static_cast<size_t>(bh) * a.c.cap;
            a.c.score[base + d] = a.c.score[base + s];
            a.c.pos[base + d] = a.c.pos[base + s];
        }
    }
}

static int evict_max_moves(const sage_kv &c, int budget) {
    const int cap = c.max_pages * c.page;
    const int m = budget < cap - budget ? budget : cap - budget;
    return m < 0 ? 0 : (m + 3) & ~3;
}

unsigned int take_kv_error() {
    unsigned int v = 0, zero = 0;
    cudaMemcpyFromSymbol(&v, g_kv_err, sizeof(v));
    cudaMemcpyToSymbol(g_kv_err, &zero, sizeof(zero));
    return v;
}

}  // namespace sage

using namespace sage;

extern "C" {

int sage_kv_append(const sage_kv *c, const void *K, const void *V, int T, const int *start, const int *count,
                   const float *mu, const int *pos0, sage_stream_t stream) {
    const int st = check_kv(c, true);
    if (st != SAGE_OK) return st;
    if (T <= 0 || !K || !V || !start) return SAGE_ERR_ARG;
    if (T >= (1 << 30)) return SAGE_ERR_UNSUPPORTED;
    if (mu && c->kind == SAGE_KV_16) return SAGE_ERR_UNSUPPORTED;
    if (misaligned(K, 16) || misaligned(V, 16) || misaligned(mu, 16) || misaligned(start, 4) ||
        misaligned(count, 4) || misaligned(pos0, 4))
        return SAGE_ERR_ALIGN;
    const AppendArgs a{kv_view(*c), K, V, start, count, pos0, mu, T};
    launch_append(*c, a, reinterpret_cast<cudaStream_t>(stream));
    return cudaGetLastError() == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA;
}

size_t sage_evict_workspace_bytes(const sage_kv *c, int budget) {
    if (check_kv(c, false) != SAGE_OK || budget <= 0) return 0;
    const size_t rows = static_cast<size_t>(c->B) * c->H;
    return (rows + 2 * rows * evict_max_moves(*c, budget)) * sizeof(int);
}

int sage_kv_evict(const sage_kv *c, const int *lens, const int *seen, int budget, int recent, int *lens_out,
                  void *workspace, size_t workspace_bytes, sage_stream_t stream) {
    const int st = check_kv(c, true);
    if (st != SAGE_OK) return st;
    if (!lens || !seen || !lens_out || lens_out == lens || !c->score || !c->pos) return SAGE_ERR_ARG;
    if (budget <= 0 || recent < 0 || recent > budget) return SAGE_ERR_ARG;
    if (misaligned(lens, 4) || misaligned(seen, 4) || misaligned(lens_out, 4)) return SAGE_ERR_ALIGN;
    if (!workspace || workspace_bytes < sage_evict_workspace_bytes(c, budget)) return SAGE_ERR_WORKSPACE;
    if (misaligned(workspace, 16)) return SAGE_ERR_ALIGN;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int rows = c->B * c->H;
    EvictArgs a;
    a.c = kv_view(*c);
    a.lens = lens; a.seen = seen; a.lens_out = lens_out;
    a.budget = budget; a.recent = recent;
    a.max_moves = evict_max_moves(*c, budget);
    a.moves = static_cast<int *>(workspace);
    a.dst = a.moves + rows;
    a.src = a.dst + static_cast<size_t>(rows) * a.max_moves;
    kv_select_kernel<<<rows, kSelThreads, 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return SAGE_ERR_CUDA;
    if (a.max_moves == 0) return SAGE_OK;
    // enough CTAs that the GPU is full whatever the number of rows, and no more than the moves fill
    const int row_bytes = c->d * (c->kind == SAGE_KV_16 ? 2 : 1);
    const int groups = 256 / (row_bytes / 16);
    int x = (152 * 8 + rows - 1) / rows;
    const int most = (a.max_moves + groups - 1) / groups;
    if (x > most) x = most;
    const dim3 grid(x, rows);
    if (row_bytes == 64) kv_move_kernel<64><<<grid, 256, 0, s>>>(a);
    else if (row_bytes == 128) kv_move_kernel<128><<<grid, 256, 0, s>>>(a);
    else kv_move_kernel<256><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA;
}

}  // extern "C"
