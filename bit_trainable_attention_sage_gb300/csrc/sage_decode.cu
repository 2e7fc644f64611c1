// sage_decode.cu -- attention of one new token a sequence over the paged key-value cache.
//
//   s_t = q . K_t / sqrt(d),  O = sum_t softmax(s)_t V_t,  L = log sum_t exp s_t,  t < lens[b].
//
// Work.  Each cached row is read once from HBM for the whole group of query heads that shares it,
// so the kernel is bound by memory bandwidth: 2 d values (and 8 bytes of scales in 8 bits) a
// token and kv head, against 4 d multiply-adds a token and query head.
//
// Split.  The work is cut into tiles of 64 or 128 tokens of one (sequence, kv head, group of query
// heads), numbered in that order, and each of a fixed number of CTAs takes an equal run of them
// whatever the lengths are: a run can cover the end of one pair, several whole pairs and the
// start of another.  Lengths stay on the device; every CTA adds them up itself.  A pair that lies
// in one CTA's run is finished there; the others leave their unnormalised sums, maxima and sums
// of exponentials in the workspace (two places a CTA: a run's first and last pair), and a second
// kernel joins them in order, so results do not depend on the order in which CTAs run.
// Short caches (ONE) take a cluster of up to 8 CTAs a pair instead, joined through distributed
// shared memory: one launch, no workspace for sums, and no length but its own to read.
//
// Inside a CTA four warps each take a quarter of a tile (a granule) and never wait for one another:
// each keeps its own ring of cp.async stages in shared memory, its own running maximum, sum and
// output accumulators, and the four are joined once at the end of a pair.
//
// Products.  m16n8k16 tensor-core products with the tokens (q K^T) and the channels (P V) as the 16
// rows and the query heads as the 8 columns, so a group of up to 8 heads wastes nothing but the
// columns it lacks, and the output takes d / 16 registers a lane and column.  The kernel needs a
// fraction of the products' rate, and both operands come from registers, where 8-bit rows can be
// widened on the way; tcgen05 would want the widened rows back in shared memory.
//   - 16-bit pool: K by ldmatrix, V by its transposing form.
//   - 8-bit pool: codes are exact in fp16.  The products run over channels (or tokens) in any
//     order as long as both operands agree, so a lane takes 16 consecutive bytes of a row with
//     one load and assigns them to the products' positions itself; no transposition is needed.
//     q is scaled by a power of two a head to stay in fp16's range: exact to 2^-39 of its largest
//     value.  sK multiplies the logit, sV the probability.
//   - The probabilities enter as hi + lo of two values with float32's exponents, 16 bits or more of
//     each: one rounding to bf16 would show in the output, and fp16's exponents would end 2^-24 below
//     the largest, where the small weights beside a key that takes nearly all of it still make up the
//     output if that key's value is small.  bf16 and 8-bit pools: bf16 (8 + 8 bits), which holds the
//     codes too.  fp16 pools: the 11-bit type of m16n8k8, which holds fp16's 11 bits.  Two fp16 terms,
//     which lose the small weights, would save 1 % in fp16 pools (32 x 8191 tokens of 16 heads, d = 128:
//     312 against 317 us) and 1 to 7 % in 8 bits (262144 tokens of 8 heads: 89.9 against 90.9 in E4M3,
//     88.3 against 92.8 in INT8).  bf16 pools in the 11-bit type: 319 against 313.
//   - They change from the first product's layout to the second's operand by movmatrix (8 x 8
//     transposition in registers).
#include <utility>

#include "sage_kv.cuh"
#include "sage_decode.h"

namespace sage {

__device__ unsigned int g_decode_err = 0;   // 1: a page or length was out of range

constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kDecCluster = 8;               // CTAs of a cluster at most

// pools: KIND 0 fp16, 1 bf16, 2 INT8, 3 E4M3; BLOCK: one scale for 16 or more rows (8 bits); ROWS: several new
// tokens a sequence (instances of their own: what they need cost one token 1 to 2 %)
template <int D, int KIND, int MR = 8>
struct DecodeShape {
    static constexpr int ES = KIND < 2 ? 2 : 1;
    static constexpr int ROW = D * ES;                       // bytes
    static constexpr int CPR = ROW / 16;                     // 16-byte chunks a row: 4, 8 or 16
    // tokens a warp takes at a time: the maximum, the rescaling and the loads' addresses are paid
    // once a granule, and its products are independent chains
    static constexpr int GRAN = ROW == 256 ? 16 : 32;
    static constexpr int TILE = GRAN * kDecWarps;
    static constexpr int SCALES = KIND < 2 ? 0 : 2 * GRAN * 4;
    static constexpr int STAGE = 2 * GRAN * ROW + SCALES;
    // Resident CTAs an SM: three where 168 registers and a third of the shared memory do.  (131072
    // tokens in E4M3, 8 kv heads, d = 128: with 4 heads a group 51 us at two, 48 at three; with 16
    // a group 63 at two and 67 at three, which spill.)
    static constexpr int CTAS = ROW == 256 || (MR == 16 && D == 128) ? 2 : 3;
    static constexpr int STAGES = ROW == 64 ? 4 : CTAS == 3 ? 2 : 3;
    static constexpr int ALIGN = 512;                        // of the ring, so that its addresses can be XORed
    // a warp's ring; its last stage also holds the sums of 16 heads, D + 4 floats each
    static constexpr int RING = STAGES * STAGE + (ROW == 256 ? 256 : 0);
    static constexpr int SMEM = kDecWarps * RING + ALIGN;
};
constexpr int decode_tile(int row_bytes) { return (row_bytes == 256 ? 16 : 32) * kDecWarps; }
constexpr int decode_ctas(int row_bytes, int d, int mr) { return row_bytes == 256 || (mr == 16 && d == 128) ? 2 : 3; }
static_assert(decode_ctas(128, 128, 16) == DecodeShape<128, 2, 16>::CTAS && decode_ctas(128, 64, 16) == DecodeShape<64, 0, 16>::CTAS &&
              decode_ctas(64, 64, 16) == DecodeShape<64, 3, 16>::CTAS && decode_ctas(256, 128, 8) == DecodeShape<128, 1, 8>::CTAS, "");

struct DecodeArgs {
    KvView c;
    const void *Q;
    void *O;
    float *L;
    const int *lens;
    int Hq, G, chunks;       // query heads, heads a kv head, groups of at most MR heads a kv head
    int ctas;                // CTAs that share the work (gridDim.x)
    int cluster;             // ONE: CTAs a pair
    int tile, tile_shift;    // tokens a unit of work, 64 or 128, and their log2
    int bf16;                // type of q and O
    float sl2;               // log2(e) / sqrt(d)
    // Several new tokens a sequence (sage_attn_extend): T of them, lens[b] the slots before the first, count[b]
    // (NULL: T) those that are there.  The rows of a kv head are its heads' tokens: Hq and G count them,
    // row r's token is r mod T.  0: one token, lens[b] its slots.
    int T;
    const int *count;
    float *part_O;           // (ctas, 2, MR, d) unnormalised sums
    float *part_ml;          // (ctas, 2, MR, 2) maxima (log2 units) and sums of exponentials
    float *row_ml;           // (B, Hq, 2) the same of rows that one run finished, with scores only
    float *logits;           // (B, Hq, cap) log2-unit logits, with scores only
};

// ---- shared-memory and tensor-core pieces ----------------------------------------------------
template <int DST, int SRC>
__device__ __forceinline__ void cp_async16_at(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0+%2], [%1+%3], 16;" ::"r"(dst), "l"(src), "n"(DST), "n"(SRC) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool valid) {
    const int n = valid ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the same over 8 rows of the second dimension, 32-bit values of 11 bits
__device__ __forceinline__ void mma1688(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Place of 16-byte chunk c of row r in half a granule (16 rows; the other half follows).  Rows of 128 and 256 bytes in 16 bits: the 8
// rows an ldmatrix reads at one chunk fall into the 8 different 16-byte bank groups.  In 8 bits
// a quarter-warp reads chunks 0-3 of rows (2i, 2i + 1), or chunks (2i, 2i + 1) of rows 0, 2, 4, 6
// (1, 3, 5, 7): the XORs put either set into 8 different bank groups.
template <int D, int KIND>
__host__ __device__ constexpr uint32_t chunk_at(int r, int c) {
    using S = DecodeShape<D, KIND>;
    if constexpr (KIND < 2) return static_cast<uint32_t>(r * S::CPR + (c ^ (r & 7))) * 16u;
    else if constexpr (D == 128) return static_cast<uint32_t>(r * 8 + (c ^ ((r & 6) ^ ((r & 1) << 2)))) * 16u;
    else return static_cast<uint32_t>((r >> 1) * 8 + ((((r & 1) << 2) | c) ^ (((r >> 1) & 3) << 1))) * 16u;
}

// Half a granule's K and V rows, all 16 of them there: 32 lanes take 512 consecutive bytes at a
// time.  Place i of a lane is that of its first 512 bytes XOR a constant, plus 512 i.
template <int D, int KIND, int... I>
__device__ __forceinline__ void load_half(uint32_t k_dst, uint32_t v_dst, const uint8_t *k, const uint8_t *v,
                                          std::integer_sequence<int, I...>) {
    using S = DecodeShape<D, KIND>;
    constexpr int RPI = 32 / S::CPR;
    (cp_async16_at<I * 512, I * 512>(k_dst ^ (chunk_at<D, KIND>(I * RPI, 0) - I * 512u), k), ...);
    (cp_async16_at<I * 512, I * 512>(v_dst ^ (chunk_at<D, KIND>(I * RPI, 0) - I * 512u), v), ...);
}

// A pool's values i and i + 1 (E4M3: codes).
template <int KIND>
__device__ __forceinline__ float2 value_pair(const void *pool, size_t i) {
    if constexpr (KIND == 0) return __half22float2(*reinterpret_cast<const __half2 *>(static_cast<const __half *>(pool) + i));
    else if constexpr (KIND == 1) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(static_cast<const __nv_bfloat16 *>(pool) + i));
    else {
        const uint32_t h = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(static_cast<const uint8_t *>(pool) + i));
        return __half22float2(*reinterpret_cast<const __half2 *>(&h));
    }
}

// 8 x 8 transposition of 16-bit values over a warp: lane (g, q) gives row g, columns 2q and 2q + 1
// and gets those of column g.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// The same of 32-bit values, by their halves: (row g, column 2q), (row g, column 2q + 1) in, (row 2q, column g),
// (row 2q + 1, column g) out.
__device__ __forceinline__ void transpose8(float &x0, float &x1) {
    const uint32_t a = __float_as_uint(x0), b = __float_as_uint(x1);
    const uint32_t lo = transpose8(prmt(a, b, 0x5410)), hi = transpose8(prmt(a, b, 0x7632));
    x0 = __uint_as_float(prmt(lo, hi, 0x5410));
    x1 = __uint_as_float(prmt(lo, hi, 0x7632));
}

// (x0, x1) as hi + lo pairs of bf16
__device__ __forceinline__ void split2(float x0, float x1, uint32_t &hi, uint32_t &lo) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 l = __floats2bfloat162_rn(x0 - f.x, x1 - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}
// x as hi + lo of 11 bits each under float32's exponents (cut: 21 bits together)
__device__ __forceinline__ void split11(float x, uint32_t &hi, uint32_t &lo) {
    hi = __float_as_uint(x) & 0xFFFFE000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) & 0xFFFFE000u;
}

// ---- the slots of a sequence and of a row -----------------------------------------------------
__device__ __forceinline__ int new_tokens(const DecodeArgs &a, int b) {
    if (!a.count) return a.T;
    const int n = __ldg(a.count + b);
    if (n >= 0 && n <= a.T) return n;
    atomicOr(&g_decode_err, 1u);
    return n < 0 ? 0 : a.T;
}
template <bool ROWS>
__device__ __forceinline__ int seq_len(const DecodeArgs &a, int b) {
    int n = kv_len(a.c, a.lens, b, &g_decode_err);
    if constexpr (ROWS) {
        const int k = new_tokens(a, b);
        if (k == 0) return 0;
        n += k;
        if (n > a.c.cap) {
            atomicOr(&g_decode_err, 1u);
            n = a.c.cap;
        }
    }
    return n;
}
// the slots that row r of a kv head sees (several tokens only): its sequence's first new slot, new tokens and slots
__device__ __forceinline__ int row_limit(const DecodeArgs &a, int r, int start, int count, int len) {
    const int t = r % a.T;
    return t < count ? min(start + t + 1, len) : 0;
}

// ---- the cut of the work ---------------------------------------------------------------------
// A pair of `tiles` tiles counts kPairUnits + tiles units, the first kPairUnits for what a pair
// costs besides its tiles (its first reads and its end take about as long as a tile): a run over
// many short sequences then holds fewer tiles.
constexpr int kPairUnits = 1;
template <bool ROWS>
__device__ __forceinline__ int pair_units(const DecodeArgs &a, int b) {
    const int tiles = (seq_len<ROWS>(a, b) + a.tile - 1) >> a.tile_shift;
    return tiles > 0 ? tiles + kPairUnits : 0;
}

// The number of units; where unit u lies: its sequence and that sequence's first unit.  Called by
// a whole CTA of NT threads; `find` gives u from the total (a u outside [0, total) is not looked
// for).
struct WorkAt {
    long long total, u, first;
    int b;
};
template <int NT, bool ROWS, typename F>
__device__ __forceinline__ WorkAt locate(const DecodeArgs &a, int pairs, F find) {
    __shared__ long long s_sum[NT / 32];
    __shared__ long long s_first;
    __shared__ int s_b;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.c.B + NT - 1) / NT;
    const int b0 = min(tid * per, a.c.B), b1 = min(b0 + per, a.c.B);
    long long mine = 0;
    for (int b = b0; b < b1; ++b)
        mine += static_cast<long long>(pair_units<ROWS>(a, b)) * pairs;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    long long total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    const long long u = find(total);
    long long at = before + incl - mine;
    if (u >= at && u < at + mine) {
        int b = b0;
        for (;; ++b) {
            const long long k = static_cast<long long>(pair_units<ROWS>(a, b)) * pairs;
            if (u < at + k) break;
            at += k;
        }
        s_first = at;
        s_b = b;
    }
    __syncthreads();
    return WorkAt{total, u, s_first, s_b};
}

// Runs that share `total` units (none of them empty), the first unit of run c, and the run that
// holds unit u.
__device__ __forceinline__ int runs_of(const DecodeArgs &a, long long total) {
    return static_cast<int>(min(static_cast<long long>(a.ctas), total));
}
// (64-bit divisions take a good part of a microsecond: 32 bits where the products fit)
__device__ __forceinline__ long long div_up_to(long long n, long long d) {
    return n <= 0xFFFFFFFFll ? static_cast<long long>(static_cast<uint32_t>(n) / static_cast<uint32_t>(d)) : n / d;
}
__device__ __forceinline__ long long run_start(long long total, int c, int runs) { return div_up_to(total * c, runs); }
__device__ __forceinline__ int run_of(long long total, long long u, int runs) {
    const long long n = (u + 1) * runs - 1;
    if (n <= 0xFFFFFFFFll && total <= 0xFFFFFFFFll) return static_cast<int>(static_cast<uint32_t>(n) / static_cast<uint32_t>(total));
    return static_cast<int>(n / total);
}

__device__ __forceinline__ void store_out(const DecodeArgs &a, size_t at, float x, float y) {
    uint32_t w;
    if (a.bf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        w = *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        w = *reinterpret_cast<const uint32_t *>(&h);
    }
    reinterpret_cast<uint32_t *>(a.O)[at / 2] = w;
}

// 1 / l, and 0 where nothing was summed; a NaN stays one
__device__ __forceinline__ float inv_of(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
// m + log2 l in natural units; -inf where nothing was summed (m = -inf, l = 0)
__device__ __forceinline__ float lse_of(float m, float l) { return (m + log2f(l)) * 0.6931471805599453f; }

// ---- main kernel ------------------------------------------------------------------------------
template <int D, int KIND, int MR, bool ONE, bool BLOCK, bool ROWS>
__global__ void __launch_bounds__(kDecThreads, DecodeShape<D, KIND, MR>::CTAS) decode_kernel(const __grid_constant__ DecodeArgs a) {
    using S = DecodeShape<D, KIND, MR>;
    constexpr bool BF16 = KIND == 1;                 // type of the product K q
    constexpr bool TF32 = KIND == 0;                 // type of the product V^T P: 11 bits under float32's exponents, or bf16
    constexpr int KS = D / 16;                       // 16-channel steps of K q, row tiles of V^T P
    constexpr int HALVES = S::GRAN / 16;             // row tiles of K q, 16-token steps of V^T P
    constexpr int NH = MR / 8;                       // column tiles: 8 heads each
    constexpr int HALF = 16 * S::ROW;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & (S::ALIGN - 1));
    __shared__ float s_m[kDecWarps][MR], s_l[kDecWarps][MR];
    __shared__ float s_part[2][MR], s_f[kDecCluster][MR];        // ONE: a CTA's M and l; factors of the cluster's
    __shared__ int s_not_finite, s_limit[MR];                    // ROWS: a V was taken out of the products; slots a row sees
    (void)s_part; (void)s_f; (void)s_not_finite; (void)s_limit;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, q = lane & 3;
    const int pairs = a.c.H * a.chunks;
    const int cta = blockIdx.x;
    if constexpr (ROWS) {
        if (tid == 0) s_not_finite = 0;
        __syncthreads();
    }
    // The lengths say where this CTA's pages stand, the pages where its rows: three reads one after
    // the other.  The table and q are brought into L2 meanwhile, a share by each CTA.
    auto fetch = [&](size_t share, const void *table, size_t table_bytes, const void *Q, size_t q_bytes) {
        const size_t at = (share * 64 + (tid & 63)) * 128;
        const char *from = static_cast<const char *>(tid < 64 ? table : Q);
        if (at < (tid < 64 ? table_bytes : q_bytes)) asm volatile("prefetch.global.L2 [%0];" ::"l"(from + at));
    };
    // the run [u, u1) of units (ONE: a share of one pair's tiles)
    long long u = 0, u1 = 0, first = 0;
    int b, rank = 0;
    if constexpr (ONE) {
        const int pr = cta / a.cluster;
        rank = cta - pr * a.cluster;
        b = pr / pairs;
        const int pair = pr - b * pairs, hk = pair / a.chunks, h0 = hk * a.G + (pair - hk * a.chunks) * MR;
        const int outs = min(MR, a.G - (h0 - hk * a.G));
        const size_t head = static_cast<size_t>(b) * a.Hq + h0;
        fetch(rank, a.c.table + static_cast<size_t>(b) * a.c.max_pages, static_cast<size_t>(a.c.max_pages) * 4,
              static_cast<const char *>(a.Q) + head * D * 2, rank == 0 ? outs * D * 2 : 0);
        if (seq_len<ROWS>(a, b) == 0) {                                // the whole cluster alike
            for (int i = (rank * kDecThreads + tid) * 2; i < outs * D; i += a.cluster * kDecThreads * 2) {
                store_out(a, head * D + i, 0.0f, 0.0f);
                if (i % D == 0) a.L[head + i / D] = -INFINITY;
            }
            return;
        }
    } else {
        // the join may take its place on the GPU; it waits for this grid's end before it reads
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        fetch(cta, a.c.table, static_cast<size_t>(a.c.B) * a.c.max_pages * 4, a.Q, static_cast<size_t>(a.c.B) * a.Hq * D * 2);
        // sequences cta, cta + gridDim.x, ... without a token: a thread looks, its warp writes
        const int grid = gridDim.x;
        for (long long e0 = cta; e0 < a.c.B; e0 += static_cast<long long>(grid) * kDecThreads) {
            const long long mine = e0 + static_cast<long long>(grid) * tid;
            uint32_t none = __ballot_sync(0xffffffffu, mine < a.c.B && seq_len<ROWS>(a, static_cast<int>(min(mine, a.c.B - 1ll))) == 0);
            for (; none; none &= none - 1) {
                const size_t head = static_cast<size_t>(e0 + static_cast<long long>(grid) * (warp * 32 + __ffs(none) - 1)) * a.Hq;
                for (int i = lane * 2; i < a.Hq * D; i += 64) {
                    store_out(a, head * D + i, 0.0f, 0.0f);
                    if (i % D == 0) a.L[head + i / D] = -INFINITY;
                }
            }
        }
        const WorkAt w = locate<kDecThreads, ROWS>(a, pairs, [&](long long total) {
            const int n = runs_of(a, total);
            return cta < n ? run_start(total, cta, n) : total;
        });
        const int runs = runs_of(a, w.total);
        if (cta >= runs) return;
        u = w.u;
        u1 = run_start(w.total, cta + 1, runs);
        first = w.first;
        b = w.b;
    }
    // a warp's ring: stages of K rows, V rows, then (8 bits) K scales, V scales
    uint8_t *ring = smem + warp * S::RING;
    const uint32_t load_lane = smem_u32(ring) + chunk_at<D, KIND>(lane / S::CPR, lane % S::CPR);

    // the run's pairs, one after the other
    int len, tiles, t0, t1, hk, head0, heads, tok0, ng, edge;
    [[maybe_unused]] int first_new = 0, count = 0;               // ROWS: of the pair's sequence
    // The next pair of the run with a tile to do, from unit u on; u moves past its units.  False at
    // the run's end.
    auto find = [&]() {
        int pair;
        if constexpr (ONE) {
            len = seq_len<ROWS>(a, b);
            tiles = (len + S::TILE - 1) / S::TILE;
            pair = cta / a.cluster - b * pairs;
            t0 = tiles * rank / a.cluster;           // tiles < 2^24
            t1 = tiles * (rank + 1) / a.cluster;
        } else {
            for (;;) {
                if (u >= u1) return false;
                len = seq_len<ROWS>(a, b);
                tiles = (len + S::TILE - 1) / S::TILE;
                const int units = tiles > 0 ? tiles + kPairUnits : 0;
                if (u - first >= static_cast<long long>(units) * pairs) {
                    first += static_cast<long long>(units) * pairs;
                    ++b;
                    continue;
                }
                pair = static_cast<int>(div_up_to(u - first, units));
                const int v0 = static_cast<int>((u - first) - static_cast<long long>(pair) * units);
                const int v1 = static_cast<int>(min(static_cast<long long>(units), v0 + (u1 - u)));
                u += v1 - v0;
                t0 = max(0, v0 - kPairUnits);
                t1 = max(0, v1 - kPairUnits);
                if (t1 > t0) break;
            }
        }
        hk = pair / a.chunks;
        const int ch = pair - hk * a.chunks;
        head0 = hk * a.G + ch * MR;                  // first query head of the group
        heads = min(MR, a.G - ch * MR);
        // the last granules, where a slot may be hidden from a row: those with fewer than `edge` slots to the end
        edge = S::GRAN;
        if constexpr (ROWS) {
            first_new = kv_len(a.c, a.lens, b, &g_decode_err);
            count = new_tokens(a, b);
            edge = S::GRAN + max(0, len - 1 - first_new);
        }
        // granules of this warp: tokens tau * TILE + warp * GRAN, tau in [t0, t1), while below len
        tok0 = t0 * S::TILE + warp * S::GRAN;
        ng = tok0 >= len ? 0 : min(t1 - t0, (len - tok0 + S::TILE - 1) / S::TILE);
        return true;
    };
    uint32_t bad;                                    // halves (2 bits a stage) whose page is not one
    uint32_t qb[NH][KS][2];                          // q: column g of the products' second operand
    int next[2][HALVES];                             // pages of the granules that are loaded next
    auto look = [&](int j, int (&to)[HALVES]) {
        const int *table = a.c.table + static_cast<size_t>(b) * a.c.max_pages;
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf) {
            const int t = tok0 + j * S::TILE + hf * 16;
            to[hf] = t < len ? __ldg(table + kv_page_of(a.c, t)) : 0;
        }
    };
    auto load = [&](int j, int stage) {
        const int tok = tok0 + j * S::TILE;
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf) {
            const int t = tok + hf * 16;
            const int left = len - t;
            int page = next[0][hf];
            next[0][hf] = next[1][hf];
            if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.c.pages)) {
                atomicOr(&g_decode_err, 1u);
                page = -1;
            }
            const int nv = page < 0 ? 0 : max(0, min(16, left));
            const uint32_t bit = 1u << (stage * 2 + hf);
            bad = page < 0 ? bad | bit : bad & ~bit;
            const size_t row = nv == 0 ? 0 : kv_row(a.c, page, hk, t);
            const uint8_t *k = static_cast<const uint8_t *>(a.c.K) + row * S::ROW + lane * 16;
            const uint8_t *v = static_cast<const uint8_t *>(a.c.V) + row * S::ROW + lane * 16;
            const uint32_t dst = load_lane + stage * S::STAGE + hf * HALF;
            if (nv == 16) {
                load_half<D, KIND>(dst, dst + S::GRAN * S::ROW, k, v, std::make_integer_sequence<int, HALF / 512>());
            } else {
                // rows past the end are zeros: what the pool holds there is never looked at
                const uint32_t k0 = smem_u32(ring) + stage * S::STAGE + hf * HALF;
#pragma unroll
                for (int i = 0; i < HALF / 512; ++i) {
                    const int r = i * (32 / S::CPR) + lane / S::CPR;
                    const uint32_t at = k0 + chunk_at<D, KIND>(r, lane % S::CPR);
                    const uint8_t *ks = r < nv ? k + i * 512 : static_cast<const uint8_t *>(a.c.K);
                    const uint8_t *vs = r < nv ? v + i * 512 : static_cast<const uint8_t *>(a.c.V);
                    cp_async16(at, ks, r < nv);
                    cp_async16(at + S::GRAN * S::ROW, vs, r < nv);
                }
            }
            if constexpr (BLOCK) {
                // the 16 rows share a scale: one word each for K and V
                const float *sc = (lane == 0 ? a.c.sK : a.c.sV) + (row >> a.c.block_shift);
                const uint32_t at = smem_u32(ring) + stage * S::STAGE + 2 * S::GRAN * S::ROW + (lane * S::GRAN + hf * 16) * 4;
                if (lane < 2) cp_async4(at, sc, nv > 0);
            } else if constexpr (KIND >= 2) {
                const int r = lane & 15;
                const float *sc = (lane < 16 ? a.c.sK : a.c.sV) + row;
                const uint32_t at = smem_u32(ring) + stage * S::STAGE + 2 * S::GRAN * S::ROW + ((lane >> 4) * S::GRAN + hf * 16 + r) * 4;
                cp_async4(at, sc + (r < nv ? r : 0), r < nv);
            }
        }
        look(j + 2, next[1]);
    };
    // A pair's first reads, all on their way together: q, the pages of two granules, the ring's rows.
    // The ring has to be idle.
    auto begin = [&]() {
        look(0, next[0]);
        look(1, next[1]);
        // 16 bits: k = 2q (+ 8 half) of step ks are channels ks * 16 + 2q (+ 8 half), as ldmatrix deals K's
        // rows out; 8 bits: channels 16 (q + 4 jj) + 4 i + 2 half of step 4 jj + i, 32 consecutive bytes a lane
        const uint32_t *Q = static_cast<const uint32_t *>(a.Q) + (static_cast<size_t>(b) * a.Hq + head0) * (D / 2);
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            const bool is = g + 8 * nh < heads;
            const uint32_t *row = Q + (is ? (g + 8 * nh) * (D / 2) : 0);
            if constexpr (KIND < 2) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int half = 0; half < 2; ++half) qb[nh][ks][half] = is ? __ldg(row + ks * 8 + q + half * 4) : 0u;
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ks += 2) {
                    const uint4 w = is ? __ldg(reinterpret_cast<const uint4 *>(row + 8 * (q + ks / 4 * 4) + 2 * (ks & 3))) : make_uint4(0u, 0u, 0u, 0u);
                    qb[nh][ks][0] = w.x;
                    qb[nh][ks][1] = w.y;
                    qb[nh][ks + 1][0] = w.z;
                    qb[nh][ks + 1][1] = w.w;
                }
            }
        }
        bad = 0;
#pragma unroll
        for (int j = 0; j < S::STAGES - 1; ++j) {
            if (j < ng) load(j, j);
            cp_commit();
        }
    };

    if (!find()) return;
    begin();
    for (bool run_first = true;; run_first = false) {
        float qs[NH][2];                                         // log2 units' factor of heads 2q, 2q + 1
        {
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
                qs[nh][0] = qs[nh][1] = a.sl2;
                if constexpr (KIND >= 2) {
                    // to fp16 under a power of two a head: the largest value lands in [2^14, 2^15)
                    float mx = 0.0f;
                    auto pair_of = [&](uint32_t x) {
                        return a.bf16 ? __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&x))
                                      : __half22float2(*reinterpret_cast<__half2 *>(&x));
                    };
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const float2 f = pair_of(qb[nh][ks][half]);
                            mx = max3f(mx, fabsf(f.x), fabsf(f.y));
                        }
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    // exponent of the largest, held to [-100, 127] so that both factors are normal
                    const int e = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100);
                    const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
                    const float down = a.sl2 * __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const float2 f = pair_of(qb[nh][ks][half]);
                            qb[nh][ks][half] = pack_half2(f.x * up, f.y * up);
                        }
                    qs[nh][0] = __shfl_sync(0xffffffffu, down, 8 * q);           // lane (g = 2q, 0)
                    qs[nh][1] = __shfl_sync(0xffffffffu, down, 8 * q + 4);
                }
            }
        }

        float acc[KS][NH][4];                                    // channels (rows g, g + 8) x heads (2q, 2q + 1)
        float m[NH][2], l[NH][2];
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][nh][i] = 0.0f;
            m[nh][0] = m[nh][1] = -INFINITY;
            l[nh][0] = l[nh][1] = 0.0f;
        }

        int stage = 0, ahead = S::STAGES - 1;                    // stages of granules j and j + STAGES - 1
        for (int j = 0; j < ng; ++j) {
            cp_wait<S::STAGES - 2>();
            __syncwarp();
            if (j + S::STAGES - 1 < ng) load(j + S::STAGES - 1, ahead);
            cp_commit();
            const uint8_t *kst = ring + stage * S::STAGE, *vst = kst + S::GRAN * S::ROW;
            const int tok = tok0 + j * S::TILE;
            const uint32_t holes = (bad >> (stage * 2)) & 3u;

            // S = K q: tokens hf * 16 + g (i = 0, 1) and + 8 (2, 3), heads nh * 8 + 2q (0, 2) and + 1 (1, 3)
            float s[HALVES][NH][4];
#pragma unroll
            for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
                for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[hf][nh][i] = 0.0f;
            if constexpr (KIND < 2) {
                const uint32_t at = smem_u32(kst) + chunk_at<D, KIND>(lane & 15, lane >> 4);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int hf = 0; hf < HALVES; ++hf) {
                        uint32_t ka[4];
                        ldsm4((at ^ (ks * 32)) + hf * HALF, ka);
#pragma unroll
                        for (int nh = 0; nh < NH; ++nh) mma16816<BF16>(s[hf][nh], ka, qb[nh][ks][0], qb[nh][ks][1]);
                    }
            } else {
                const uint32_t at = chunk_at<D, KIND>(g, q);     // rows 8 apart are 8 * ROW apart
#pragma unroll
                for (int jj = 0; jj < D / 64; ++jj)
#pragma unroll
                    for (int hf = 0; hf < HALVES; ++hf) {
                        const uint8_t *from = kst + (at ^ (jj * 64)) + hf * HALF;
                        const uint4 k0 = *reinterpret_cast<const uint4 *>(from), k1 = *reinterpret_cast<const uint4 *>(from + 8 * S::ROW);
                        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t ka[4];
                            widen4<false, KIND == 3>(w0[i], ka[0], ka[2]);
                            widen4<false, KIND == 3>(w1[i], ka[1], ka[3]);
#pragma unroll
                            for (int nh = 0; nh < NH; ++nh)
                                mma16816<false>(s[hf][nh], ka, qb[nh][4 * jj + i][0], qb[nh][4 * jj + i][1]);
                        }
                    }
            }
            // log2 units; tokens past the end of the sequence, or without a page, do not exist
            float fv[HALVES][2];                                 // sV of the lane's tokens
#pragma unroll
            for (int hf = 0; hf < HALVES; ++hf) {
                float fk[2] = {1.0f, 1.0f};
                if constexpr (KIND >= 2) {
                    const float *sc = reinterpret_cast<const float *>(kst + 2 * S::GRAN * S::ROW) + hf * 16 + (BLOCK ? 0 : g);
                    constexpr int next_row = BLOCK ? 0 : 8;
                    fk[0] = sc[0];
                    fk[1] = sc[next_row];
                    fv[hf][0] = sc[S::GRAN];
                    fv[hf][1] = sc[S::GRAN + next_row];
                }
#pragma unroll
                for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (KIND >= 2) s[hf][nh][i] *= fk[i >> 1];
                        s[hf][nh][i] *= qs[nh][i & 1];
                    }
            }
            const bool hidden = ROWS && len - tok < edge;
            if (ROWS && hidden) {
                // several tokens: each row ends at a slot of its own
                int limit[NH][2];
#pragma unroll
                for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                    for (int e = 0; e < 2; ++e) limit[nh][e] = row_limit(a, head0 - hk * a.G + nh * 8 + 2 * q + e, first_new, count, len) - tok;
#pragma unroll
                for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
                    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (hf * 16 + g + 8 * (i >> 1) >= limit[nh][i & 1] || (holes >> hf) & 1u) s[hf][nh][i] = -INFINITY;
                // 0 times a V that is not finite would reach the rows that do not see it: it is taken out, and
                // added at the end to those that do (INT8 codes are finite)
                if constexpr (KIND != 2) {
                    uint32_t bad = 0;
                    for (int i = lane; i < S::GRAN * S::ROW / 16; i += 32) {
                        uint4 *at = reinterpret_cast<uint4 *>(const_cast<uint8_t *>(vst)) + i;
                        const uint4 w = *at;
                        const uint32_t m0 = not_finite_mask<KIND == 1, KIND == 3>(w.x), m1 = not_finite_mask<KIND == 1, KIND == 3>(w.y);
                        const uint32_t m2 = not_finite_mask<KIND == 1, KIND == 3>(w.z), m3 = not_finite_mask<KIND == 1, KIND == 3>(w.w);
                        if (m0 | m1 | m2 | m3) *at = make_uint4(w.x & ~m0, w.y & ~m1, w.z & ~m2, w.w & ~m3);
                        bad |= m0 | m1 | m2 | m3;
                    }
                    if (bad) s_not_finite = 1;
                    __syncwarp();
                }
            } else if (len - tok < S::GRAN || holes) {
#pragma unroll
                for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (hf * 16 + g + 8 * (i >> 1) >= len - tok || (holes >> hf) & 1u) {
#pragma unroll
                            for (int nh = 0; nh < NH; ++nh) s[hf][nh][i] = -INFINITY;
                        }
            }
            if (a.logits) {
#pragma unroll
                for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int head = nh * 8 + 2 * q + (i & 1);
                        float *to = a.logits + (static_cast<size_t>(b) * a.Hq + head0 + head) * a.c.cap + tok + g + 8 * (i >> 1);
#pragma unroll
                        for (int hf = 0; hf < HALVES; ++hf)
                            if (head < heads && len - tok > hf * 16) to[hf * 16] = s[hf][nh][i];   // (slots up to the next multiple of 16 exist)
                    }
            }
            float alpha[NH][2];
#pragma unroll
            for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(s[0][nh][e], s[0][nh][2 + e]);
#pragma unroll
                    for (int hf = 1; hf < HALVES; ++hf) mx = max3f(mx, s[hf][nh][e], s[hf][nh][2 + e]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float mn = fmaxf(m[nh][e], mx);
                    const float ref = mn == -INFINITY ? 0.0f : mn;   // nothing seen yet: all terms are 0
                    alpha[nh][e] = ex2_approx(m[nh][e] - ref);
                    m[nh][e] = mn;
                    float sum = 0.0f;
#pragma unroll
                    for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float &x = s[hf][nh][2 * i + e];
                            x = ex2_approx(x - ref);
                            sum += x;
                        }
                    l[nh][e] = l[nh][e] * alpha[nh][e] + sum;
                }
            if constexpr (KIND >= 2) {
                if (ROWS && hidden) {                                // (a hidden slot's scale may be anything)
#pragma unroll
                    for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
                        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (s[hf][nh][i] != 0.0f) s[hf][nh][i] *= fv[hf][i >> 1];
                } else {
#pragma unroll
                    for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
                        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                            for (int i = 0; i < 4; ++i) s[hf][nh][i] *= fv[hf][i >> 1];
                }
            }
            bool moved = false;
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) moved = moved || alpha[nh][0] != 1.0f || alpha[nh][1] != 1.0f;
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                    for (int jn = 0; jn < KS; ++jn) {
                        acc[jn][nh][0] *= alpha[nh][0]; acc[jn][nh][1] *= alpha[nh][1];
                        acc[jn][nh][2] *= alpha[nh][0]; acc[jn][nh][3] *= alpha[nh][1];
                    }
            }
#pragma unroll
            for (int hf = 0; hf < HALVES; ++hf) {
                if constexpr (TF32) {
                    uint32_t ph[NH][4], pl[NH][4];               // hi, lo: tokens 2q, 2q + 1, 2q + 8, 2q + 9 of head g
#pragma unroll
                    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                        for (int x = 0; x < 4; x += 2) {
                            transpose8(s[hf][nh][x], s[hf][nh][x + 1]);
                            split11(s[hf][nh][x], ph[nh][x], pl[nh][x]);
                            split11(s[hf][nh][x + 1], ph[nh][x + 1], pl[nh][x + 1]);
                        }
                    const uint32_t at = smem_u32(vst) + hf * HALF + chunk_at<D, KIND>((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
#pragma unroll
                    for (int jn = 0; jn < KS; ++jn) {
                        uint32_t va[4];
                        ldsm4t(at ^ (jn * 32), va);
#pragma unroll
                        for (int x = 0; x < 4; x += 2) {
                            // rows g, g + 8; the products' rows q and q + 4 of the second dimension are tokens 2q and 2q + 1
                            const float2 v0 = __half22float2(*reinterpret_cast<const __half2 *>(&va[x]));
                            const float2 v1 = __half22float2(*reinterpret_cast<const __half2 *>(&va[x + 1]));
                            const uint32_t a0 = __float_as_uint(v0.x), a1 = __float_as_uint(v1.x), a2 = __float_as_uint(v0.y), a3 = __float_as_uint(v1.y);
#pragma unroll
                            for (int nh = 0; nh < NH; ++nh) mma1688(acc[jn][nh], a0, a1, a2, a3, ph[nh][x], ph[nh][x + 1]);
#pragma unroll
                            for (int nh = 0; nh < NH; ++nh) mma1688(acc[jn][nh], a0, a1, a2, a3, pl[nh][x], pl[nh][x + 1]);
                        }
                    }
                } else {
                    uint32_t ph[NH][2], pl[NH][2];                   // hi, lo: tokens 2q, 2q + 1 (+ 8) of head g
#pragma unroll
                    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            split2(s[hf][nh][2 * x], s[hf][nh][2 * x + 1], ph[nh][x], pl[nh][x]);
                            ph[nh][x] = transpose8(ph[nh][x]);
                            pl[nh][x] = transpose8(pl[nh][x]);
                        }
                    auto pv = [&](int jn, const uint32_t (&va)[4]) {
#pragma unroll
                        for (int nh = 0; nh < NH; ++nh) mma16816<true>(acc[jn][nh], va, ph[nh][0], ph[nh][1]);
#pragma unroll
                        for (int nh = 0; nh < NH; ++nh) mma16816<true>(acc[jn][nh], va, pl[nh][0], pl[nh][1]);
                    };
                    if constexpr (KIND < 2) {
                        const uint32_t at = smem_u32(vst) + hf * HALF + chunk_at<D, KIND>((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
#pragma unroll
                        for (int jn = 0; jn < KS; ++jn) {
                            uint32_t va[4];
                            ldsm4t(at ^ (jn * 32), va);
                            pv(jn, va);
                        }
                    } else {
                        // tokens 2q, 2q + 1, 2q + 8, 2q + 9; row g of tile jn is channel D / 8 g + 2 jn, row g + 8 the next
                        constexpr int W = D / 32;
                        uint32_t x[4][W];
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const uint8_t *at = vst + hf * HALF + (t >> 1) * 8 * S::ROW;
                            if constexpr (D == 128) {
                                const uint4 v = *reinterpret_cast<const uint4 *>(at + chunk_at<D, KIND>(2 * q + (t & 1), g));
                                x[t][0] = v.x; x[t][1] = v.y; x[t][2] = v.z; x[t][3] = v.w;
                            } else {
                                const uint2 v = *reinterpret_cast<const uint2 *>(at + chunk_at<D, KIND>(2 * q + (t & 1), g >> 1) + (g & 1) * 8);
                                x[t][0] = v.x; x[t][1] = v.y;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            uint32_t va[2][4];
                            widen4<true, KIND == 3>(prmt(x[0][i], x[1][i], 0x5140), va[0][0], va[0][1]);
                            widen4<true, KIND == 3>(prmt(x[2][i], x[3][i], 0x5140), va[0][2], va[0][3]);
                            widen4<true, KIND == 3>(prmt(x[0][i], x[1][i], 0x7362), va[1][0], va[1][1]);
                            widen4<true, KIND == 3>(prmt(x[2][i], x[3][i], 0x7362), va[1][2], va[1][3]);
                            pv(2 * i, va[0]);
                            pv(2 * i + 1, va[1]);
                        }
                    }
                }
            }
            stage = stage + 1 == S::STAGES ? 0 : stage + 1;
            ahead = ahead + 1 == S::STAGES ? 0 : ahead + 1;
        }
        cp_wait<0>();
        __syncwarp();

        // what the end of this pair needs, and the next pair's first reads on their way meanwhile
        const bool whole = t0 == 0 && t1 == tiles;
        // a run's first pair that began in an earlier run goes to place 0, one that goes on to place 1
        const int place = run_first && t0 > 0 ? 0 : 1;
        const size_t out0 = static_cast<size_t>(b) * a.Hq + head0;
        const int outs = heads;
        // (of this pair, for values that are not finite: its sequence, kv head, and the slots of its tiles)
        if constexpr (ROWS) {
            if (tid < MR) s_limit[tid] = row_limit(a, head0 - hk * a.G + tid, first_new, count, len);
        }
        [[maybe_unused]] const int pb = b, pk = hk, pfrom = max(t0 * S::TILE, edge >= len ? 0 : len - edge), pto = t1 * S::TILE;
        bool more = false;
        if constexpr (!ONE) {
            more = find();
            if (more) begin();
        }

        // join the four warps, in their order
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[nh][e] += __shfl_xor_sync(0xffffffffu, l[nh][e], o);
                if (g == 0) {
                    s_m[warp][nh * 8 + 2 * q + e] = m[nh][e];
                    s_l[warp][nh * 8 + 2 * q + e] = l[nh][e];
                }
            }
        // Each warp's sums, (MR, D) floats, in the last stage of its own ring.  Heads PITCH apart, and in 8 bits the
        // channels in the order (k, g) of D / 8 g + k, put a store's 32 lanes into 32 banks.
        constexpr int PITCH = D + 4;
        constexpr int SUMS = (S::STAGES - 1) * S::STAGE;
        static_assert(SUMS + MR * PITCH * 4 <= S::RING, "the sums do not fit the last stage");
        float *so = reinterpret_cast<float *>(ring + SUMS);
#pragma unroll
        for (int jn = 0; jn < KS; ++jn)
#pragma unroll
            for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    so[(nh * 8 + 2 * q + (i & 1)) * PITCH + jn * 16 + 8 * (i >> 1) + g] = acc[jn][nh][i];
        __syncthreads();
        // ONE: the CTA's sums, (MR, D) floats, in the first stage of the first ring
        float *sums = reinterpret_cast<float *>(smem);
        static_assert(MR * D * 4 <= S::STAGE && S::STAGES > 1, "the sums do not fit a stage");
        for (int idx = tid; idx < outs * (D / 2); idx += kDecThreads) {
            const int r = idx / (D / 2), x2 = idx % (D / 2);
            // two channels c, c + 1 and their places
            const int c = KIND < 2 ? 2 * x2 : D / 8 * (x2 & 7) + 2 * (x2 >> 3);
            const int p0 = r * PITCH + (KIND < 2 ? c : 16 * (x2 >> 3) + (x2 & 7)), p1 = p0 + (KIND < 2 ? 1 : 8);
            float M = -INFINITY;
#pragma unroll
            for (int x = 0; x < kDecWarps; ++x) M = fmaxf(M, s_m[x][r]);
            const float ref = M == -INFINITY ? 0.0f : M;
            float o0 = 0.0f, o1 = 0.0f, sum = 0.0f;
#pragma unroll
            for (int x = 0; x < kDecWarps; ++x) {
                const float f = ex2_approx(s_m[x][r] - ref);
                const float *from = reinterpret_cast<const float *>(smem + x * S::RING + SUMS);
                o0 += f * from[p0];
                o1 += f * from[p1];
                sum += f * s_l[x][r];
            }
            if constexpr (ROWS) {
                // a row behind its sequence's last token has seen what it was not hidden from
                if (s_limit[r] == 0) {
                    o0 = o1 = sum = 0.0f;
                    M = -INFINITY;
                }
            }
            if constexpr (ROWS && KIND != 2) {
                if (s_not_finite) {
                    const int to = min(s_limit[r], pto);
                    for (int t = pfrom; t < to; ++t) {
                        const int p = kv_page(a.c, pb, t, &g_decode_err);
                        if (p < 0) continue;
                        const float2 v = value_pair<KIND>(a.c.V, kv_row(a.c, p, pk, t) * D + c);
                        if (!(fabsf(v.x) < INFINITY)) o0 += v.x;
                        if (!(fabsf(v.y) < INFINITY)) o1 += v.y;
                    }
                }
            }
            if constexpr (ONE) {
                *reinterpret_cast<float2 *>(sums + r * D + c) = make_float2(o0, o1);
                if (c == 0) {
                    s_part[0][r] = M;
                    s_part[1][r] = sum;
                }
                continue;
            }
            const size_t head = out0 + r;
            if (whole) {
                const float inv = inv_of(sum);
                store_out(a, head * D + c, o0 * inv, o1 * inv);
                if (c == 0) {
                    a.L[head] = lse_of(M, sum);
                    if (a.row_ml) {
                        a.row_ml[2 * head] = M;
                        a.row_ml[2 * head + 1] = sum;
                    }
                }
            } else {
                const size_t at = (static_cast<size_t>(cta) * 2 + place) * MR + r;
                *reinterpret_cast<float2 *>(a.part_O + at * D + c) = make_float2(o0, o1);
                if (c == 0) {
                    a.part_ml[2 * at] = M;
                    a.part_ml[2 * at + 1] = sum;
                }
            }
        }
        if constexpr (ONE) {
            // the cluster's sums: each head's M and 1 / l, then a share of the outputs for each CTA
            cluster_sync();
            float M = -INFINITY, sum = 0.0f;
            if (tid < outs) {
                float ml[kDecCluster][2];
#pragma unroll
                for (int k = 0; k < kDecCluster; ++k)
                    if (k < a.cluster) {
                        ml[k][0] = cluster_float(&s_part[0][tid], k);
                        ml[k][1] = cluster_float(&s_part[1][tid], k);
                        M = fmaxf(M, ml[k][0]);
                    }
                const float ref = M == -INFINITY ? 0.0f : M;
#pragma unroll
                for (int k = 0; k < kDecCluster; ++k)
                    if (k < a.cluster) {
                        const float f = ex2_approx(ml[k][0] - ref);
                        s_f[k][tid] = f;
                        sum += f * ml[k][1];
                    }
                s_m[0][tid] = ref;
                s_l[0][tid] = inv_of(sum);
                if (rank == 0) a.L[out0 + tid] = lse_of(M, sum);
            }
            __syncthreads();
            for (int i = (rank * kDecThreads + tid) * 4; i < outs * D; i += a.cluster * kDecThreads * 4) {
                const int r = i / D;
                float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < kDecCluster; ++k)
                    if (k < a.cluster) {
                        const int4 w4 = cluster_words(reinterpret_cast<const int *>(sums + i), k);
                        const float f = s_f[k][r];
                        o.x += f * __int_as_float(w4.x); o.y += f * __int_as_float(w4.y);
                        o.z += f * __int_as_float(w4.z); o.w += f * __int_as_float(w4.w);
                    }
                const float inv = s_l[0][r];
                store_out(a, out0 * D + i, o.x * inv, o.y * inv);
                store_out(a, out0 * D + i + 2, o.z * inv, o.w * inv);
            }
            if (a.logits) {
                // scores of this CTA's own tokens (one group of heads a kv head), heads in order
                float *score = a.c.score + (static_cast<size_t>(b) * a.c.H + hk) * a.c.cap;
                const int end = min(len, t1 * S::TILE);
                for (int t = t0 * S::TILE + tid; t < end; t += kDecThreads) {
                    float w = 0.0f;
                    for (int r = 0; r < outs; ++r) w += ex2_approx(a.logits[(out0 + r) * a.c.cap + t] - s_m[0][r]) * s_l[0][r];
                    score[t] += w;
                }
            }
            cluster_sync();                                      // no CTA leaves while its sums are read
            return;
        }
        if (!more) break;
        __syncthreads();                                         // before the last stage is filled again
    }
}

// ---- join ---------------------------------------------------------------------------------------
// A pair that several runs share is the sum of their parts, each under 2^(m_part - M), in their
// order.  Launched while the main kernel still runs (programmatic dependent launch): the lengths
// are added up before the wait for its end, which every block does, work or none: what is launched
// after this kernel then comes after the main kernel too.
constexpr int kJoinThreads = 256;

// The runs c0 .. c1 that hold tiles of the pair whose first unit is p0; part c is in place 1 of the
// first, place 0 of the others.
__device__ __forceinline__ void runs_of_pair(long long total, int runs, long long p0, int tiles, int &c0, int &c1) {
    c0 = run_of(total, p0 + kPairUnits, runs);
    c1 = run_of(total, p0 + kPairUnits + tiles - 1, runs);
}
__device__ __forceinline__ size_t part_of(int c, int c0, int mr, int r) {
    return (static_cast<size_t>(c) * 2 + (c == c0 ? 1 : 0)) * mr + r;
}

// M and the sum over parts c0 .. c1 of row r, by a warp
__device__ __forceinline__ float2 join_ml(const DecodeArgs &a, int c0, int c1, int mr, int r, int lane) {
    float M = -INFINITY, sum = 0.0f;                 // a lane's parts under its own maximum first
    for (int c = c0 + lane; c <= c1; c += 32) {
        const float2 ml = reinterpret_cast<const float2 *>(a.part_ml)[part_of(c, c0, mr, r)];
        const float mn = fmaxf(M, ml.x), to = mn == -INFINITY ? 0.0f : mn;
        sum = sum * ex2_approx(M - to) + ml.y * ex2_approx(ml.x - to);
        M = mn;
    }
    const float mine = M;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    sum *= ex2_approx(mine - (M == -INFINITY ? 0.0f : M));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return make_float2(M, sum);
}

// grid: (pairs, heads of a group) with at most as many pairs as runs, one head a block, its threads
// over the parts; or (runs, 1), where the block of run c joins the pair that starts in run c and
// goes on, if there is one: few parts, its threads over the heads.
template <int D, int MR, bool PAIRS, bool ROWS>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const __grid_constant__ DecodeArgs a) {
    constexpr int VEC = D / 4, GROUPS = kJoinThreads / VEC;
    __shared__ float4 s_o[GROUPS][VEC];
    __shared__ float s_M[MR], s_inv[MR];
    __shared__ long long s_lo[kJoinThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int v = tid % VEC, grp = tid / VEC;
    const int pairs = a.c.H * a.chunks;
    int b = 0, pair = 0, c0 = 0, c1 = 0;             // c0 == c1: nothing to join
    if constexpr (PAIRS) {
        b = blockIdx.x / pairs;
        pair = blockIdx.x - b * pairs;
        long long lo = 0;                            // units of the sequences before
        for (int i = tid; i < b; i += kJoinThreads) lo += static_cast<long long>(pair_units<ROWS>(a, i)) * pairs;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lo += __shfl_xor_sync(0xffffffffu, lo, o);
        if (lane == 0) s_lo[warp] = lo;
        const WorkAt w = locate<kJoinThreads, ROWS>(a, pairs, [](long long total) { return total; });
        lo = 0;
#pragma unroll
        for (int x = 0; x < kJoinThreads / 32; ++x) lo += s_lo[x];
        const int units = pair_units<ROWS>(a, b);
        if (units > 0)
            runs_of_pair(w.total, runs_of(a, w.total), lo + static_cast<long long>(pair) * units, units - kPairUnits, c0, c1);
    } else {
        const int c = blockIdx.x;
        const WorkAt w = locate<kJoinThreads, ROWS>(a, pairs, [&](long long total) {
            const int n = runs_of(a, total);
            return c + 1 < n ? run_start(total, c + 1, n) - 1 : total;
        });
        if (w.u < w.total) {
            b = w.b;
            const int units = pair_units<ROWS>(a, b);
            pair = static_cast<int>(div_up_to(w.u - w.first, units));
            runs_of_pair(w.total, runs_of(a, w.total), w.first + static_cast<long long>(pair) * units, units - kPairUnits, c0, c1);
            if (c0 != c) c0 = c1;                    // another block's
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c0 == c1) return;
    const int hk = pair / a.chunks, ch = pair - hk * a.chunks;
    const int heads = min(MR, a.G - ch * MR);
    const size_t head0 = static_cast<size_t>(b) * a.Hq + hk * a.G + ch * MR;
    if (PAIRS && static_cast<int>(blockIdx.y) >= heads) return;
    // (PAIRS: a thread's first parts are asked for before the maximum is known)
    constexpr int EARLY = PAIRS ? 8 : 1;
    float4 part[EARLY];
    float part_m[EARLY];
    if constexpr (PAIRS) {
#pragma unroll
        for (int x = 0; x < EARLY; ++x) {
            const int c = c0 + grp + x * GROUPS;
            part[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            part_m[x] = -INFINITY;
            if (c > c1) continue;
            const size_t at = part_of(c, c0, MR, blockIdx.y);
            part[x] = reinterpret_cast<const float4 *>(a.part_O + at * D)[v];
            part_m[x] = a.part_ml[2 * at];
        }
    }
    for (int r = PAIRS ? blockIdx.y + warp * MR : warp; r < heads; r += PAIRS ? MR * kJoinThreads : kJoinThreads / 32) {
        const float2 ml = join_ml(a, c0, c1, MR, r, lane);
        if (lane == 0) {
            s_M[r] = ml.x == -INFINITY ? 0.0f : ml.x;
            s_inv[r] = inv_of(ml.y);
            a.L[head0 + r] = lse_of(ml.x, ml.y);
        }
    }
    __syncthreads();
    // a thread's four channels of row r from parts c, c + step, ...
    auto sums = [&](int r, int c, int step) {
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (; c <= c1; c += step) {
            const size_t at = part_of(c, c0, MR, r);
            const float f = ex2_approx(a.part_ml[2 * at] - s_M[r]);
            const float4 x = reinterpret_cast<const float4 *>(a.part_O + at * D)[v];
            o.x += f * x.x; o.y += f * x.y; o.z += f * x.z; o.w += f * x.w;
        }
        return o;
    };
    auto store = [&](int r, float4 o) {
        const float inv = s_inv[r];
        store_out(a, (head0 + r) * D + v * 4, o.x * inv, o.y * inv);
        store_out(a, (head0 + r) * D + v * 4 + 2, o.z * inv, o.w * inv);
    };
    if constexpr (PAIRS) {
        const int r = blockIdx.y;
        float4 o = sums(r, c0 + grp + EARLY * GROUPS, GROUPS);
#pragma unroll
        for (int x = 0; x < EARLY; ++x) {
            const float f = ex2_approx(part_m[x] - s_M[r]);
            o.x += f * part[x].x; o.y += f * part[x].y; o.z += f * part[x].z; o.w += f * part[x].w;
        }
        s_o[grp][v] = o;
        __syncthreads();
        if (tid < VEC) {
            o = s_o[0][v];
#pragma unroll
            for (int x = 1; x < GROUPS; ++x) {
                const float4 y = s_o[x][v];
                o.x += y.x; o.y += y.y; o.z += y.z; o.w += y.w;
            }
            store(r, o);
        }
    } else {
        for (int r = grp; r < heads; r += GROUPS) store(r, sums(r, c0, 1));
    }
}

// ---- join and scores ----------------------------------------------------------------------------
// grid: (sequences * kv heads, blocks of 1024 slots at a time), in place of the join.  Every block forms M and l of
// its kv head's query heads, a warp each, from the parts or (whole pairs) from what the main kernel
// left; blocks 0, 1, ... take the output rows of the shared pairs in turn; then
// score[b][hk][t] += sum over the heads of 2^(logit - M) / l, from the logits that the main kernel kept:
// four slots a thread, heads in order.
constexpr int kScoreHeads = 64;              // heads whose M and 1 / l are held at a time

template <int D, int MR>
__global__ void __launch_bounds__(kJoinThreads) decode_score_kernel(const __grid_constant__ DecodeArgs a) {
    constexpr bool ROWS = false;
    constexpr int VEC = D / 4, GROUPS = kJoinThreads / VEC;
    __shared__ float4 s_o[GROUPS][VEC];
    __shared__ float s_M[kScoreHeads], s_inv[kScoreHeads];
    __shared__ long long s_lo[kJoinThreads / 32];
    const int bh = blockIdx.x, b = bh / a.c.H, hk = bh - b * a.c.H, y = blockIdx.y, ys = gridDim.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int v = tid % VEC, grp = tid / VEC;
    const int pairs = a.c.H * a.chunks;
    const int len = seq_len<ROWS>(a, b);
    const size_t head0 = static_cast<size_t>(b) * a.Hq + static_cast<size_t>(hk) * a.G;
    const bool idle = len == 0 || (y >= a.G && y * (kJoinThreads * 4) >= len);
    long long lo = 0;                                // units of the sequences before
    WorkAt w{};
    if (!idle) {
        for (int i = tid; i < b; i += kJoinThreads) lo += static_cast<long long>(pair_units<ROWS>(a, i)) * pairs;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lo += __shfl_xor_sync(0xffffffffu, lo, o);
        if (lane == 0) s_lo[warp] = lo;
        w = locate<kJoinThreads, ROWS>(a, pairs, [](long long total) { return total; });
        lo = 0;
#pragma unroll
        for (int x = 0; x < kJoinThreads / 32; ++x) lo += s_lo[x];
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");       // by every block, as above
    if (idle) return;
    const int units = pair_units<ROWS>(a, b), runs = runs_of(a, w.total);
    for (int h0 = 0; h0 < a.G; h0 += kScoreHeads) {
        const int n = min(kScoreHeads, a.G - h0);
        for (int i = warp; i < n; i += kJoinThreads / 32) {
            const int h = h0 + i, ch = h / MR, r = h - ch * MR;
            int c0, c1;
            runs_of_pair(w.total, runs, lo + (static_cast<long long>(hk) * a.chunks + ch) * units, units - kPairUnits, c0, c1);
            float2 ml;
            if (c0 == c1) {
                ml = reinterpret_cast<const float2 *>(a.row_ml)[head0 + h];
            } else {
                ml = join_ml(a, c0, c1, MR, r, lane);
                if (lane == 0 && h % ys == y) a.L[head0 + h] = lse_of(ml.x, ml.y);
            }
            if (lane == 0) {
                s_M[i] = ml.x == -INFINITY ? 0.0f : ml.x;
                s_inv[i] = inv_of(ml.y);
            }
        }
        __syncthreads();
        for (int i = (y - h0 % ys + ys) % ys; i < n; i += ys) {      // heads h = y, y + ys, ...
            const int h = h0 + i, ch = h / MR, r = h - ch * MR;
            int c0, c1;
            runs_of_pair(w.total, runs, lo + (static_cast<long long>(hk) * a.chunks + ch) * units, units - kPairUnits, c0, c1);
            if (c0 == c1) continue;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
            for (int c = c0 + grp; c <= c1; c += GROUPS) {
                const size_t at = part_of(c, c0, MR, r);
                const float f = ex2_approx(a.part_ml[2 * at] - s_M[i]);
                const float4 x = reinterpret_cast<const float4 *>(a.part_O + at * D)[v];
                o.x += f * x.x; o.y += f * x.y; o.z += f * x.z; o.w += f * x.w;
            }
            s_o[grp][v] = o;
            __syncthreads();
            if (tid < VEC) {
                o = s_o[0][v];
#pragma unroll
                for (int x = 1; x < GROUPS; ++x) {
                    const float4 z = s_o[x][v];
                    o.x += z.x; o.y += z.y; o.z += z.z; o.w += z.w;
                }
                const float inv = s_inv[i];
                store_out(a, (head0 + h) * D + v * 4, o.x * inv, o.y * inv);
                store_out(a, (head0 + h) * D + v * 4 + 2, o.z * inv, o.w * inv);
            }
            __syncthreads();
        }
        for (int t = (y * kJoinThreads + tid) * 4; t < len; t += ys * kJoinThreads * 4) {
            const float *x = a.logits + (head0 + h0) * a.c.cap + t;
            float4 add = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float4 z = *reinterpret_cast<const float4 *>(x + static_cast<size_t>(i) * a.c.cap);
                const float M = s_M[i], inv = s_inv[i];
                add.x += ex2_approx(z.x - M) * inv;
                add.y += ex2_approx(z.y - M) * inv;
                add.z += ex2_approx(z.z - M) * inv;
                add.w += ex2_approx(z.w - M) * inv;
            }
            float *to = a.c.score + static_cast<size_t>(bh) * a.c.cap + t;
            if (t + 4 <= len) {
                float4 z = *reinterpret_cast<const float4 *>(to);
                z.x += add.x; z.y += add.y; z.z += add.z; z.w += add.w;
                *reinterpret_cast<float4 *>(to) = z;
            } else {                                 // slots past the end keep what they hold
                to[0] += add.x;
                if (t + 1 < len) to[1] += add.y;
                if (t + 2 < len) to[2] += add.z;
            }
        }
        __syncthreads();
    }
}

unsigned int take_decode_error() {
    unsigned int v = 0, zero = 0;
    cudaMemcpyFromSymbol(&v, g_decode_err, sizeof(v));
    cudaMemcpyToSymbol(g_decode_err, &zero, sizeof(zero));
    return v;
}

// ---- host -------------------------------------------------------------------------------------
constexpr int kDecOneTiles = 4;              // tiles a CTA of a pair's cluster takes at most

struct DecodePlan {
    int mr, chunks, ctas, tile;
    int cluster;             // not 0: a cluster a pair
    size_t off_ml, off_rows, off_logits, bytes;
};

static DecodePlan decode_plan(const sage_kv &c, int Hq, int add_score) {
    DecodePlan p;
    const int G = Hq / c.H;
    p.mr = G <= 8 ? 8 : 16;
    p.chunks = (G + p.mr - 1) / p.mr;
    const int row = c.d * (kv_format(c) == SAGE_KV_16 ? 2 : 1);
    // one resident wave; never more CTAs than there can be tiles
    p.tile = decode_tile(row);
    long long n = kSMs * decode_ctas(row, c.d, p.mr);
    const long long tiles = static_cast<long long>(c.B) * c.H * p.chunks * ((static_cast<long long>(c.max_pages) * c.page + p.tile - 1) / p.tile);
    // A cluster a pair while all pairs are resident together and a CTA takes few tiles: as many CTAs as
    // there are tiles and room.  (Device us in a graph, cluster / split: 8 pairs of 1000 tokens in INT8, d = 128
    // 5.9 / 8.0, of 4000, 4 tiles a CTA, 9.6 / 9.0, where the second launch costs the host 3; 64 pairs of up to
    // 4000, 8 tiles a CTA, 16.9 / 14.8; 256 of up to 300 8.4 / 14.0; 1024 of 64, more than are resident, 15.5 / 13.8.)
    const long long pairs = static_cast<long long>(c.B) * c.H * p.chunks, most = tiles / pairs;
    int cl = 1;
    while (cl < kDecCluster && cl < most && pairs * cl * 2 <= n) cl *= 2;
    p.cluster = pairs <= n && (most + cl - 1) / cl <= kDecOneTiles && (!add_score || p.chunks == 1) ? cl : 0;
    if (n > tiles) n = tiles;
    p.ctas = static_cast<int>(p.cluster ? pairs * cl : n);
    auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    const size_t parts = p.cluster ? 0 : static_cast<size_t>(p.ctas) * 2 * p.mr;
    const size_t heads = static_cast<size_t>(c.B) * Hq;
    p.off_ml = up(parts * c.d * sizeof(float));
    p.off_rows = p.off_ml + up(parts * 2 * sizeof(float));
    p.off_logits = p.off_rows + (add_score && !p.cluster ? up(heads * 2 * sizeof(float)) : 0);
    p.bytes = p.off_logits + (add_score ? heads * c.max_pages * c.page * sizeof(float) : 0);
    return p;
}

static int check_decode(const sage_kv *c, int Hq, int add_score) {
    const int st = check_kv(c, false);
    if (st != SAGE_OK) return st;
    if (Hq <= 0 || Hq % c->H != 0 || (add_score & ~1)) return SAGE_ERR_ARG;
    if (static_cast<long long>(c->B) * Hq > (1 << 24)) return SAGE_ERR_UNSUPPORTED;
    return SAGE_OK;
}

template <int D, int KIND, int MR, bool BLOCK, bool ROWS>
static cudaError_t launch_decode_k(const DecodeArgs &a, cudaStream_t st) {
    using S = DecodeShape<D, KIND, MR>;
    static bool raised[2][16] = {{false}};
    if (a.cluster) {
        const cudaError_t e = raise_smem(reinterpret_cast<const void *>(decode_kernel<D, KIND, MR, true, BLOCK, ROWS>), S::SMEM, raised[1]);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(a.ctas);
        cfg.blockDim = dim3(kDecThreads);
        cfg.dynamicSmemBytes = S::SMEM;
        cfg.stream = st;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = a.cluster;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, decode_kernel<D, KIND, MR, true, BLOCK, ROWS>, a);
    }
    cudaError_t e = raise_smem(reinterpret_cast<const void *>(decode_kernel<D, KIND, MR, false, BLOCK, ROWS>), S::SMEM, raised[0]);
    if (e != cudaSuccess) return e;
    decode_kernel<D, KIND, MR, false, BLOCK, ROWS><<<a.ctas, kDecThreads, S::SMEM, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (!ROWS && a.logits) {
        const int y = (a.c.cap + 4 * kJoinThreads - 1) / (4 * kJoinThreads);
        cfg.gridDim = dim3(static_cast<unsigned>(a.c.B) * a.c.H, y < 1024 ? y : 1024);
        return cudaLaunchKernelEx(&cfg, decode_score_kernel<D, MR>, a);
    }
    const long long pairs = static_cast<long long>(a.c.B) * a.c.H * a.chunks;
    if (pairs <= a.ctas) {
        cfg.gridDim = dim3(static_cast<unsigned>(pairs), a.G < MR ? a.G : MR);
        return cudaLaunchKernelEx(&cfg, decode_join_kernel<D, MR, true, ROWS>, a);
    }
    cfg.gridDim = dim3(a.ctas);
    return cudaLaunchKernelEx(&cfg, decode_join_kernel<D, MR, false, ROWS>, a);
}

template <int D, int KIND, int MR, bool BLOCK>
static cudaError_t launch_decode_t(const DecodeArgs &a, cudaStream_t st) {
    return a.T ? launch_decode_k<D, KIND, MR, BLOCK, true>(a, st) : launch_decode_k<D, KIND, MR, BLOCK, false>(a, st);
}

template <int D, int KIND>
static cudaError_t launch_decode_m(const DecodeArgs &a, int mr, cudaStream_t st) {
    if constexpr (KIND >= 2) {
        if (a.c.block_shift) return mr == 8 ? launch_decode_t<D, KIND, 8, true>(a, st) : launch_decode_t<D, KIND, 16, true>(a, st);
    }
    return mr == 8 ? launch_decode_t<D, KIND, 8, false>(a, st) : launch_decode_t<D, KIND, 16, false>(a, st);
}

template <int KIND>
static cudaError_t launch_decode_d(const DecodeArgs &a, int d, int mr, cudaStream_t st) {
    return d == 64 ? launch_decode_m<64, KIND>(a, mr, st) : launch_decode_m<128, KIND>(a, mr, st);
}

static cudaError_t run_decode(const sage_kv &c, const DecodePlan &p, int Hq, const void *Q, const int *lens, void *O, float *L, int add_score,
                              int T, const int *count, void *workspace, cudaStream_t st) {
    uint8_t *w = static_cast<uint8_t *>(workspace);
    DecodeArgs a;
    a.c = kv_view(c);
    a.Q = Q; a.O = O; a.L = L; a.lens = lens;
    a.Hq = Hq; a.G = Hq / c.H; a.chunks = p.chunks; a.ctas = p.ctas; a.cluster = p.cluster; a.tile = p.tile; a.tile_shift = p.tile == 64 ? 6 : 7;
    a.T = T; a.count = count;
    a.bf16 = c.dtype == SAGE_BF16;
    a.sl2 = scale_log2(c.d);
    a.part_O = reinterpret_cast<float *>(w);
    a.part_ml = reinterpret_cast<float *>(w + p.off_ml);
    a.row_ml = add_score && !p.cluster ? reinterpret_cast<float *>(w + p.off_rows) : nullptr;
    a.logits = add_score ? reinterpret_cast<float *>(w + p.off_logits) : nullptr;
    cudaError_t e;
    if (kv_format(c) == SAGE_KV_INT8) e = launch_decode_d<2>(a, c.d, p.mr, st);
    else if (kv_format(c) == SAGE_KV_FP8) e = launch_decode_d<3>(a, c.d, p.mr, st);
    else if (a.bf16) e = launch_decode_d<1>(a, c.d, p.mr, st);
    else e = launch_decode_d<0>(a, c.d, p.mr, st);
    return e;
}

size_t decode_rows_bytes(const sage_kv &c, int Hq, int T) { return decode_plan(c, Hq * T, 0).bytes; }

cudaError_t decode_rows(const sage_kv &c, int Hq, int T, const void *Q, const int *start, const int *count, void *O, float *L, void *workspace,
                        cudaStream_t st) {
    return run_decode(c, decode_plan(c, Hq * T, 0), Hq * T, Q, start, O, L, 0, T, count, workspace, st);
}

}  // namespace sage

using namespace sage;

extern "C" {

size_t sage_decode_workspace_bytes(const sage_kv *c, int Hq, int add_score) {
    if (check_decode(c, Hq, add_score) != SAGE_OK) return 0;
    return decode_plan(*c, Hq, add_score).bytes;
}

int sage_attn_decode(const sage_kv *c, int Hq, const void *Q, const int *lens, void *O, float *L, int add_score,
                     void *workspace, size_t workspace_bytes, sage_stream_t stream) {
    int st = check_decode(c, Hq, add_score);
    if (st != SAGE_OK) return st;
    st = check_kv(c, true);
    if (st != SAGE_OK) return st;
    if (!Q || !lens || !O || !L || O == Q || (add_score && !c->score)) return SAGE_ERR_ARG;
    if (misaligned(Q, 16) || misaligned(O, 16) || misaligned(L, 16) || misaligned(lens, 4)) return SAGE_ERR_ALIGN;
    const DecodePlan p = decode_plan(*c, Hq, add_score);
    if (p.bytes) {                               // else it is not looked at
        if (!workspace || workspace_bytes < p.bytes) return SAGE_ERR_WORKSPACE;
        if (misaligned(workspace, 256)) return SAGE_ERR_ALIGN;
    }
    const cudaError_t e = run_decode(*c, p, Hq, Q, lens, O, L, add_score, 0, nullptr, workspace, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA;
}

}  // extern "C"
