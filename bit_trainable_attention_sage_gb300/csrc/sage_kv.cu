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
// Every element is read once and written once: bound by memory bandwidth (16-bit pools: 64 us for 64
// heads of up to 8192 tokens, d = 128, 6.8 TB/s), in 8 bits by issuing the arithmetic (to E4M3 with
// smoothing 59 us, 5.6 TB/s), or by latency (single tokens).  d / 16 lanes hold a row, two 16-byte
// chunks each, so what is done once a row (its place, scale and reciprocal) is shared by 16 values
// (8 values a lane: 70 us), the maximum is 2 or 3 shuffles and loads and stores are whole sectors.
// One row a lane group and 40 warps an SM keep enough reads in flight (several rows a group: 65 us
// and more).
// ---------------------------------------------------------------------------------------------
constexpr int kAppendThreads = 128;

struct AppendArgs {
    KvView c;
    const void *K, *V;
    const int *start, *count, *pos0;
    const float *mu;
    int T;
};

template <typename T>
__device__ __forceinline__ void unpack16(const uint4 (&u)[2], f2 (&v)[8]) {
    const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float2 f;
        if constexpr (std::is_same<T, __half>::value)
            f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        else
            f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
        v[i] = f2{f.x, f.y};
    }
}

// -fl32(x / d) for two values, nr = -fl32(1 / d): Markstein's correction of a quotient ("Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990).  The residual x - q d is
// exact where q is off by a unit in the last place (ulp) or less, and rounded once where it is off by more:
// a correction leaves the quotient's error times r's and that rounding's, and one rounding.
//   ONCE: for x of at most 11 significant bits (a 16-bit value), one correction of q0 = fl(x r) gives
//   fl32(x / d) for every pair of significands (tests/test_gpu_quotients.py tries all 2^10 x 2^23).
//   Otherwise two.  With significands x, d in [1, 2) and u = 2^-24: r is off by at most d u / 2 of itself,
//   q0 by at most 1.5 ulp, and the first correction by less than
//   0.5 + 3 u ulp; the second then rounds a value within (0.5 + 3 u) d u / 2 ulp of x / d, and
//   x / d is at least u / d ulp from any value half way between two floats (25 bits times d's 24
//   never make x's 24).  (0.5 + 3 u) d / 2 < 1 / d for every d < 2: it rounds as x / d does.
// The negated quotient is what is corrected, because its zeros keep their sign: the residual of either
// zero is +0, and +0 * nr is the -0 that leaves both alone (+0 * r would make +0 of a -0).
// d and nr are pairs (of a value twice, or of two rows' scales).
template <bool ONCE>
__device__ __forceinline__ f2 neg_quotient2(f2 x, f2 d, f2 nr) {
    f2 n = mul2(x, nr);
    if constexpr (!ONCE) n = fma2(fma2(n, d, x), nr, n);
    return fma2(fma2(n, d, x), nr, n);
}

// m / M of two rows, M = 127 or 448.  (Out of the range where the residuals are normal: divisions.)
template <int KIND>
__device__ __forceinline__ f2 scales_of(f2 m) {
    constexpr float M = KIND == SAGE_KV_INT8 ? 127.0f : 448.0f, r = 1.0f / M;
    if (fminf(m.x, m.y) >= 0x1p-80f && fmaxf(m.x, m.y) <= 0x1p96f) return neg_quotient2<false>(f2{-m.x, -m.y}, f2{M, M}, f2{-r, -r});
    return f2{__fdiv_rn(m.x, M), __fdiv_rn(m.y, M)};
}

// One row's 16 values of a lane, and the row's scale -> 16 codes.  n: the negated quotients.
template <int KIND, bool ONCE>
__device__ __forceinline__ void kv_codes(const f2 (&x)[8], float delta, uint2 (&out)[2]) {
    f2 n[8];
    if (delta >= 0x1p-90f && delta <= 0x1p90f) {
        const float nr = -__frcp_rn(delta);
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = neg_quotient2<ONCE>(x[i], f2{delta, delta}, f2{nr, nr});
    } else if (delta == 0.0f) {
        out[0] = out[1] = make_uint2(0u, 0u);
        return;
    } else {
        // a subnormal delta can be rounded so far down that the quotient exceeds 127 (E4M3 saturates)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            constexpr float top = KIND == SAGE_KV_INT8 ? 127.0f : 448.0f;
            n[i].x = -fminf(fmaxf(__fdiv_rn(x[i].x, delta), -top), top);
            n[i].y = -fminf(fmaxf(__fdiv_rn(x[i].y, delta), -top), top);
        }
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (KIND == SAGE_KV_INT8) {
            // 1.5 2^23 - n holds the nearest integer (ties to even) in its low bits
            const f2 magic{12582912.0f, 12582912.0f};
            const f2 a = sub2(magic, n[2 * i]), b = sub2(magic, n[2 * i + 1]);
            const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
            const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
            w[i] = __byte_perm(lo, hi, 0x5410);
        } else {
            w[i] = (e4m3x2(n[2 * i].x, n[2 * i].y) | static_cast<uint32_t>(e4m3x2(n[2 * i + 1].x, n[2 * i + 1].y)) << 16) ^ 0x80808080u;
        }
    }
    out[0] = make_uint2(w[0], w[1]);
    out[1] = make_uint2(w[2], w[3]);
}

// max(|a|, |b|), under some sign; a NaN stays one, so that a row with one gets a scale that says so
// (INT8 has no code for it)
__device__ __forceinline__ float larger(float a, float b) {
    float d;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// The largest magnitude of a row that LANES lanes hold.  (Shuffles: a reduction instruction under
// half-warp masks runs once a half, 83 against 76 us for 8192-token prompts.)
template <int LANES>
__device__ __forceinline__ float largest(const f2 (&x)[8]) {
    float m = larger(x[0].x, x[0].y);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = larger(m, larger(x[i].x, x[i].y));
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) m = larger(m, __shfl_xor_sync(0xffffffffu, m, o));
    return fabsf(m);
}

// grid: (row groups of a head, B * H); a row a lane group.
template <typename T, int KIND, int D, bool SMOOTH>
__global__ void __launch_bounds__(kAppendThreads, 10) kv_append_kernel(const AppendArgs a) {
    constexpr int LANES = D / 16, GROUPS = kAppendThreads / LANES;
    const int bh = blockIdx.y, b = bh / a.c.H, h = bh - b * a.c.H;
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    int n = a.T;
    if (a.count) {
        n = __ldg(a.count + b);
        if (n < 0 || n > a.T) {
            if (threadIdx.x == 0) atomicOr(&g_kv_err, 1u);
            n = n < 0 ? 0 : a.T;
        }
    }
    if (static_cast<int>(blockIdx.x) * GROUPS >= n) return;
    const int t = blockIdx.x * GROUPS + group;
    uint4 k[2], v[2];                                // 16-byte chunks lane and lane + LANES of the row
    k[0] = k[1] = v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u);
    long long row = -1;                              // of the pool; -1: nothing to write
    if (t < n) {
        const size_t at = (static_cast<size_t>(bh) * a.T + t) * (2 * LANES) + lane;
        const uint4 *K = static_cast<const uint4 *>(a.K) + at, *V = static_cast<const uint4 *>(a.V) + at;
        k[0] = __ldg(K);
        k[1] = __ldg(K + LANES);
        v[0] = __ldg(V);
        v[1] = __ldg(V + LANES);
        const long long s = static_cast<long long>(__ldg(a.start + b)) + t;
        if (s < 0 || s >= a.c.cap) {
            atomicOr(&g_kv_err, 1u);
        } else {
            const int p = kv_page(a.c, b, static_cast<int>(s), &g_kv_err);
            if (p >= 0) {
                row = static_cast<long long>(kv_row(a.c, p, h, static_cast<int>(s)));
                if (lane == 0) {
                    const size_t slot = static_cast<size_t>(bh) * a.c.cap + s;
                    if (a.c.score) a.c.score[slot] = 0.0f;
                    if (a.c.pos) a.c.pos[slot] = a.pos0 ? __ldg(a.pos0 + b) + t : static_cast<int>(s);
                }
            }
        }
    }
    if constexpr (KIND == SAGE_KV_16) {
        if (row < 0) return;
        uint4 *K = static_cast<uint4 *>(a.c.K) + row * (2 * LANES) + lane, *V = static_cast<uint4 *>(a.c.V) + row * (2 * LANES) + lane;
        K[0] = k[0];
        K[LANES] = k[1];
        V[0] = v[0];
        V[LANES] = v[1];
    } else {
        // every lane of a warp takes part in the shuffles, row or none
        f2 x[8], y[8];
        unpack16<T>(k, x);
        unpack16<T>(v, y);
        if constexpr (SMOOTH) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float4 *m = reinterpret_cast<const float4 *>(a.mu + static_cast<size_t>(bh) * D + (lane + c * LANES) * 8);
                const float4 m0 = __ldg(m), m1 = __ldg(m + 1);
                x[4 * c] = sub2(x[4 * c], f2{m0.x, m0.y});
                x[4 * c + 1] = sub2(x[4 * c + 1], f2{m0.z, m0.w});
                x[4 * c + 2] = sub2(x[4 * c + 2], f2{m1.x, m1.y});
                x[4 * c + 3] = sub2(x[4 * c + 3], f2{m1.z, m1.w});
            }
        }
        const f2 delta = scales_of<KIND>(f2{largest<LANES>(x), largest<LANES>(y)});
        uint2 ck[2], cv[2];
        kv_codes<KIND, !SMOOTH>(x, delta.x, ck);
        kv_codes<KIND, true>(y, delta.y, cv);
        if (row < 0) return;
        uint2 *K = static_cast<uint2 *>(a.c.K) + row * (2 * LANES) + lane, *V = static_cast<uint2 *>(a.c.V) + row * (2 * LANES) + lane;
        K[0] = ck[0];
        K[LANES] = ck[1];
        V[0] = cv[0];
        V[LANES] = cv[1];
        if (lane == 0) {
            a.c.sK[row] = delta.x;
            a.c.sV[row] = delta.y;
        }
    }
}

template <typename T, int KIND, int D, bool SMOOTH>
static void launch_append_k(const AppendArgs &a, cudaStream_t st) {
    constexpr int GROUPS = kAppendThreads / (D / 16);
    const dim3 grid((a.T + GROUPS - 1) / GROUPS, static_cast<unsigned>(a.c.B) * a.c.H);
    kv_append_kernel<T, KIND, D, SMOOTH><<<grid, kAppendThreads, 0, st>>>(a);
}

template <typename T, int KIND>
static void launch_append_d(const AppendArgs &a, int d, cudaStream_t st) {
    if constexpr (KIND != SAGE_KV_16) {
        if (a.mu) {
            if (d == 64) launch_append_k<T, KIND, 64, true>(a, st);
            else launch_append_k<T, KIND, 128, true>(a, st);
            return;
        }
    }
    if (d == 64) launch_append_k<T, KIND, 64, false>(a, st);
    else launch_append_k<T, KIND, 128, false>(a, st);
}

// ---------------------------------------------------------------------------------------------
// append to a cache with one scale a block
//
// Blocks of R = 16, 32 or 64 slots share s = fl32(max|x| / M).  A block that begins with the call's rows
// takes its scale from them; one that goes on (rows before `start`) keeps the larger of its scale and theirs,
// and where that grows its kept rows' codes become the nearest of fl32(code * fl32(s_old / s)).
// A CTA takes a block of K or of V of one head (both would hold twice the registers): its rows stay in registers between the maximum and the codes, so that
// every element is read once and written once, and only a block whose scale grows reads codes.  Few threads
// with four rows each, so that the barrier between the two holds few up: 64 heads of up to 8192 tokens, d = 128, to
// E4M3 with smoothing 60 us, 5.4 TB/s (256 threads 70, 512 threads 94; K and V in one CTA 80), bound by issuing the
// arithmetic as above; single tokens by latency (3 us).
// ---------------------------------------------------------------------------------------------
template <int D, int R>
struct AppendBlock {
    static constexpr int LANES = D / 16;
    static constexpr int THREADS = R * LANES < 128 ? 32 : R * LANES / 4;
    static constexpr int GROUPS = THREADS / LANES;               // rows at a time
    static constexpr int ROWS = R / GROUPS;                      // rows a lane group
};

// 16 codes times r <= 1, to the nearest code
template <int KIND>
__device__ __forceinline__ uint2 kv_rescaled(uint2 codes, float r) {
    uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (KIND == SAGE_KV_INT8) {
            uint32_t o = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float c = static_cast<float>(static_cast<int8_t>(w[i] >> (8 * k)));
                o |= static_cast<uint32_t>(__float2int_rn(__fmul_rn(c, r)) & 255) << (8 * k);
            }
            w[i] = o;
        } else {
            const uint32_t lo = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i])), hi = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] >> 16));
            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo)), b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
            w[i] = e4m3x2(__fmul_rn(a.x, r), __fmul_rn(a.y, r)) | static_cast<uint32_t>(e4m3x2(__fmul_rn(b.x, r), __fmul_rn(b.y, r))) << 16;
        }
    }
    return make_uint2(w[0], w[1]);
}

// One block of K or of V: x, its pool and scales.
template <typename T, int KIND, int D, int R, bool SMOOTH>
__device__ __forceinline__ void append_block(const AppendArgs &a, const void *x_in, void *pool, float *scales, const float *mu_in, int bh, int n, long long start,
                                             long long s0, int b, int h) {
    using S = AppendBlock<D, R>;
    constexpr int LANES = S::LANES, WARPS = S::THREADS / 32;
    constexpr int SHIFT = R == 16 ? 4 : R == 32 ? 5 : 6;
    __shared__ float s_max[WARPS];
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    // this lane group's rows: slots s0 + group + i * GROUPS, tokens t0 + i * GROUPS
    uint4 in[S::ROWS][2];
    const int t0 = static_cast<int>(s0 - start) + group;             // (at least -R, below 2^30)
#pragma unroll
    for (int i = 0; i < S::ROWS; ++i) {
        const int t = t0 + i * S::GROUPS;
        in[i][0] = in[i][1] = make_uint4(0u, 0u, 0u, 0u);
        if (t >= 0 && t < n) {
            const uint4 *X = static_cast<const uint4 *>(x_in) + (static_cast<size_t>(bh) * a.T + t) * (2 * LANES) + lane;
            in[i][0] = __ldg(X);
            in[i][1] = __ldg(X + LANES);
        }
    }
    const int p = kv_page(a.c, b, static_cast<int>(s0), &g_kv_err);
    if (p < 0) return;                               // the whole CTA alike
    const size_t row0 = kv_row(a.c, p, h, static_cast<int>(s0)), place = row0 >> SHIFT;
    const bool goes_on = start > s0;
    const float old = goes_on ? scales[place] : 0.0f;
    // (kept as float32: forming the values again for the codes costs more than the registers)
    f2 x[S::ROWS][8];
#pragma unroll
    for (int i = 0; i < S::ROWS; ++i) unpack16<T>(in[i], x[i]);
    if constexpr (SMOOTH) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float4 *m = reinterpret_cast<const float4 *>(mu_in + static_cast<size_t>(bh) * D + (lane + c * LANES) * 8);
            const float4 m0 = __ldg(m), m1 = __ldg(m + 1);
#pragma unroll
            for (int i = 0; i < S::ROWS; ++i) {
                x[i][4 * c] = sub2(x[i][4 * c], f2{m0.x, m0.y});
                x[i][4 * c + 1] = sub2(x[i][4 * c + 1], f2{m0.z, m0.w});
                x[i][4 * c + 2] = sub2(x[i][4 * c + 2], f2{m1.x, m1.y});
                x[i][4 * c + 3] = sub2(x[i][4 * c + 3], f2{m1.z, m1.w});
            }
        }
    }
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < S::ROWS; ++i) {
        const int t = t0 + i * S::GROUPS;
        float m = larger(x[i][0].x, x[i][0].y);
#pragma unroll
        for (int j = 1; j < 8; ++j) m = larger(m, larger(x[i][j].x, x[i][j].y));
        if (t >= 0 && t < n) most = larger(most, m);                 // (other rows' zeros less mu are no values)
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = larger(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (threadIdx.x % 32 == 0) s_max[threadIdx.x / 32] = most;
    __syncthreads();                                 // and every thread has the old scale
#pragma unroll
    for (int w = 0; w < WARPS; ++w) most = larger(most, s_max[w]);
    float s = scales_of<KIND>(f2{fabsf(most), fabsf(most)}).x;
    if (goes_on) s = fabsf(larger(s, old));
    if (threadIdx.x == 0) scales[place] = s;
    const bool grew = goes_on && s > old;
    const float ratio = grew ? __fdiv_rn(old, s) : 1.0f;
#pragma unroll
    for (int i = 0; i < S::ROWS; ++i) {
        const int t = t0 + i * S::GROUPS;
        uint2 *to = static_cast<uint2 *>(pool) + (row0 + group + i * S::GROUPS) * (2 * LANES) + lane;
        if (t >= 0 && t < n) {
            uint2 c[2];
            kv_codes<KIND, !SMOOTH>(x[i], s, c);
            to[0] = c[0];
            to[LANES] = c[1];
        } else if (t < 0 && grew) {                  // a kept row
            to[0] = kv_rescaled<KIND>(to[0], ratio);
            to[LANES] = kv_rescaled<KIND>(to[LANES], ratio);
        }
    }
}

// grid: (blocks of a sequence that T tokens can touch, B * H, K and V)
template <typename T, int KIND, int D, int R, bool SMOOTH>
__global__ void __launch_bounds__(AppendBlock<D, R>::THREADS, 896 / AppendBlock<D, R>::THREADS) kv_append_block_kernel(const AppendArgs a) {
    constexpr int SHIFT = R == 16 ? 4 : R == 32 ? 5 : 6;
    const int bh = blockIdx.y, b = bh / a.c.H, h = bh - b * a.c.H;
    int n = a.T;
    if (a.count) {
        n = __ldg(a.count + b);
        if (n < 0 || n > a.T) {
            if (threadIdx.x == 0) atomicOr(&g_kv_err, 1u);
            n = n < 0 ? 0 : a.T;
        }
    }
    const long long start = __ldg(a.start + b);
    const long long s0 = ((start >> SHIFT) + blockIdx.x) << SHIFT;   // the block's first slot
    if (s0 >= start + n || n == 0) return;
    if (s0 < 0 || s0 >= a.c.cap) {                   // the capacity is a multiple of the block
        if (threadIdx.x == 0) atomicOr(&g_kv_err, 1u);
        return;
    }
    if (blockIdx.z == 0) append_block<T, KIND, D, R, SMOOTH>(a, a.K, a.c.K, a.c.sK, a.mu, bh, n, start, s0, b, h);
    else append_block<T, KIND, D, R, false>(a, a.V, a.c.V, a.c.sV, nullptr, bh, n, start, s0, b, h);
}

template <typename T, int KIND, int D, int R>
static void launch_append_block_r(const AppendArgs &a, cudaStream_t st) {
    const dim3 grid((a.T + R - 2) / R + 1, static_cast<unsigned>(a.c.B) * a.c.H, 2);
    if (a.mu) kv_append_block_kernel<T, KIND, D, R, true><<<grid, AppendBlock<D, R>::THREADS, 0, st>>>(a);
    else kv_append_block_kernel<T, KIND, D, R, false><<<grid, AppendBlock<D, R>::THREADS, 0, st>>>(a);
}

template <typename T, int KIND>
static void launch_append_block(const AppendArgs &a, int d, int block, cudaStream_t st) {
    if (d == 64) {
        if (block == 16) launch_append_block_r<T, KIND, 64, 16>(a, st);
        else if (block == 32) launch_append_block_r<T, KIND, 64, 32>(a, st);
        else launch_append_block_r<T, KIND, 64, 64>(a, st);
    } else {
        if (block == 16) launch_append_block_r<T, KIND, 128, 16>(a, st);
        else if (block == 32) launch_append_block_r<T, KIND, 128, 32>(a, st);
        else launch_append_block_r<T, KIND, 128, 64>(a, st);
    }
}

template <typename T, int KIND>
static void launch_append_8(const AppendArgs &a, const sage_kv &c, cudaStream_t st) {
    if (kv_block(c)) launch_append_block<T, KIND>(a, c.d, kv_block(c), st);
    else launch_append_d<T, KIND>(a, c.d, st);
}

static void launch_append(const sage_kv &c, const AppendArgs &a, cudaStream_t st) {
    const int format = kv_format(c);
    // a 16-bit pool is copied: one instance serves both 16-bit types
    if (format == SAGE_KV_16) launch_append_d<__half, SAGE_KV_16>(a, c.d, st);
    else if (format == SAGE_KV_INT8 && c.dtype == SAGE_FP16) launch_append_8<__half, SAGE_KV_INT8>(a, c, st);
    else if (format == SAGE_KV_INT8) launch_append_8<__nv_bfloat16, SAGE_KV_INT8>(a, c, st);
    else if (c.dtype == SAGE_FP16) launch_append_8<__half, SAGE_KV_FP8>(a, c, st);
    else launch_append_8<__nv_bfloat16, SAGE_KV_FP8>(a, c, st);
}

// ---------------------------------------------------------------------------------------------
// eviction
//
// Which slots stay is a selection, not a sort: the budget-th largest key of a row of n keys by
// radix selection (8 bits a pass, most often three of the four passes), then one pass in slot order
// that takes what is above it and the first of what is equal.  Only stayers in slots >= budget move, into the freed slots
// below: sources and destinations are disjoint, so the moves need no order among them, and a
// cache that is cut back by a few tokens moves a few rows instead of being compacted.
//
// One cluster of C CTAs a (sequence, kv head), each with a contiguous C-th of the slots: scores and
// positions are read once, the keys stay in shared memory (CACHED; rows of more than
// 8 * 20 K slots read them again each pass), histograms and counts are added up over the cluster
// through distributed shared memory, and the same CTAs then move the rows.  One launch, and with
// C up to 8 a few long rows still use many SMs.  Bound by latency: 32 rows of up to 32768 slots cut
// to 8192 (E4M3, d = 128) take 36 us, 18 of them for the selection's phases (a barrier of the
// cluster each) and 9 for 57 MB of moves; 64 rows of 1088 cut to 1024 take 9.  (Digits of 11 bits,
// whose histograms are 64 KB of remote reads a CTA and pass: 39 and 8.8; clusters half as large: 43;
// four keys a lane and step, a third of the instructions: 36 and 8.7.)
// ---------------------------------------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 256;
constexpr int kSelMaxCluster = 8;
constexpr int kMoves = 2 * kSelThreads;
constexpr int kSelMaxKeys = 20 * 1024;       // of a CTA in shared memory; two CTAs an SM

struct EvictArgs {
    KvView c;
    const int *lens, *seen;
    int *lens_out;
    int *dst, *src;      // (B*H, max_moves)
    int budget, recent, max_moves;
    int cluster;
};

// Larger key = stays longer.  Recent tokens above every score; scores in the order of the reals
// (-0 = +0), NaN last.
__device__ __forceinline__ uint32_t evict_key(float s, bool recent) {
    if (recent) return 0xFFFFFFFFu;
    if (s != s) return 0u;
    const uint32_t u = __float_as_uint(s + 0.0f);           // -0 becomes +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);      // at most 0xFF800000 (+inf)
}

// Moves begin .. end - 1 of a row, kMoves at a time: a thread looks up two moves' rows and
// moves what is a word (scales, score, position), then ROW_BYTES / 16 lanes copy a row's K and V, whose
// addresses all wait in shared memory.
template <int ROW_BYTES>
__device__ __forceinline__ void evict_moves(const EvictArgs &a, int bh, int b, int h, int begin, int end, size_t (*rows)[kMoves]) {
    constexpr int CHUNKS = ROW_BYTES / 16, GROUPS = kSelThreads / CHUNKS, UNROLL = 4;
    const size_t list = static_cast<size_t>(bh) * a.max_moves, base = static_cast<size_t>(bh) * a.c.cap;
    const int tid = threadIdx.x, lane = tid % CHUNKS, group = tid / CHUNKS;
    uint4 *K = static_cast<uint4 *>(a.c.K) + lane, *V = static_cast<uint4 *>(a.c.V) + lane;
    constexpr size_t kNone = ~static_cast<size_t>(0);
    for (int i0 = begin; i0 < end; i0 += kMoves) {
        const int n = min(kMoves, end - i0);
#pragma unroll
        for (int x = 0; x < kMoves / kSelThreads; ++x) {
            const int i = x * kSelThreads + tid;
            if (i >= n) break;
            const int d = a.dst[list + i0 + i], s = a.src[list + i0 + i];
            const int pd = kv_page(a.c, b, d, &g_kv_err), ps = kv_page(a.c, b, s, &g_kv_err);
            size_t rd = kNone, rs = 0;
            if (pd >= 0 && ps >= 0) {
                rd = kv_row(a.c, pd, h, d);
                rs = kv_row(a.c, ps, h, s);
                const float score = a.c.score[base + s];
                const int pos = a.c.pos[base + s];
                if (a.c.sK) {
                    const float sk = a.c.sK[rs], sv = a.c.sV[rs];
                    a.c.sK[rd] = sk;
                    a.c.sV[rd] = sv;
                }
                a.c.score[base + d] = score;
                a.c.pos[base + d] = pos;
            }
            rows[0][i] = rd;
            rows[1][i] = rs;
        }
        __syncthreads();
        for (int i = group; i < n; i += GROUPS * UNROLL) {
            uint4 k[UNROLL], v[UNROLL];
            size_t rd[UNROLL];
#pragma unroll
            for (int x = 0; x < UNROLL; ++x) {
                const int j = i + x * GROUPS;
                rd[x] = j < n ? rows[0][j] : kNone;
                if (rd[x] != kNone) {
                    const size_t rs = rows[1][j] * CHUNKS;
                    k[x] = K[rs];
                    v[x] = V[rs];
                }
            }
#pragma unroll
            for (int x = 0; x < UNROLL; ++x)
                if (rd[x] != kNone) {
                    K[rd[x] * CHUNKS] = k[x];
                    V[rd[x] * CHUNKS] = v[x];
                }
        }
        __syncthreads();
    }
}

// grid: (cluster, B * H)
template <bool CACHED, int ROW_BYTES>
__global__ void __launch_bounds__(kSelThreads, 2) kv_evict_kernel(const __grid_constant__ EvictArgs a) {
    extern __shared__ uint32_t s_key[];
    __shared__ __align__(16) int hist[4][kSelBins];
    __shared__ size_t s_rows[2][kMoves];
    __shared__ int s_warp[2][kSelWarps];
    __shared__ __align__(16) int s_count[4];                   // of this CTA, read by the others: equal keys; freed, movers
    __shared__ int s_digit, s_above, s_here;
    const int bh = blockIdx.y, b = bh / a.c.H, h = bh - b * a.c.H, rank = blockIdx.x;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int n = kv_len(a.c, a.lens, b, &g_kv_err);
    if (tid == 0 && rank == 0 && h == 0) a.lens_out[b] = min(n, a.budget);
    if (n <= a.budget) return;                   // the whole cluster alike
    const size_t base = static_cast<size_t>(bh) * a.c.cap;
    const long long newest = static_cast<long long>(__ldg(a.seen + b)) - a.recent;   // recent from here on
    // this CTA's slots [lo, lo + len), a warp's contiguous: slot lo + (warp * its + i) * 32 + lane
    const int seg = ((n + a.cluster - 1) / a.cluster + kSelThreads - 1) / kSelThreads * kSelThreads;
    const int lo = min(n, rank * seg), len = min(n - lo, seg), its = seg / kSelThreads;
    const int mine = warp * its * 32 + lane;
    for (int i = tid; i < 4 * kSelBins; i += kSelThreads) (&hist[0][0])[i] = 0;
    __syncthreads();
    // score and pos are read with plain loads: the moves below write them (after every read here)
    auto key = [&](int i) -> uint32_t {
        const int s = mine + i * 32;
        if constexpr (CACHED) return s_key[s];
        else return evict_key(a.c.score[base + lo + s], a.c.pos[base + lo + s] >= newest);
    };
    // equal digits of a warp are added once: keys crowd into few of them
    auto count = [&](int pass, bool in, uint32_t digit) {
        const uint32_t same = __match_any_sync(0xffffffffu, in ? digit : 256u);
        if (in && lane == __ffs(same) - 1) atomicAdd(&hist[pass][digit], __popc(same));
    };
    constexpr int BATCH = 8;                     // reads in flight together
    for (int i0 = 0; i0 < its; i0 += BATCH) {
        float score[BATCH];
        int pos[BATCH];
#pragma unroll
        for (int x = 0; x < BATCH; ++x) {
            const int s = mine + (i0 + x) * 32;
            const bool in = i0 + x < its && s < len;
            score[x] = in ? a.c.score[base + lo + s] : 0.0f;
            pos[x] = in ? a.c.pos[base + lo + s] : 0;
        }
#pragma unroll
        for (int x = 0; x < BATCH; ++x) {
            const int s = mine + (i0 + x) * 32;
            const bool in = i0 + x < its && s < len;
            const uint32_t k = evict_key(score[x], pos[x] >= newest);
            if (CACHED && in) s_key[s] = k;
            count(0, in, k >> 24);
        }
    }
    // the budget-th largest key: `T` its leading digits, `need` its rank among the keys that share them
    uint32_t T = 0;
    int need = a.budget, equal = 0;
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        if (pass > 0) {
            for (int i = 0; i < its; ++i) {
                const int s = mine + i * 32;
                const uint32_t k = s < len ? key(i) : 0u;
                const bool in = s < len && ((k ^ T) >> (shift + 8)) == 0u;
                if (__any_sync(0xffffffffu, in)) count(pass, in, (k >> shift) & 255u);
            }
        }
        if (a.cluster > 1) cluster_sync();
        else __syncthreads();
        // thread t holds the DIG digits from 255 - DIG t down
        constexpr int DIG = 4;
        int c[DIG] = {};
        const int d0 = kSelBins - 1 - DIG * tid;
        if (d0 > 0) {
            int4 v[kSelMaxCluster];
#pragma unroll
            for (int r = 0; r < kSelMaxCluster; ++r)
                if (r < a.cluster) v[r] = cluster_words(&hist[pass][d0 - 3], r);
#pragma unroll
            for (int r = 0; r < kSelMaxCluster; ++r)
                if (r < a.cluster) {
                    c[0] += v[r].w; c[1] += v[r].z; c[2] += v[r].y; c[3] += v[r].x;
                }
        }
        const int sum = c[0] + c[1] + c[2] + c[3];
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) s_warp[0][warp] = incl;
        __syncthreads();
        int above = incl - sum;
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) above += w < warp ? s_warp[0][w] : 0;
#pragma unroll
        for (int i = 0; i < DIG; ++i) {
            if (above < need && need <= above + c[i]) {
                s_digit = d0 - i;
                s_above = above;
                s_here = c[i];
            }
            above += c[i];
        }
        __syncthreads();
        T |= static_cast<uint32_t>(s_digit) << shift;
        need -= s_above;
        equal = s_here;
        __syncthreads();
        if (equal == need) break;                // all that share these digits stay: T is their lower bound
    }
    // Of the `equal` keys equal to T, the first `need` in slot order stay.  How many lie before this
    // warp's slots matters only when not all of them do.
    int eq0 = 0;
    if (equal > need) {
        int eq = 0;
        for (int i = 0; i < its; ++i) eq += __popc(__ballot_sync(0xffffffffu, mine + i * 32 < len && key(i) == T));
        if (lane == 0) s_warp[0][warp] = eq;
        __syncthreads();
        if (tid == 0) {
            int sum = 0;
            for (int w = 0; w < kSelWarps; ++w) sum += s_warp[0][w];
            s_count[0] = sum;
        }
        if (a.cluster > 1) cluster_sync();
        else __syncthreads();
        for (int r = 0; r < rank; ++r) eq0 += cluster_word(&s_count[0], r);
        for (int w = 0; w < warp; ++w) eq0 += s_warp[0][w];
        __syncthreads();
    }
    // freed slots below the budget and stayers from it on, counted, then numbered
    const uint32_t before = (1u << lane) - 1u;
    int at[2] = {0, 0}, moves = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int e = eq0, freed = at[0], moved = at[1];
        for (int i = 0; i < its; ++i) {
            const int s = mine + i * 32, slot = lo + s;
            const bool in = s < len;
            const uint32_t k = in ? key(i) : 0u;
            const bool iseq = in && k == T;
            const uint32_t beq = __ballot_sync(0xffffffffu, iseq);
            const bool stays = in && (k > T || (iseq && (equal <= need || e + __popc(beq & before) < need)));
            e += __popc(beq);
            const bool f = in && !stays && slot < a.budget, m = stays && slot >= a.budget;
            const uint32_t bf = __ballot_sync(0xffffffffu, f), bm = __ballot_sync(0xffffffffu, m);
            if (pass == 1) {
                const size_t o = static_cast<size_t>(bh) * a.max_moves;
                if (f) a.dst[o + freed + __popc(bf & before)] = slot;
                if (m) a.src[o + moved + __popc(bm & before)] = slot;
            }
            freed += __popc(bf);
            moved += __popc(bm);
        }
        if (pass == 0) {
            if (lane == 0) {
                s_warp[0][warp] = freed;
                s_warp[1][warp] = moved;
            }
            __syncthreads();
            if (warp < 2) {
                const int sum = __reduce_add_sync(0xffffffffu, lane < kSelWarps ? s_warp[warp][lane] : 0);
                if (lane == 0) s_count[2 + warp] = sum;
            }
            if (a.cluster > 1) cluster_sync();
            else __syncthreads();
            for (int r = 0; r < a.cluster; ++r) {
                const int4 n4 = cluster_words(s_count, r);
                const int f = n4.z, m = n4.w;
                if (r < rank) {
                    at[0] += f;
                    at[1] += m;
                }
                moves += m;
            }
#pragma unroll
            for (int w = 0; w < kSelWarps; ++w) {
                at[0] += w < warp ? s_warp[0][w] : 0;
                at[1] += w < warp ? s_warp[1][w] : 0;
            }
        }
    }
    // every CTA's part of the lists is written, every read of another's shared memory done
    if (a.cluster > 1) cluster_sync();
    else __syncthreads();
    const int share = (moves + a.cluster - 1) / a.cluster;
    evict_moves<ROW_BYTES>(a, bh, b, h, rank * share, min(moves, (rank + 1) * share), s_rows);
}

static int evict_max_moves(const sage_kv &c, int budget) {
    const int cap = c.max_pages * c.page;
    const int m = budget < cap - budget ? budget : cap - budget;
    return m < 0 ? 0 : (m + 3) & ~3;
}

// Clusters as large as 4096 slots a CTA ask for, but no more than give every SM two CTAs.
template <bool CACHED, int ROW_BYTES>
static cudaError_t launch_evict_c(const EvictArgs &a, int rows, size_t smem, cudaStream_t st) {
    if (CACHED) {
        static bool raised[16] = {false};
        const cudaError_t e = raise_smem(reinterpret_cast<const void *>(kv_evict_kernel<CACHED, ROW_BYTES>),
                                         kSelMaxKeys * sizeof(uint32_t), raised);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.cluster, rows);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = a.cluster;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_evict_kernel<CACHED, ROW_BYTES>, a);
}

template <int ROW_BYTES>
static cudaError_t launch_evict(EvictArgs a, int rows, cudaStream_t st) {
    int c = 1;
    while (c < kSelMaxCluster && c * 4096 < a.c.cap) c *= 2;
    while (c > 1 && static_cast<long long>(rows) * c > 304 && c / 2 * kSelMaxKeys >= a.c.cap) c /= 2;
    a.cluster = c;
    // keys of a CTA, rounded as the kernel rounds its share of the longest row
    const size_t keys = ((static_cast<size_t>(a.c.cap) + c - 1) / c + kSelThreads - 1) / kSelThreads * kSelThreads;
    if (keys <= kSelMaxKeys) return launch_evict_c<true, ROW_BYTES>(a, rows, keys * sizeof(uint32_t), st);
    return launch_evict_c<false, ROW_BYTES>(a, rows, 0, st);
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
    if (mu && kv_format(*c) == SAGE_KV_16) return SAGE_ERR_UNSUPPORTED;
    if (misaligned(K, 16) || misaligned(V, 16) || misaligned(mu, 16) || misaligned(start, 4) ||
        misaligned(count, 4) || misaligned(pos0, 4))
        return SAGE_ERR_ALIGN;
    const AppendArgs a{kv_view(*c), K, V, start, count, pos0, mu, T};
    launch_append(*c, a, reinterpret_cast<cudaStream_t>(stream));
    return cudaGetLastError() == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA;
}

size_t sage_evict_workspace_bytes(const sage_kv *c, int budget) {
    if (check_kv(c, false) != SAGE_OK || budget <= 0) return 0;
    const size_t n = 2 * static_cast<size_t>(c->B) * c->H * evict_max_moves(*c, budget);
    return (n ? n : 4) * sizeof(int);
}

int sage_kv_evict(const sage_kv *c, const int *lens, const int *seen, int budget, int recent, int *lens_out,
                  void *workspace, size_t workspace_bytes, sage_stream_t stream) {
    const int st = check_kv(c, true);
    if (st != SAGE_OK) return st;
    if (kv_block(*c)) return SAGE_ERR_UNSUPPORTED;                   // rows that share a scale do not move alone
    if (!lens || !seen || !lens_out || !c->score || !c->pos) return SAGE_ERR_ARG;
    const size_t nl = static_cast<size_t>(c->B) * sizeof(int);       // one sequence's length may be read after another's is written
    if (overlap(lens_out, nl, lens, nl) || overlap(lens_out, nl, seen, nl)) return SAGE_ERR_ARG;
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
    a.dst = static_cast<int *>(workspace);
    a.src = a.dst + static_cast<size_t>(rows) * a.max_moves;
    const int row_bytes = c->d * (kv_format(*c) == SAGE_KV_16 ? 2 : 1);
    cudaError_t e;
    if (row_bytes == 64) e = launch_evict<64>(a, rows, s);
    else if (row_bytes == 128) e = launch_evict<128>(a, rows, s);
    else e = launch_evict<256>(a, rows, s);
    return e == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA;
}

}  // extern "C"
