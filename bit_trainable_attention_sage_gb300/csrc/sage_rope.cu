// sage_rope.cu -- rotary positions with several axes, forward and inverse (the gradient).
//
// y0 = x0 cos - x1 sin, y1 = x0 sin + x1 cos for each of a token's pairs.  Every element is read
// and written once, so the kernel is bound by memory bandwidth; what must not show is the cost of
// the angles.  One thread holds the sines and cosines of 8 pairs of one token in registers and
// uses them for every head it visits, so a sine is computed once per (token, pair, head chunk); the
// rows of several heads are in flight together.  2 x (16 + 16) heads of 8192 tokens, d = 128, fp16:
// 42.7 us, 6.3 TB/s, 93 % of the measured copy rate.
//
// The angle of pair j at position p is p * freq[j] mod 2 pi.  In units of a turn, freq[j] / 2 pi
// mod 1 is held as a 64-bit fixed-point fraction f (whole turns a position vanish because p is an
// integer), and p * f mod 2^64 is then one wrapping integer product: the error is |p| 2^-64 of a
// turn plus |p| times that of freq[j] / 2 pi in float64, where a float32 product p * freq[j] would
// be off by a good part of a radian for far positions.  The nearest quarter turn is taken off while
// it is an integer, and the next 32 bits are rounded to a float, at most a quarter of a half turn: the
// angle is off by at most 2^-24 of what is left of it and 2^-33 of a half turn.  Its sine and cosine are short
// series there (sincospif, which reduces its argument once more, made the kernel 11 % slower).
#include <math.h>

#include "sage_device.cuh"
#include "sage_internal.h"

namespace sage {

constexpr int kRopeThreads = 128;
constexpr int kRopeMaxPairs = 64;        // d = 128
constexpr int kRopeFly16 = 4, kRopeFly32 = 2;   // heads in flight, 16-bit and float32

struct RopeArgs {
    const void *src[2];                  // Q, K
    void *dst[2];
    const int *pos;
    int H, Hk, N, d, rotary, tokens;     // tokens = B * N
    int pos_batch_stride;
    long long pos_axis_stride;
    int heads_per_block;
    float sign;                          // -1: inverse
    unsigned long long f[kRopeMaxPairs];
    unsigned char axis[kRopeMaxPairs];
};

// 8 channels as they are stored
template <typename T>
struct RopeRaw {
    uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ RopeRaw<T> rope_load8(const T *p) {
    RopeRaw<T> r;
#pragma unroll
    for (size_t i = 0; i < sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const uint4 *>(p)[i];
    return r;
}
template <typename T>
__device__ __forceinline__ void rope_values(const RopeRaw<T> &r, float (&v)[8]) {
#pragma unroll
    for (size_t k = 0; k < sizeof(T) / 2; ++k) {
        const uint32_t w[4] = {r.w[k].x, r.w[k].y, r.w[k].z, r.w[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<T, float>::value) {
                v[4 * k + i] = __uint_as_float(w[i]);
            } else {
                float2 f;
                if constexpr (std::is_same<T, __half>::value)
                    f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                else
                    f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ void rope_store8(T *p, const float (&v)[8]) {
    if constexpr (std::is_same<T, float>::value) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Sines and cosines of two angles of t 2^-64 turns.  With x the half turns beside the nearest quarter turn,
// |x| <= 1/4, the Taylor series of sin(pi x) to x^9 and of cos(pi x) to x^10: what is left out is below
// (pi / 4)^11 / 11! = 1.8e-9 and (pi / 4)^12 / 12! = 1.2e-10, a thirtieth of a rounding.  pi x is taken with pi in
// two parts, so that the sine keeps its bits where it is small.
__device__ __forceinline__ void rope_sincos(unsigned long long t0, unsigned long long t1, float *sn, float *cs) {
    const uint32_t hi[2] = {static_cast<uint32_t>(t0 >> 32), static_cast<uint32_t>(t1 >> 32)};
    // 2^-32 of a quarter turn
    const int r0 = static_cast<int>(__funnelshift_l(static_cast<uint32_t>(t0), hi[0], 2));
    const int r1 = static_cast<int>(__funnelshift_l(static_cast<uint32_t>(t1), hi[1], 2));
    auto both = [](float v) { return f2{v, v}; };
    const f2 x = mul2(f2{static_cast<float>(r0), static_cast<float>(r1)}, both(0x1p-33f)), x2 = mul2(x, x);
    f2 s = fma2(x2, both(0.0821458866f), both(-0.599264529f));       // pi^9 / 9!, -pi^7 / 7!
    s = fma2(x2, s, both(2.55016404f));                              // pi^5 / 5!
    s = fma2(x2, s, both(-5.16771278f));                             // -pi^3 / 3!
    s = fma2(x2, s, both(-8.74227800e-8f));                          // pi - fl32(pi)
    s = fma2(x, both(3.14159274f), mul2(x, s));
    f2 c = fma2(x2, both(-0.0258068914f), both(0.235330630f));       // -pi^10 / 10!, pi^8 / 8!
    c = fma2(x2, c, both(-1.33526277f));                             // -pi^6 / 6!
    c = fma2(x2, c, both(4.05871213f));                              // pi^4 / 4!
    c = fma2(x2, c, both(-4.93480220f));                             // -pi^2 / 2
    c = fma2(x2, c, both(1.0f));
    const float ss[2] = {s.x, s.y}, cc[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        // each quarter turn makes (-sin, cos) of (cos, sin)
        const uint32_t quarter = (hi[i] + 0x20000000u) >> 30;        // the nearest, mod 4
        const uint32_t a = __float_as_uint(quarter & 1u ? ss[i] : cc[i]), b = __float_as_uint(quarter & 1u ? cc[i] : ss[i]);
        cs[i] = __uint_as_float(a ^ ((quarter + 1u) & 2u) << 30);
        sn[i] = __uint_as_float(b ^ (quarter & 2u) << 30);
    }
}

// grid: (token groups, head chunks).  A token's row takes d / 16 threads of 16 channels each: the
// first rotary / 16 hold 8 pairs, the others copy.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    const int per_row = a.d / 16;
    const int v = threadIdx.x % per_row;
    const int tok = blockIdx.x * (kRopeThreads / per_row) + threadIdx.x / per_row;
    if (tok >= a.tokens) return;
    const int b = tok / a.N, n = tok - b * a.N;
    const bool turns = v * 16 < a.rotary;
    // the thread's two runs of 8 channels
    const int c0 = INTERLEAVED || !turns ? v * 16 : v * 8;
    const int c1 = INTERLEAVED || !turns ? v * 16 + 8 : v * 8 + a.rotary / 2;
    float cs[8], sn[8];
    if (turns) {
        const int *pos = a.pos + static_cast<long long>(b) * a.pos_batch_stride + n;
        auto turns_of = [&](int i) {
            const int j = v * 8 + i;
            const long long p = pos[static_cast<long long>(a.axis[j]) * a.pos_axis_stride];
            return static_cast<unsigned long long>(p) * a.f[j];
        };
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            rope_sincos(turns_of(i), turns_of(i + 1), sn + i, cs + i);
            sn[i] *= a.sign;
            sn[i + 1] *= a.sign;
        }
    }
    const int h0 = blockIdx.y * a.heads_per_block;
    const int h1 = min(h0 + a.heads_per_block, a.H + a.Hk);
    // the rows of FLY heads are read before any is written (in place they are different elements)
    constexpr int FLY = sizeof(T) == 2 ? kRopeFly16 : kRopeFly32;
    for (int h = h0; h < h1; h += FLY) {
        RopeRaw<T> r0[FLY], r1[FLY];
        T *dst[FLY];
#pragma unroll
        for (int i = 0; i < FLY; ++i) {
            const int hi = min(h + i, h1 - 1);
            const bool isk = hi >= a.H;
            const int heads = isk ? a.Hk : a.H, hh = isk ? hi - a.H : hi;
            const size_t row = ((static_cast<size_t>(b) * heads + hh) * a.N + n) * a.d;
            const T *src = static_cast<const T *>(a.src[isk]) + row;
            dst[i] = static_cast<T *>(a.dst[isk]) + row;
            if (h + i < h1) {
                r0[i] = rope_load8(src + c0);
                r1[i] = rope_load8(src + c1);
            }
        }
#pragma unroll
        for (int i = 0; i < FLY; ++i) {
            if (h + i >= h1) break;
            float x[8], y[8], o0[8], o1[8];
            rope_values(r0[i], x);
            rope_values(r1[i], y);
            if (!turns) {
                rope_store8(dst[i] + c0, x);
                rope_store8(dst[i] + c1, y);
                continue;
            }
            if constexpr (INTERLEAVED) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    o0[2 * j] = x[2 * j] * cs[j] - x[2 * j + 1] * sn[j];
                    o0[2 * j + 1] = x[2 * j] * sn[j] + x[2 * j + 1] * cs[j];
                    o1[2 * j] = y[2 * j] * cs[4 + j] - y[2 * j + 1] * sn[4 + j];
                    o1[2 * j + 1] = y[2 * j] * sn[4 + j] + y[2 * j + 1] * cs[4 + j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    o0[j] = x[j] * cs[j] - y[j] * sn[j];
                    o1[j] = x[j] * sn[j] + y[j] * cs[j];
                }
            }
            rope_store8(dst[i] + c0, o0);
            rope_store8(dst[i] + c1, o1);
        }
    }
}

template <typename T>
static void launch_rope_t(const RopeArgs &a, bool interleaved, dim3 grid, cudaStream_t st) {
    if (interleaved) rope_kernel<T, true><<<grid, kRopeThreads, 0, st>>>(a);
    else rope_kernel<T, false><<<grid, kRopeThreads, 0, st>>>(a);
}

static int check_rope(const sage_rope_params *r) {
    if (!r || r->B <= 0 || r->H <= 0 || r->Hk < 0 || r->N <= 0 || r->d <= 0) return SAGE_ERR_ARG;
    if (r->dtype != SAGE_FP16 && r->dtype != SAGE_BF16 && r->dtype != SAGE_FP32) return SAGE_ERR_UNSUPPORTED;
    if (r->d != 64 && r->d != 128) return SAGE_ERR_UNSUPPORTED;
    if (r->axes < 1 || r->axes > SAGE_ROPE_MAX_AXES || !r->sections || !r->freq) return SAGE_ERR_ARG;
    if (r->pos_batch != 1 && r->pos_batch != r->B) return SAGE_ERR_ARG;
    if (r->rotary < 16 || r->rotary > r->d || r->rotary % 16) return SAGE_ERR_ARG;
    if ((r->interleaved | r->inverse) & ~1) return SAGE_ERR_ARG;
    if (static_cast<long long>(r->H) + r->Hk > 65535) return SAGE_ERR_UNSUPPORTED;
    if (static_cast<long long>(r->B) * r->N >= (1ll << 31) - kRopeThreads) return SAGE_ERR_UNSUPPORTED;
    int sum = 0;
    for (int i = 0; i < r->axes; ++i) {
        if (r->sections[i] < 0 || r->sections[i] > r->rotary / 2) return SAGE_ERR_ARG;
        sum += r->sections[i];
    }
    if (sum != r->rotary / 2) return SAGE_ERR_ARG;
    for (int j = 0; j < r->rotary / 2; ++j)
        if (!(fabs(r->freq[j]) <= 1e15)) return SAGE_ERR_ARG;   // NaN, infinite, or without a fraction
    return SAGE_OK;
}

}  // namespace sage

using namespace sage;

extern "C" int sage_rope(const sage_rope_params *r, const void *Q, const void *K, const int *pos, void *Qo,
                         void *Ko, sage_stream_t stream) {
    const int st = check_rope(r);
    if (st != SAGE_OK) return st;
    if (!Q || !Qo || !pos || (r->Hk > 0 && (!K || !Ko))) return SAGE_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(pos) & 3u) return SAGE_ERR_ALIGN;
    const void *ptrs[] = {Q, Qo, r->Hk > 0 ? K : nullptr, r->Hk > 0 ? Ko : nullptr};
    for (const void *p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & 15u) return SAGE_ERR_ALIGN;
    RopeArgs a;
    a.src[0] = Q; a.src[1] = K;
    a.dst[0] = Qo; a.dst[1] = Ko;
    a.pos = pos;
    a.H = r->H; a.Hk = r->Hk; a.N = r->N; a.d = r->d; a.rotary = r->rotary;
    a.tokens = r->B * r->N;
    a.pos_batch_stride = r->pos_batch == 1 ? 0 : r->N;
    a.pos_axis_stride = static_cast<long long>(r->pos_batch) * r->N;
    a.sign = r->inverse ? -1.0f : 1.0f;
    int j = 0;
    for (int ax = 0; ax < r->axes; ++ax)
        for (int i = 0; i < r->sections[ax]; ++i, ++j) {
            const double turns = r->freq[j] * 0.15915494309189533577;    // 1 / (2 pi)
            double frac = turns - floor(turns);
            if (frac >= 1.0) frac = 0.0;                                 // floor of a tiny negative
            a.f[j] = static_cast<unsigned long long>(frac * 18446744073709551616.0);
            a.axis[j] = static_cast<unsigned char>(ax);
        }
    // Heads a thread visits: as many as leave 152 SMs with about 2048 threads each, at most 8 in 16
    // bits, 4 in float32 (a sine then costs little beside the heads' loads; measured: 2 x 16 + 16 heads
    // of 8192 tokens in fp16 43.7 us at most 4, 42.7 at 8, 44.1 at 16; 4 x 16 + 16 of 4096 in float32
    // 85.6, 87.8, 87.2).
    const int per_row = r->d / 16, heads = r->H + r->Hk;
    const long long threads = static_cast<long long>(a.tokens) * per_row * heads;
    long long hpb = threads / (152ll * 2048);
    const int most = r->dtype == SAGE_FP32 ? 4 : 8;
    hpb = hpb < 1 ? 1 : hpb > most ? most : hpb;
    a.heads_per_block = static_cast<int>(hpb);
    const int tpb = kRopeThreads / per_row;
    const dim3 grid((a.tokens + tpb - 1) / tpb, (heads + a.heads_per_block - 1) / a.heads_per_block);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (r->dtype == SAGE_FP16) launch_rope_t<__half>(a, r->interleaved, grid, s);
    else if (r->dtype == SAGE_BF16) launch_rope_t<__nv_bfloat16>(a, r->interleaved, grid, s);
    else launch_rope_t<float>(a, r->interleaved, grid, s);
    return cudaGetLastError() == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA;
}
