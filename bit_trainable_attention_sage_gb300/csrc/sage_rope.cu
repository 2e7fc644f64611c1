// sage_rope.cu -- rotary positions with several axes, forward and inverse (the gradient).
//
// y0 = x0 cos - x1 sin, y1 = x0 sin + x1 cos for each of a token's pairs.  Every element is read
// and written once, so the kernel is bound by memory bandwidth; what must not show is the cost of
// the angles.  One thread holds the sines and cosines of 8 pairs of one token in registers and
// uses them for every head it visits, so a sine is computed once per (token, pair, head chunk).
//
// The angle of pair j at position p is p * freq[j] mod 2 pi.  In units of a turn, freq[j] / 2 pi
// mod 1 is held as a 64-bit fixed-point fraction f (whole turns a position vanish because p is an
// integer), and p * f mod 2^64 is then one wrapping integer product: the error is |p| 2^-64 of a
// turn plus |p| times that of freq[j] / 2 pi in float64, where a float32 product p * freq[j] would
// be off by a good part of a radian for far positions.  Its top 32 bits, read as a signed number of
// half turns in [-1, 1), go to sincospif.
#include <math.h>

#include "sage_device.cuh"
#include "sage_internal.h"

namespace sage {

constexpr int kRopeThreads = 128;
constexpr int kRopeMaxPairs = 64;        // d = 128

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

template <typename T>
__device__ __forceinline__ void rope_load8(const T *p, float (&v)[8]) {
    if constexpr (std::is_same<T, float>::value) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
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
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = v * 8 + i;
            const long long p = pos[static_cast<long long>(a.axis[j]) * a.pos_axis_stride];
            const unsigned long long t = static_cast<unsigned long long>(p) * a.f[j];
            const float half_turns = static_cast<float>(static_cast<int>(t >> 32)) * 4.656612873077393e-10f;   // 2^-31
            sincospif(half_turns, &sn[i], &cs[i]);
            sn[i] *= a.sign;
        }
    }
    const int h0 = blockIdx.y * a.heads_per_block;
    const int h1 = min(h0 + a.heads_per_block, a.H + a.Hk);
#pragma unroll 2
    for (int h = h0; h < h1; ++h) {
        const bool isk = h >= a.H;
        const int heads = isk ? a.Hk : a.H, hh = isk ? h - a.H : h;
        const size_t row = ((static_cast<size_t>(b) * heads + hh) * a.N + n) * a.d;
        const T *src = static_cast<const T *>(a.src[isk]) + row;
        T *dst = static_cast<T *>(a.dst[isk]) + row;
        float x[8], y[8];
        rope_load8(src + c0, x);
        rope_load8(src + c1, y);
        if (turns) {
            float o0[8], o1[8];
            if constexpr (INTERLEAVED) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o0[2 * i] = x[2 * i] * cs[i] - x[2 * i + 1] * sn[i];
                    o0[2 * i + 1] = x[2 * i] * sn[i] + x[2 * i + 1] * cs[i];
                    o1[2 * i] = y[2 * i] * cs[4 + i] - y[2 * i + 1] * sn[4 + i];
                    o1[2 * i + 1] = y[2 * i] * sn[4 + i] + y[2 * i + 1] * cs[4 + i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    o0[i] = x[i] * cs[i] - y[i] * sn[i];
                    o1[i] = x[i] * sn[i] + y[i] * cs[i];
                }
            }
            rope_store8(dst + c0, o0);
            rope_store8(dst + c1, o1);
        } else {
            rope_store8(dst + c0, x);
            rope_store8(dst + c1, y);
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
    // Heads a thread visits: as many as leave 152 SMs with about 2048 threads each, at most 8 (a
    // sine then costs an eighth of what a head's loads and arithmetic do).
    const int per_row = r->d / 16, heads = r->H + r->Hk;
    const long long threads = static_cast<long long>(a.tokens) * per_row * heads;
    long long hpb = threads / (152ll * 2048);
    hpb = hpb < 1 ? 1 : hpb > 8 ? 8 : hpb;
    a.heads_per_block = static_cast<int>(hpb);
    const int tpb = kRopeThreads / per_row;
    const dim3 grid((a.tokens + tpb - 1) / tpb, (heads + a.heads_per_block - 1) / a.heads_per_block);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (r->dtype == SAGE_FP16) launch_rope_t<__half>(a, r->interleaved, grid, s);
    else if (r->dtype == SAGE_BF16) launch_rope_t<__nv_bfloat16>(a, r->interleaved, grid, s);
    else launch_rope_t<float>(a, r->interleaved, grid, s);
    return cudaGetLastError() == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA;
}
