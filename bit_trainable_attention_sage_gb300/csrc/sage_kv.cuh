// sage_kv.cuh -- what the cache kernels (sage_kv.cu, sage_decode.cu, sage_extend.cu, sage_pages.cu) share: the device view
// of a paged key-value cache, the lookup of a slot's row with its bounds checks, codes widened to 16 bits, copies to
// shared memory, and the checks of the C entry points.
#pragma once

#include "sage_device.cuh"
#include "sage_internal.h"

namespace sage {

// sage_kv.cu, sage_decode.cu: nonzero if a page, length or slot was out of range (and clear it)
unsigned int take_kv_error();
unsigned int take_decode_error();

// ---- thread-block clusters ---------------------------------------------------------------------
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the word at this address of CTA `rank`'s shared memory
__device__ __forceinline__ int cluster_word(const int *p, int rank) {
    uint32_t at;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ long long cluster_long(const long long *p, int rank) {
    uint32_t at;
    long long v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float cluster_float(const float *p, int rank) {
    return __int_as_float(cluster_word(reinterpret_cast<const int *>(p), rank));
}
// and the four (16-byte aligned)
__device__ __forceinline__ int4 cluster_words(const int *p, int rank) {
    uint32_t at;
    int4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.s32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// ---- copies to shared memory that a thread does not wait for ------------------------------------
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    const int n = valid ? 16 : 0;            // 0: the 16 bytes are zeroed and nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ---- codes in 16 bits -------------------------------------------------------------------------
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

// Four codes as two pairs of fp16 or bf16.  All exact.
//   fp16: INT8: byte ^ 0x80 under 0x64 is 1024 + 128 + code, less 1152 the code; E4M3 by the conversion instruction.
//   bf16: INT8: the low seven bits under 0x43 are 128 + them, the sign under 0x43 128 or 256; E4M3 through float32.
template <bool BF16, bool FP8>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (FP8) {
        lo = e4m3x2_to_f16x2(static_cast<uint16_t>(w & 0xFFFFu));
        hi = e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
        if constexpr (BF16) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo)), b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
            const __nv_bfloat162 x = __floats2bfloat162_rn(a.x, a.y), y = __floats2bfloat162_rn(b.x, b.y);
            lo = *reinterpret_cast<const uint32_t *>(&x);
            hi = *reinterpret_cast<const uint32_t *>(&y);
        }
    } else if constexpr (BF16) {
        const uint32_t u = w & 0x7F7F7F7Fu, s = w & 0x80808080u, k = 0x43434343u;
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(prmt(u, k, 0x4140)), "r"(prmt(s, k, 0x4140)));
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(prmt(u, k, 0x4342)), "r"(prmt(s, k, 0x4342)));
    } else {
        const uint32_t u = w ^ 0x80808080u, k = 0x64806480u;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(prmt(u, 0x64646464u, 0x4140)), "r"(k));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(prmt(u, 0x64646464u, 0x4342)), "r"(k));
    }
}

// Which 16-bit values (E4M3 codes) of a word are not finite, as a mask of their bits.
template <bool BF16, bool FP8>
__device__ __forceinline__ uint32_t not_finite_mask(uint32_t w) {
    if constexpr (FP8) return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    else if constexpr (BF16) return __vcmpeq2(w & 0x7F807F80u, 0x7F807F80u);
    else return __vcmpeq2(w & 0x7C007C00u, 0x7C007C00u);
}

struct KvView {
    void *K, *V;
    float *sK, *sV;
    const int *table;
    float *score;
    int *pos;
    int B, H, page, pages, max_pages, cap;   // cap = max_pages * page
    uint32_t page_mul, page_shift;           // s / page = s * page_mul >> page_shift for s < 2^30
    int block_shift;                         // row >> block_shift: its scale's place (0: a scale a row)
};

// struct sage_kv's kind: the rows' format, and the tokens that share a scale (0: each row has its own)
inline int kv_format(const sage_kv &c) { return c.kind & 255; }
inline int kv_block(const sage_kv &c) { return c.kind >> 8; }

// s / page without a division: page_mul = ceil(2^(30 + k) / page) with 2^k >= page exceeds the
// quotient by less than 2^k / page / 2^(30 + k) of s, so by less than 1 / page for s < 2^30: the
// floor is exact.
__device__ __forceinline__ int kv_page_of(const KvView &c, int s) {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(s)) * c.page_mul) >> c.page_shift);
}

// The page that holds slot s of sequence b, or -1 (and the error word raised) where the table's
// entry is not a page of the pool.  s must be in [0, cap).
__device__ __forceinline__ int kv_page(const KvView &c, int b, int s, unsigned int *err) {
    const int p = __ldg(c.table + static_cast<size_t>(b) * c.max_pages + kv_page_of(c, s));
    if (static_cast<unsigned>(p) < static_cast<unsigned>(c.pages)) return p;
    atomicOr(err, 1u);
    return -1;
}

// Row (of d elements) of slot s of kv head h in page p: 64-bit, pools exceed 2^31 elements.
__device__ __forceinline__ size_t kv_row(const KvView &c, int p, int h, int s) {
    return (static_cast<size_t>(p) * c.H + h) * c.page + (s - kv_page_of(c, s) * c.page);
}

// lens[b], held to [0, cap] (and the error word raised where it is not).
__device__ __forceinline__ int kv_len(const KvView &c, const int *lens, int b, unsigned int *err) {
    const int n = __ldg(lens + b);
    if (n >= 0 && n <= c.cap) return n;
    atomicOr(err, 1u);
    return n < 0 ? 0 : c.cap;
}

inline KvView kv_view(const sage_kv &c) {
    uint32_t k = 0;
    while ((1ull << k) < static_cast<uint64_t>(c.page)) ++k;
    const uint64_t mul = ((1ull << (30 + k)) + c.page - 1) / c.page;     // at most 2^31
    int shift = 0;
    while ((1 << shift) < kv_block(c)) ++shift;
    return KvView{c.K, c.V, c.sK, c.sV, c.table, c.score, c.pos, c.B, c.H, c.page, c.pages,
                  c.max_pages, c.max_pages * c.page, static_cast<uint32_t>(mul), 30 + k, shift};
}

// A kernel's dynamic shared-memory limit, raised once a device (`raised`; again is harmless).
inline cudaError_t raise_smem(const void *kernel, size_t bytes, bool (&raised)[16]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 16 && raised[dev])) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess && dev < 16) raised[dev] = true;
    return e;
}

// Whether two ranges of bytes share one.
inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}
inline bool misaligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// The rules of struct sage_kv (`pointers` false: sizes only, for the workspace queries).
inline int check_kv(const sage_kv *c, bool pointers) {
    if (!c) return SAGE_ERR_ARG;
    if (c->B <= 0 || c->H <= 0 || c->d <= 0 || c->page <= 0 || c->pages <= 0 || c->max_pages <= 0) return SAGE_ERR_ARG;
    if (c->dtype != SAGE_FP16 && c->dtype != SAGE_BF16) return SAGE_ERR_UNSUPPORTED;
    const int format = kv_format(*c), block = kv_block(*c);
    if (c->kind < 0 || (format != SAGE_KV_16 && format != SAGE_KV_INT8 && format != SAGE_KV_FP8)) return SAGE_ERR_UNSUPPORTED;
    // blocks of 16, 32 or 64 rows that divide the page, in 8 bits, and not with what eviction needs: it moves single rows
    if (block && (format == SAGE_KV_16 || (block != 16 && block != 32 && block != 64) || c->page % block != 0 || c->score || c->pos))
        return SAGE_ERR_UNSUPPORTED;
    if (c->d != 64 && c->d != 128) return SAGE_ERR_UNSUPPORTED;
    if (c->page % 16 != 0) return SAGE_ERR_UNSUPPORTED;
    if (static_cast<long long>(c->max_pages) * c->page >= (1ll << 30)) return SAGE_ERR_UNSUPPORTED;
    if (static_cast<long long>(c->B) * c->H > 65535) return SAGE_ERR_UNSUPPORTED;
    if (!pointers) return SAGE_OK;
    if (!c->K || !c->V || !c->table) return SAGE_ERR_ARG;
    if (misaligned(c->K, 16) || misaligned(c->V, 16) || misaligned(c->table, 4)) return SAGE_ERR_ALIGN;
    if (format == SAGE_KV_16 ? (c->sK || c->sV) : (!c->sK || !c->sV)) return SAGE_ERR_ARG;
    if (misaligned(c->sK, 16) || misaligned(c->sV, 16) || misaligned(c->score, 16) || misaligned(c->pos, 16))
        return SAGE_ERR_ALIGN;
    return SAGE_OK;
}

}  // namespace sage
