// sage_kv.cuh -- what the cache kernels (sage_kv.cu, sage_decode.cu) share: the device view of a
// paged key-value cache, the lookup of a slot's row with its bounds checks, and the checks of the
// C entry points.
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

struct KvView {
    void *K, *V;
    float *sK, *sV;
    const int *table;
    float *score;
    int *pos;
    int B, H, page, pages, max_pages, cap;   // cap = max_pages * page
    uint32_t page_mul, page_shift;           // s / page = s * page_mul >> page_shift for s < 2^30
};

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
    return KvView{c.K, c.V, c.sK, c.sV, c.table, c.score, c.pos, c.B, c.H, c.page, c.pages,
                  c.max_pages, c.max_pages * c.page, static_cast<uint32_t>(mul), 30 + k};
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
    if (c->kind != SAGE_KV_16 && c->kind != SAGE_KV_INT8 && c->kind != SAGE_KV_FP8) return SAGE_ERR_UNSUPPORTED;
    if (c->d != 64 && c->d != 128) return SAGE_ERR_UNSUPPORTED;
    if (c->page % 16 != 0) return SAGE_ERR_UNSUPPORTED;
    if (static_cast<long long>(c->max_pages) * c->page >= (1ll << 30)) return SAGE_ERR_UNSUPPORTED;
    if (static_cast<long long>(c->B) * c->H > 65535) return SAGE_ERR_UNSUPPORTED;
    if (!pointers) return SAGE_OK;
    if (!c->K || !c->V || !c->table) return SAGE_ERR_ARG;
    if (misaligned(c->K, 16) || misaligned(c->V, 16) || misaligned(c->table, 4)) return SAGE_ERR_ALIGN;
    if (c->kind == SAGE_KV_16 ? (c->sK || c->sV) : (!c->sK || !c->sV)) return SAGE_ERR_ARG;
    if (misaligned(c->sK, 16) || misaligned(c->sV, 16) || misaligned(c->score, 16) || misaligned(c->pos, 16))
        return SAGE_ERR_ALIGN;
    return SAGE_OK;
}

}  // namespace sage
