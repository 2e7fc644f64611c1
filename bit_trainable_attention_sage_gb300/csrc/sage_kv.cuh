// sage_kv.cuh -- what the cache kernels (sage_kv.cu, sage_decode.cu) share: the device view of a
// paged key-value cache, the lookup of a slot's row with its bounds checks, and the checks of the
// C entry points.
#pragma once

#include "sage_device.cuh"
#include "sage_internal.h"

namespace sage {

struct KvView {
    void *K, *V;
    float *sK, *sV;
    const int *table;
    float *score;
    int *pos;
    int B, H, page, pages, max_pages, cap;   // cap = max_pages * page
};

// The page that holds slot s of sequence b, or -1 (and the error word raised) where the table's
// entry is not a page of the pool.  s must be in [0, cap).
__device__ __forceinline__ int kv_page(const KvView &c, int b, int s, unsigned int *err) {
    const int p = __ldg(c.table + static_cast<size_t>(b) * c.max_pages + s / c.page);
    if (static_cast<unsigned>(p) < static_cast<unsigned>(c.pages)) return p;
    atomicOr(err, 1u);
    return -1;
}

// Row (of d elements) of slot s of kv head h in page p: 64-bit, pools exceed 2^31 elements.
__device__ __forceinline__ size_t kv_row(const KvView &c, int p, int h, int s) {
    return (static_cast<size_t>(p) * c.H + h) * c.page + s % c.page;
}

// lens[b], held to [0, cap] (and the error word raised where it is not).
__device__ __forceinline__ int kv_len(const KvView &c, const int *lens, int b, unsigned int *err) {
    const int n = __ldg(lens + b);
    if (n >= 0 && n <= c.cap) return n;
    atomicOr(err, 1u);
    return n < 0 ? 0 : c.cap;
}

inline KvView kv_view(const sage_kv &c) {
    return KvView{c.K, c.V, c.sK, c.sV, c.table, c.score, c.pos, c.B, c.H, c.page, c.pages,
                  c.max_pages, c.max_pages * c.page};
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
