// sage_decode.h -- what the kernels over few query rows (sage_decode.cu) and over many (sage_extend.cu) share.
#pragma once

#include "sage_internal.h"

namespace sage {

constexpr int kSMs = 152;

// sage_decode.cu: T new tokens a sequence from slot start[b] on, count[b] of them there (NULL: all), over the
// one-token kernel, whose query heads the Hq * T rows become.
size_t decode_rows_bytes(const sage_kv &c, int Hq, int T);
cudaError_t decode_rows(const sage_kv &c, int Hq, int T, const void *Q, const int *start, const int *count, void *O,
                        float *L, void *workspace, cudaStream_t st);

// sage_extend.cu: nonzero if a bounded wait gave up; if a page, start or count was out of range (and clear it)
unsigned int take_extend_error();
unsigned int take_extend_index();

}  // namespace sage
