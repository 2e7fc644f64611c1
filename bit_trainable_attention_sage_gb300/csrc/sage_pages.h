// sage_pages.h -- the page calls' error word, and the arithmetic of places in the list of free pages.  Plain C++.
#pragma once

#ifdef __CUDACC__
#define SAGE_PAGES_FN __host__ __device__ __forceinline__
#else
#define SAGE_PAGES_FN inline
#endif

namespace sage {

// sage_pages.cu: which of the bits `which` are set (and clear them): 1 a page, length or sequence was out of
// range, 2 the pool had no free page left
unsigned int take_pages_error(unsigned int which);

// Pages that sequences together want, and a place among them: each wants fewer than 2^26, all of them (up to
// 65535) can want more than 32 bits hold, far more than any pool has.
using PageSum = long long;

SAGE_PAGES_FN PageSum pages_more(int want, int held) { return want > held ? want - held : 0; }

// How many of the `more` pages that a sequence wants it gets: those at place `first` and behind it, of `free`.
SAGE_PAGES_FN int pages_got(int more, PageSum first, int free) {
    const PageSum left = static_cast<PageSum>(free) - first;
    return left <= 0 ? 0 : left < more ? static_cast<int>(left) : more;
}

}  // namespace sage
