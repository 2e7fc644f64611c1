// sage_pages.h -- the page calls' error word.
#pragma once

namespace sage {

// sage_pages.cu: which of the bits `which` are set (and clear them): 1 a page, length or sequence was out of
// range, 2 the pool had no free page left
unsigned int take_pages_error(unsigned int which);

}  // namespace sage
