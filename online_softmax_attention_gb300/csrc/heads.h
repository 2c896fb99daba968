// Key / value head of a query head, of which a group of `group` share one: h / group as
// a product with the group's reciprocal.  The forward's loading warps look it up in front
// of every item's loads, where a division shows (500 packed sequences of 1 to 60 rows,
// ungrouped: 125.4 us a forward with one, 123.1 so).
#pragma once

#include "hd.h"

namespace attn {

// ceil(2^63 / group), group >= 1
ATTN_HD unsigned long long group_inverse(int group) { return ((1ull << 63) + group - 1) / group; }

// floor(h / group) for 0 <= h, group < 2^31: the product exceeds 2^63 h / group by less
// than h, and h / group lies 1 / group below the next whole number at least, so it is
// exact while h group < 2^63.
ATTN_HD int key_head(int h, unsigned long long inverse) {
#if defined(__CUDA_ARCH__)
    return (int)__umul64hi((unsigned long long)h << 1, inverse);
#else
    return (int)(((unsigned __int128)((unsigned long long)h << 1) * inverse) >> 64);
#endif
}

}  // namespace attn
