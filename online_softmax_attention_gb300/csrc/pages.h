// Lengths of cached sequences and the pages that hold them, for any 32-bit value that
// the caller's `lens` may hold.
#pragma once

#include "hd.h"

namespace attn {

// Pages of 2^shift rows that hold `tokens` >= 0 tokens.  (Rounding up by adding a page's
// size first would pass 2^31 and come out negative.)
ATTN_HD int pages_of(int tokens, int shift) { return (tokens >> shift) + ((tokens & ((1 << shift) - 1)) != 0); }

// Whether a sequence of max_pages pages of 2^shift rows can have that length.
ATTN_HD bool length_fits(int len, int max_pages, int shift) {
    return len >= 0 && (long long)len <= (long long)max_pages << shift;
}

}  // namespace attn
