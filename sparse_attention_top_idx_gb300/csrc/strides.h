// strides.h -- whether the rows of a strided tensor share elements (host only).
#pragma once

#include <stdint.h>

namespace dsaidx {

// [tokens, heads] rows of `width` consecutive elements at any strides: true
// where no two rows share an element.  Rows (i, j) and (i + a, j + b) do where
// |a ts + b hs| < width.  A dimension of one row has no stride.
inline bool rows_apart(int64_t tokens, int64_t heads, int64_t width, int64_t token_stride, int64_t head_stride) {
    typedef __int128 wide;      // products of any two arguments
    wide ts = token_stride, hs = head_stride, nt = tokens, nh = heads;
    if (ts < 0) ts = -ts;
    if (hs < 0) hs = -hs;
    if (nt > 1 && ts < width) return false;
    if (nh > 1 && hs < width) return false;
    if (nt <= 1 || nh <= 1) return true;
    // one dimension steps over all of the other
    if (ts >= (nh - 1) * hs + width || hs >= (nt - 1) * ts + width) return true;
    // they interleave: for each b of the shorter one the two nearest a
    if (nt < nh) {
        wide t = ts;
        ts = hs, hs = t;
        t = nt;
        nt = nh, nh = t;
    }
    for (wide b = 1; b < nh; ++b) {
        const wide at = b * hs, a = at / ts, rest = at - a * ts;
        if (a < nt && rest < width) return false;
        if (a + 1 < nt && ts - rest < width) return false;
    }
    return true;
}

}  // namespace dsaidx
