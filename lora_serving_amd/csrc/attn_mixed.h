// The order of the workgroups of a launch that holds two kinds of them.
#pragma once

#include "attention.h"

namespace mlora {

// Workgroup *i of `wide` wide ones and `shares` others: is it a wide one, and (*i) which of its kind.
__device__ __forceinline__ bool mixed_place(uint32_t wide, uint32_t shares, uint32_t *at)
{
    // the first 256 of the wide ones, the first 256 of the others, then groups of each in turn.  Workgroups go to the 8
    // XCDs, and within one to its shader engines and their CUs, in turn: smaller groups would give each kind to some
    // of them alone (groups of 8: a chunk of 2048 with empty shares between 319 us, groups of 256 232).
    constexpr uint32_t GROUP = 256;
    const uint32_t w0 = min(wide, (uint32_t)CUS), d0 = min(shares, (uint32_t)CUS);
    uint32_t i = *at;
    bool is_wide = i < w0;
    if (!is_wide) {
        i -= w0;
        if (i >= d0) {
            i -= d0;
            const uint32_t both = min(wide - w0, shares - d0) & ~(GROUP - 1);
            if (i < 2 * both) {
                is_wide = (i / GROUP & 1) == 0;
                i = i / (2 * GROUP) * GROUP + (i & (GROUP - 1)) + (is_wide ? w0 : d0);
            } else {
                i -= 2 * both;
                is_wide = i < wide - w0 - both;
                i = is_wide ? i + w0 + both : i - (wide - w0 - both) + d0 + both;
            }
        }
    }
    *at = i;
    return is_wide;
}

}  // namespace mlora
