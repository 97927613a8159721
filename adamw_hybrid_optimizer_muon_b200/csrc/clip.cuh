// Device side of the clipping coefficient that grad_clip.cu leaves in a clip
// buffer: how the AdamW and momentum passes apply it to the gradients they read.
#pragma once

#include "internal.h"

namespace ma {

// coef * g; a zero coefficient (a norm that was not finite, or max_norm = 0)
// drops the gradient, infinities and NaN included. The product is rounded to
// fp32 on its own and kept opaque, so that what follows is compiled as it is
// for a gradient that was loaded: a clipped update has the bits of an update
// on gradients that hold the product.
__device__ __forceinline__ float clip_value(float g, float coef) {
    float r = coef == 0.f ? 0.f : __fmul_rn(g, coef);
    asm("" : "+f"(r));
    return r;
}

}  // namespace ma
