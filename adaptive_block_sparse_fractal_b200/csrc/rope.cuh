// Arguments of the rotary position kernels (rope.cu), passed by value.
#pragma once

#include <stdint.h>

namespace nabla {

constexpr int kRopeMaxPairs = 128;

struct RopeTensor {
    const void *in;
    void *out;
    int64_t in_batch, in_head, in_token, out_batch, out_head, out_token;  // elements
    int heads;
};

struct RopeArgs {
    RopeTensor t[2];
    int count, B, N, T, H, W, P, D, pairs;
    int flat_in, flat_out, heads_per_cta;
    const int32_t *pos;  // [B or 1, N, pos_axes] or null: grid coordinates
    int64_t pos_batch;
    int pos_axes;
    double offset[3];
    int8_t axis[kRopeMaxPairs];
    double turn[kRopeMaxPairs];  // turns (angle / 2 pi) per unit of position, sign included
};

}  // namespace nabla
