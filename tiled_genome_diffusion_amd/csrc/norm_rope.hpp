// Arguments and launchers of the norm of queries and keys per head with the
// position rotation (norm_rope.hip).
#pragma once

#include "attn.hpp"

namespace pc {

constexpr int kMaxPairs2 = 64;  // rotated pairs of a head of 128

struct NormSide {
    const void *x, *dy;
    void *y, *dx;            // y: forward's output; dx: backward's
    const float *w;          // [D] or null (ones)
    float *dw;               // [D] or null
    const int32_t *pos;      // [.][len] or null (0 .. len - 1)
    int64_t pos_b;           // elements between batches of pos
    HeadStrides sx, sy, sdy, sdx;
    FastDiv len, heads;
    int64_t tokens;          // batch * len
    uint32_t tiles;          // of `tile` tokens
    uint32_t blocks;         // workgroups of this side
    float *part;             // backward: [blocks][D] partial sums of dw
};

struct NormArgs {
    NormSide side[2];        // queries, keys (tokens = 0: absent)
    uint64_t turns[kMaxPairs2];  // 2^64 * (angle per position of pair i) / 2 pi, modulo 2^64
    int32_t D, half;         // head size, rotated pairs
    FastDiv per;             // D - half: pairs and values that are not rotated
    uint32_t tile;           // tokens a workgroup takes at a time
    float eps, inv_d;
};

int64_t norm_bwd_workspace(NormArgs &a, int32_t dtype);
hipError_t launch_norm_fwd(NormArgs &a, int32_t dtype, bool interleaved, hipStream_t stream);
hipError_t launch_norm_bwd(NormArgs &a, int32_t dtype, bool interleaved, char *workspace, hipStream_t stream);

}  // namespace pc
