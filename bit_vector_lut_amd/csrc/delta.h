// delta.h -- shared by the gated delta rule's kernels (delta.hip, delta_chunk.hip).
#pragma once
#include "op.h"

namespace vqmlp {

constexpr int kDeltaC = 64;  // tokens of a chunk
constexpr int kDeltaBlock = 26624;  // bytes of a chunk and value head in the workspace

struct DeltaArgs {
    const uint16_t *q, *k, *v;
    const float *g, *beta;
    uint16_t* y;
    const float* sin;
    float* sout;
    Packed p;
    uint8_t* blocks;   // [unit][v_heads][kDeltaBlock]
    uint16_t* images;  // [unit][k_heads] queries in binary16 as operands, of bfloat16 inputs also keys, [64][Dk padded] each
    int64_t ld_q, ld_k, ld_v, ld_y, ld_g, ld_b;
    // Of segments (NULL: whole requests): [unit][v_heads][Dk][Dv] states, then [unit][v_heads][Dk][Dk] factors.
    float* seg;
    int64_t seg_units;
    int64_t id0;       // number of the launch's first workgroup
    int h0;            // of the recurrence: the launch's first head
    int L;             // tokens of a segment
    int few;           // requests of up to so many tokens go through the recurrence, the others in chunks
    int hk, hv, Dk, Dv;
    float scale;

    __device__ uint16_t* image(int64_t unit, int head, int dkp, bool half) const {
        return images + (unit * hk + head) * ((half ? 1 : 2) * kDeltaC * dkp);
    }
    __device__ float* ends(int64_t unit, int h) const { return seg + (unit * hv + h) * Dk * Dv; }
    __device__ float* factor(int64_t unit, int h) const {
        return seg + seg_units * hv * Dk * Dv + (unit * hv + h) * Dk * Dk;
    }
};

// Chunks of 64 tokens on the matrix cores.
template <class E>
void launch_delta_chunks(const DeltaArgs& a, int cus, hipStream_t s);

}  // namespace vqmlp
