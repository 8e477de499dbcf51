// conv.hip -- short causal convolution with its state (gfx950).
//
//   z[t][c] = bias[c] + sum_w weight[c][w] x[t - W + 1 + w][c],  y = silu(z),
//   heads of the first channels brought to length one.
//
// A wave owns up to L tokens of one request and 512 channels (or as many whole heads as fit where
// they are brought to length one), eight neighbouring channels a lane; the last W - 1 rows stay in
// registers, so that every row of x is read once but for W - 1 rows in front of each unit.
#include "op.h"

#include <algorithm>

namespace vqmlp {

namespace {

constexpr int kAhead = 4;  // rows on their way

struct ConvArgs {
    const uint16_t *x, *w, *bias;
    uint16_t* y;
    const uint16_t* sin;
    uint16_t* sout;
    Packed p;
    int64_t ld_x, ld_y;
    int C, silu, unit_heads, unit_dim, unit_sets, lanes;  // sets of heads; lanes of a head
    int L, sets;
    int64_t id0;
    float eps;
};

template <class E>
__device__ __forceinline__ void unpack8(u32x4 w, float* f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[2 * j] = lo16<E>(w[j]), f[2 * j + 1] = hi16<E>(w[j]);
}

template <class E, int W>
__global__ void __launch_bounds__(256) k_short_conv(ConvArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t id = a.id0 + blockIdx.x;
    const int groups = (a.sets + 3) / 4;
    const int set = uniform(int(id % groups) * 4 + (threadIdx.x >> 6));
    PackedUnit u;
    if (!packed_unit(a.p, a.L, int(id / groups), u) || set >= a.sets) return;
    const bool unit = set < a.unit_sets;
    int c;  // first of the lane's channels
    bool in;
    if (unit) {
        const int head = set * (64 / a.lanes) + lane / a.lanes, at = lane % a.lanes * 8;
        c = head * a.unit_dim + at;
        in = head < a.unit_heads && at < a.unit_dim;
    } else {
        c = a.unit_heads * a.unit_dim + (set - a.unit_sets) * 512 + lane * 8;
        in = c < a.C;
    }
    const int t0 = u.seg * a.L, t1 = min(u.n, t0 + a.L);
    const u32x4 zero = {0, 0, 0, 0};
    if (u.r == a.p.R) {  // rows behind the last request
        for (int t = t0; t < t1; ++t)
            if (in) *reinterpret_cast<u32x4*>(a.y + (u.c0 + t) * a.ld_y + c) = zero;
        return;
    }
    bool old;
    const int slot = packed_slot(a.p, u.r, &old);
    const int64_t sbase = int64_t(max(slot, 0)) * (W - 1) * a.C + c;
    const uint16_t* const x = a.x + u.c0 * a.ld_x + c;
    // row t of the request; from -(W - 1) on those of its state
    auto row = [&](int t) __attribute__((always_inline)) {
        u32x4 r = zero;
        if (!in) return r;
        if (t >= 0) {
            if (t < u.n) r = *reinterpret_cast<const u32x4*>(x + t * a.ld_x);
        } else if (old) {
            r = *reinterpret_cast<const u32x4*>(a.sin + sbase + int64_t(t + W - 1) * a.C);
        }
        return r;
    };
    u32x4 ring[kAhead], before[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) before[j] = row(t0 - (W - 1) + j);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) ring[j] = t0 + j < t1 ? row(t0 + j) : zero;
    // The unit with the request's first rows is the only one that reads its state, and so the one that
    // writes the new one, also where both are one array.
    if (u.seg == 0 && slot >= 0) {
        u32x4 next[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) next[j] = row(u.n - (W - 1) + j);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            if (in) *reinterpret_cast<u32x4*>(a.sout + sbase + int64_t(j) * a.C) = next[j];
    }
    float wt[W][8], bias[8], win[W][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) bias[i] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w)  // the lane's 8 W filter taps lie one after another
#pragma unroll
        for (int i = 0; i < 8; ++i) wt[w][i] = 0.f;
    if (in) {
        float f[8 * W];
#pragma unroll
        for (int j = 0; j < W; ++j) unpack8<E>(*reinterpret_cast<const u32x4*>(a.w + int64_t(c) * W + 8 * j), f + 8 * j);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int w = 0; w < W; ++w) wt[w][i] = f[i * W + w];
        if (a.bias) unpack8<E>(*reinterpret_cast<const u32x4*>(a.bias + c), bias);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) unpack8<E>(before[j], win[j + 1]);
    for (int t = t0; t < t1; t += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (t + j >= t1) break;
#pragma unroll
            for (int w = 0; w < W - 1; ++w)
#pragma unroll
                for (int i = 0; i < 8; ++i) win[w][i] = win[w + 1][i];
            unpack8<E>(ring[j], win[W - 1]);
            if (t + j + kAhead < t1) ring[j] = row(t + j + kAhead);
            float z[8], sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                z[i] = bias[i];
#pragma unroll
                for (int w = 0; w < W; ++w) z[i] = fmaf(wt[w][i], win[w][i], z[i]);
                if (a.silu) z[i] = silu(z[i]);
            }
            if (unit) {
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = fmaf(z[i], z[i], sum);
                for (int o = 1; o < a.lanes; o <<= 1) sum += __shfl_xor(sum, o);
                const float by = 1.f / sqrtf(sum + a.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] *= by;
            }
            if (in)
                *reinterpret_cast<u32x4*>(a.y + (u.c0 + t + j) * a.ld_y + c) =
                    u32x4{pack16<E>(z[0], z[1]), pack16<E>(z[2], z[3]), pack16<E>(z[4], z[5]), pack16<E>(z[6], z[7])};
        }
    }
}

template <class E>
void launch_conv(ConvArgs a, int W, int64_t all, hipStream_t s) {
    constexpr int64_t most = 8 << 20;  // a launch holds fewer than 2^32 threads
    for (int64_t at = 0; at < all; at += most) {
        const unsigned grid = unsigned(std::min(most, all - at));
        a.id0 = at;
        if (W == 2) k_short_conv<E, 2><<<grid, 256, 0, s>>>(a);
        else if (W == 3) k_short_conv<E, 3><<<grid, 256, 0, s>>>(a);
        else k_short_conv<E, 4><<<grid, 256, 0, s>>>(a);
    }
}

}  // namespace

}  // namespace vqmlp

extern "C" vqmlp_status vqmlp_short_conv(const vqmlp_conv_desc* p, void* stream) {
    using namespace vqmlp;
    OP_REQUIRE(p, "vqmlp_short_conv: null description");
    const vqmlp_conv_desc& d = *p;
    OP_REQUIRE(op_dtype16(d.dtype), "vqmlp_short_conv: dtype %d is not F16 or BF16", d.dtype);
    OP_REQUIRE(d.T >= 0 && d.R >= 1 && d.n_states >= 0 && d.unit_heads >= 0, "vqmlp_short_conv: a size is out of range");
    OP_REQUIRE(d.C >= 8 && d.C % 8 == 0, "vqmlp_short_conv: C=%d is not a multiple of 8", d.C);
    OP_REQUIRE(d.W >= 2 && d.W <= 4, "vqmlp_short_conv: W=%d is not 2, 3 or 4", d.W);
    if (d.R > 65535 || d.T > 0x3FFFFFFF || d.C > 1 << 20)
        OP_FAIL(VQMLP_ERR_UNSUPPORTED, "vqmlp_short_conv: R above 65535, T above 2^30 - 1 or C above 2^20");
    OP_REQUIRE(d.unit_heads == 0 || (d.unit_dim >= 8 && d.unit_dim <= 256 && d.unit_dim % 8 == 0),
               "vqmlp_short_conv: unit_dim=%d is not a multiple of 8 up to 256", d.unit_dim);
    OP_REQUIRE(d.unit_heads == 0 || int64_t(d.unit_heads) * d.unit_dim <= d.C,
               "vqmlp_short_conv: the unit heads pass C");
    OP_REQUIRE(d.unit_heads == 0 || (d.eps >= 0.f && d.eps - d.eps == 0.f), "vqmlp_short_conv: eps is negative or not finite");
    OP_REQUIRE(d.cu_q && op_aligned(d.cu_q, 4) && op_aligned(d.ctx_len, 4) && op_aligned(d.state_index, 4),
               "vqmlp_short_conv: null cu_q or an unaligned index array");
    OP_REQUIRE((d.state_in && d.state_out) || d.n_states == 0, "vqmlp_short_conv: null state");
    OP_REQUIRE(op_aligned(d.state_in, 16) && op_aligned(d.state_out, 16),
               "vqmlp_short_conv: states have to be 16-byte aligned");
    OP_REQUIRE(d.weight && op_aligned(d.weight, 16) && op_aligned(d.bias, 16),
               "vqmlp_short_conv: weight is null, or weight or bias not 16-byte aligned");
    if (d.T > 0) {
        OP_REQUIRE(d.x && d.y && op_aligned(d.x, 16) && op_aligned(d.y, 16),
                   "vqmlp_short_conv: x or y is null or not 16-byte aligned");
        OP_REQUIRE(d.x != d.y, "vqmlp_short_conv: y is x");
        for (const int64_t ld : {d.ld_x, d.ld_y})
            OP_REQUIRE((d.T == 1 || ld >= d.C) && ld >= 0 && ld <= 1 << 24 && ld % 8 == 0,
                       "vqmlp_short_conv: token strides have to be multiples of 8 from C up to 2^24");
    }
    int cus = 0;
    if (const int st = device_cus(&cus)) return static_cast<vqmlp_status>(st);
    ConvArgs a{};
    a.x = static_cast<const uint16_t*>(d.x);
    a.w = static_cast<const uint16_t*>(d.weight);
    a.bias = static_cast<const uint16_t*>(d.bias);
    a.y = static_cast<uint16_t*>(d.y);
    a.sin = static_cast<const uint16_t*>(d.state_in);
    a.sout = static_cast<uint16_t*>(d.state_out);
    a.p = Packed{d.cu_q, d.ctx_len, d.state_index, d.T, d.R, d.n_states};
    a.ld_x = d.ld_x;
    a.ld_y = d.ld_y;
    a.C = d.C;
    a.silu = d.silu;
    a.unit_heads = d.unit_heads;
    a.unit_dim = d.unit_heads ? d.unit_dim : 0;
    a.eps = d.eps;
    a.lanes = 1;
    while (a.lanes * 8 < a.unit_dim) a.lanes *= 2;
    a.unit_sets = (d.unit_heads * a.lanes + 63) / 64;
    a.sets = a.unit_sets + (d.C - d.unit_heads * a.unit_dim + 511) / 512;
    a.L = 32;
    const int64_t units = d.T / a.L + d.R + 1, all = units * ((a.sets + 3) / 4);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (d.dtype == VQMLP_F16) launch_conv<F16>(a, d.W, all, s);
    else launch_conv<BF16>(a, d.W, all, s);
    if (trace_enabled())
        trace_line("short_conv T=%d R=%d C=%d W=%d: units of %d tokens, %d channel sets", d.T, d.R, d.C, d.W, a.L, a.sets);
    return op_launched("vqmlp_short_conv");
}
