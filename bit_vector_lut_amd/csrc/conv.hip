// conv.hip -- short causal convolution with its state (gfx950).
//
//   z[t][c] = bias[c] + sum_w weight[c][w] x[t - W + 1 + w][c],  y = silu(z),
//   heads of the first channels brought to length one.
//
// A wave owns up to L tokens of one request and 512 channels (or as many whole heads as fit where
// they are brought to length one), eight neighbouring channels a lane; the last W - 1 rows stay in
// registers, so that every row of x is read once but for the W - 1 rows in front of each unit, which a
// neighbour has just read. Sums are FP32, the outputs' rounding is the only one to 16 bits.
//
// Bound by memory for prompts: 8,073 tokens of 10,240 FP16 channels, W = 4, 32 heads of 128 to length one,
// in 66 us, 331 MB at 5.0 TB/s. What it took: whole rounds of four rows without a branch between
// them, so that four rows are on their way and the sums over heads of four tokens are taken together
// (104 -> 73 us); units of 16 tokens instead of 32 (-> 66; 64: 74). Eight rows on their way need 172
// registers, and two waves on a SIMD instead of three (binary16, W = 4: 134 registers) cost more than the loads give (130 us).
// Bound by latency for few tokens: the search for the unit, one round of loads, one row's sums.
// 8 tokens in 5.2 us, 64 requests with a token each in 5.8 us.
#include "op.h"

#include <algorithm>

namespace vqmlp {

namespace {

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
    // rows on their way: a multiple of W, so that the last W rows stand where the unrolled loop finds them
    constexpr int AHEAD = W == 3 ? 3 : 4;
    const int lane = threadIdx.x & 63;
    const int64_t id = a.id0 + blockIdx.x;
    const int groups = (a.sets + 3) / 4;
    const int set = uniform(int(id % groups) * 4 + (threadIdx.x >> 6));
    if (set >= a.sets) return;
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
    if (!in) c = 0;  // such lanes read the first channels, count nothing and write nothing
    // the lane's 8 W filter taps lie one after another; on their way while the unit is looked for
    const u32x4 zero = {0, 0, 0, 0};
    u32x4 taps[W], bits = zero;
#pragma unroll
    for (int j = 0; j < W; ++j) taps[j] = *reinterpret_cast<const u32x4*>(a.w + int64_t(c) * W + 8 * j);
    if (a.bias) bits = *reinterpret_cast<const u32x4*>(a.bias + c);
    PackedUnit u;
    if (!packed_unit(a.p, a.L, int(id / groups), u)) return;
    const int t0 = u.seg * a.L, t1 = min(u.n, t0 + a.L);
    uint16_t* y = a.y + (u.c0 + t0) * a.ld_y + c;
    if (u.r == a.p.R) {  // rows behind the last request
        for (int t = t0; t < t1; ++t, y += a.ld_y)
            if (in) *reinterpret_cast<u32x4*>(y) = zero;
        return;
    }
    bool old;
    const int slot = packed_slot(a.p, u.r, &old);
    const int64_t sbase = int64_t(max(slot, 0)) * (W - 1) * a.C + c;
    const uint16_t* const x = a.x + u.c0 * a.ld_x + c;
    // row t < n of the request; from -(W - 1) on those of its state
    auto row = [&](int t) __attribute__((always_inline)) {
        if (t >= 0) return *reinterpret_cast<const u32x4*>(x + t * a.ld_x);
        return old ? *reinterpret_cast<const u32x4*>(a.sin + sbase + int64_t(t + W - 1) * a.C) : zero;
    };
    u32x4 ring[AHEAD], before[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) before[j] = row(t0 - (W - 1) + j);
    if (t0 < t1) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) ring[j] = row(min(t0 + j, t1 - 1));
    }
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
    float wt[W][8], bias[8], win[W][8];  // row t of the unit stands in win[t % W]
    {
        float f[8 * W];
#pragma unroll
        for (int j = 0; j < W; ++j) unpack8<E>(taps[j], f + 8 * j);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int w = 0; w < W; ++w) wt[w][i] = f[i * W + w];
        unpack8<E>(bits, bias);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) unpack8<E>(before[j], win[j + 1]);
    auto rows = [&](auto count, int t) __attribute__((always_inline)) {
        constexpr int N = decltype(count)::value;
        float z[N][8];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            unpack8<E>(ring[j], win[j % W]);
            ring[j] = *reinterpret_cast<const u32x4*>(x + min(t + j + AHEAD, t1 - 1) * a.ld_x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                z[j][i] = bias[i];
#pragma unroll
                for (int w = 0; w < W; ++w) z[j][i] = fmaf(wt[w][i], win[(j + 1 + w) % W][i], z[j][i]);
                if (a.silu) z[j][i] = silu(z[j][i]);
            }
        }
        if (unit) {
            float sum[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                sum[j] = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[j] = fmaf(z[j][i], z[j][i], sum[j]);
                if (!in) sum[j] = 0.f;
            }
            head_sums(sum, a.lanes);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float by = __builtin_amdgcn_rsqf(sum[j] + a.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[j][i] *= by;
            }
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (in)
                *reinterpret_cast<u32x4*>(y) = u32x4{pack16<E>(z[j][0], z[j][1]), pack16<E>(z[j][2], z[j][3]),
                                                     pack16<E>(z[j][4], z[j][5]), pack16<E>(z[j][6], z[j][7])};
            y += a.ld_y;
        }
    };
    int t = t0;
    for (; t + AHEAD <= t1; t += AHEAD) rows(std::integral_constant<int, AHEAD>{}, t);
    for (; t < t1; ++t) {
        rows(std::integral_constant<int, 1>{}, t);
#pragma unroll
        for (int j = 0; j + 1 < AHEAD; ++j) ring[j] = ring[j + 1];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int j = 1; j < W - 1; ++j) win[j][i] = win[j + 1][i];
            win[W - 1][i] = win[0][i];
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
    // Tokens of a unit: whole rounds of rows, 16 (15) where there are tokens enough for two waves on each of the card's
    // SIMDs, fewer where not.  Never fewer than W - 1: the second unit would read the state that the first writes.
    const int step = d.W == 3 ? 3 : 4;
    a.L = int(std::min<int64_t>(16 / step, std::max<int64_t>(1, int64_t(d.T) * a.sets / (8 * cus * step)))) * step;
    const int64_t units = d.T / a.L + d.R + 1, all = units * ((a.sets + 3) / 4);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (d.dtype == VQMLP_F16) launch_conv<F16>(a, d.W, all, s);
    else launch_conv<BF16>(a, d.W, all, s);
    if (trace_enabled())
        trace_line("short_conv T=%d R=%d C=%d W=%d: units of %d tokens, %d channel sets", d.T, d.R, d.C, d.W, a.L, a.sets);
    return op_launched("vqmlp_short_conv");
}
