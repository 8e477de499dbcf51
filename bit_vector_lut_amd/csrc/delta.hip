// delta.hip -- gated delta rule (gfx950).
//
//   S' = e^{g_t} S_{t-1},  u_t = beta_t (v_t - S'^T k_t),  S_t = S' + k_t u_t^T,  y_t = scale S_t^T q_t.
#include "delta.h"

#include <algorithm>
#include <climits>

namespace vqmlp {

namespace {

constexpr int64_t kMaxLd = 1 << 24;

// ---------------------------------------------------------------- the recurrence
// A wave owns a head's Dk x 32 (or 16) columns of the state: lane = (row block, four columns), a row block's
// rows contiguous so that a token's q and k come as 16-byte chunks.  Both sums over the rows are taken over
// the state before the token: y_t = scale (e^{g} S^T q + (k . q) u), so one round of lane moves serves both.
// No LDS and no barrier.
// Many requests: bound by reading and writing the states (64 requests of 48 heads of 128 x 128, a token each: 402 MB
// in 73 to 87 us).  Few: by a wave's own instructions, 0.6 us a token behind 5 us for the launch, the search
// and the state (8 tokens of one request, 48 heads: 9.6 us).  Half the columns a wave there; a quarter, with
// 32 lanes to a column, was slower (12.1 us), and more tokens read ahead (8 instead of 2) gave nothing.
template <class E, int RPL, int RB>  // rows per lane, row blocks: Dk <= RPL RB
__global__ void __launch_bounds__(64) k_delta_step(DeltaArgs a) {
    constexpr int CB = 64 / RB;
    const int r = blockIdx.x, h = a.h0 + blockIdx.y;
    const int lane = threadIdx.x, cb = lane % CB, rb = lane / CB;
    const int col = (blockIdx.z * CB + cb) * 4, row0 = rb * RPL;
    const bool cin = col < a.Dv;
    const int own = col + (lane >> 5) + (lane >> 3 & 2);  // the column whose sums a row of 16 lanes ends up with
    if (r == a.p.R) {  // rows behind the last request
        for (int64_t t = packed_row(a.p, r) + rb; t < a.p.T; t += RB)
            if (cin) *reinterpret_cast<u32x2*>(a.y + t * a.ld_y + int64_t(h) * a.Dv + col) = u32x2{0, 0};
        return;
    }
    const int c0 = packed_row(a.p, r), n = packed_row(a.p, r + 1) - c0;
    if (n > a.few) return;
    bool old;
    const int slot = packed_slot(a.p, r, &old);
    const int64_t base = (int64_t(max(slot, 0)) * a.hv + h) * a.Dk * a.Dv;
    const int hk = h / (a.hv / a.hk);
    f32x4 s[RPL];
    constexpr int CH = RPL / 8, AHEAD = 2;
    struct Token {
        u32x4 k[CH], q[CH];
        uint16_t v;
        float g, beta;
    } ring[AHEAD];
    auto fetch = [&](int t, Token& x) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            x.k[c] = x.q[c] = u32x4{0, 0, 0, 0};
            if (row0 + 8 * c < a.Dk) {
                x.k[c] = *reinterpret_cast<const u32x4*>(a.k + t * a.ld_k + int64_t(hk) * a.Dk + row0 + 8 * c);
                x.q[c] = *reinterpret_cast<const u32x4*>(a.q + t * a.ld_q + int64_t(hk) * a.Dk + row0 + 8 * c);
            }
        }
        x.v = 0;
        if (cin) x.v = a.v[t * a.ld_v + int64_t(h) * a.Dv + own];
        x.g = a.g[t * a.ld_g + h];
        x.beta = a.beta[t * a.ld_b + h];
    };
    // Sums over the row blocks.  Of four columns at once each swap of halves or of rows halves how many a lane has,
    // until it has one: 3 swaps instead of 8.
    struct Two {
        float x, y;
    };
    auto half = [](float x, float y) __attribute__((always_inline)) {  // halves (x, y), in the other (x, y)
        const auto z = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y), false, false);
        const uint32_t z0 = z[0], z1 = z[1];
        return Two{__builtin_bit_cast(float, z0), __builtin_bit_cast(float, z1)};
    };
    auto row = [](float x, float y) __attribute__((always_inline)) {  // rows of 16 lanes x, y, x, y
        const auto z = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y), false, false);
        const uint32_t z0 = z[0], z1 = z[1];
        return Two{__builtin_bit_cast(float, z0), __builtin_bit_cast(float, z1)};
    };
    // one value twice: two values to the compiler, as a swap writes both
    auto twice = [](float x) __attribute__((always_inline)) {
        return __builtin_bit_cast(float, fresh(__builtin_bit_cast(int, x)));
    };
    auto in_row = [&](float v) __attribute__((always_inline)) {
        v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x128, 0xF, 0xF, false));
        if constexpr (RB == 16)
            v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x124, 0xF, 0xF, false));
        return v;
    };
    auto all = [&](float v) __attribute__((always_inline)) {
        const Two p = half(v, twice(v));
        const float w = p.x + p.y;
        const Two q = row(w, twice(w));
        return in_row(q.x + q.y);
    };
    auto each = [&](const f32x4& v) __attribute__((always_inline)) {  // of the lane's own column
        const Two p = half(v[0], v[1]), q = half(v[2], v[3]), r = row(p.x + p.y, q.x + q.y);
        return in_row(r.x + r.y);
    };
    auto token = [&](int t, const Token& x) __attribute__((always_inline)) {
        const float e = exp_f32(bounded(x.g));
        f32x4 sk = {0.f, 0.f, 0.f, 0.f}, sq = sk;
        float kq = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float kk = j & 1 ? hi16<E>(x.k[c][j / 2]) : lo16<E>(x.k[c][j / 2]);
                const float qq = j & 1 ? hi16<E>(x.q[c][j / 2]) : lo16<E>(x.q[c][j / 2]);
                kq = fmaf(kk, qq, kq);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sk[i] = fmaf(kk, s[8 * c + j][i], sk[i]);
                    sq[i] = fmaf(qq, s[8 * c + j][i], sq[i]);
                }
            }
        float one = x.beta * fmaf(-e, each(sk), lo16<E>(x.v));
        one += one - one;  // NaN of what is not finite, as in chunks
        const float y = a.scale * fmaf(all(kq), one, e * each(sq));
        if ((lane & 15) < CB && cin) a.y[int64_t(t) * a.ld_y + int64_t(h) * a.Dv + own] = uint16_t(pack16<E>(y, y));
        // the four columns' u from the four rows
        const Two p = row(one, twice(one)), u01 = half(p.x, twice(p.x)), u23 = half(p.y, twice(p.y));
        const f32x4 u = {u01.x, u01.y, u23.x, u23.y};
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float kk = j & 1 ? hi16<E>(x.k[c][j / 2]) : lo16<E>(x.k[c][j / 2]);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[8 * c + j][i] = fmaf(kk, u[i], s[8 * c + j][i] * e);
            }
    };
    if (n > 0) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) fetch(c0 + min(j, n - 1), ring[j]);
    }
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
        s[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (old && cin && row0 + i < a.Dk)
            s[i] = *reinterpret_cast<const f32x4*>(a.sin + base + int64_t(row0 + i) * a.Dv + col);
    }
    for (int i = 0; i < n; i += AHEAD) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (i + j >= n) break;
            const Token x = ring[j];
            if (i + j + AHEAD < n) fetch(c0 + i + j + AHEAD, ring[j]);
            token(c0 + i + j, x);
        }
    }
    if (slot >= 0 && cin) {
#pragma unroll
        for (int i = 0; i < RPL; ++i)
            if (row0 + i < a.Dk)
                *reinterpret_cast<f32x4*>(a.sout + base + int64_t(row0 + i) * a.Dv + col) = s[i];
    }
}

// ---------------------------------------------------------------- host half

struct DeltaGeom {
    bool step, split;
    int few;                   // with chunks: requests of up to so many tokens through the recurrence first
    int L;                     // tokens of a segment
    size_t images, seg, bytes;  // where they start; in all
    int64_t seg_units;
};

// room: bytes of the caller's workspace, SIZE_MAX when the call's own wish is asked for.  A workspace that was made for
// more tokens, requests and max_q holds the chunks of this call, but maybe not the segments that only this one would
// take: then longer ones that fit, or whole requests.
DeltaGeom delta_geom(const vqmlp_delta_desc& d, int cus, size_t room) {
    DeltaGeom G{};
    // A token of the recurrence takes 0.6 us, or more where its waves fill the card; a chunk takes the same for one token
    // as for 64.  They meet, for heads of 128 x 128, at 24 tokens for one request of 48 heads (19 us), 29 for eight (50 us)
    // and 48 for 64 (370 us), of 8 heads at 25, 25 and 31; for heads of 64 x 64 at 20 (15 us), 40 (30 us) and
    // over 48, of 8 heads at 18, 19 and 34: the bounds are those of 128 x 128, and smaller heads of many requests take up
    // to 1.4 times as long between them and where they meet (64 requests of 41 tokens: 155 us in chunks, 111 by the recurrence).
    // Requests of different lengths that fill the card with a chunk each (64 requests of 48
    // heads, 63 of them with one token, one with 512: 377 us in chunks, 142 so) go each its own way.
    const int64_t heads = int64_t(d.R) * d.v_heads;
    constexpr int most_few = 40;
    const int few = heads >= 8 * cus ? most_few : heads >= cus ? 28 : 20;
    const size_t units = size_t(d.T) / kDeltaC + d.R + 1;
    const size_t images = units * d.v_heads * kDeltaBlock;
    const size_t chunks_bytes = images + units * d.k_heads * ((d.dtype == VQMLP_BF16 ? 2 : 1) * kDeltaC * (d.Dk <= 64 ? 64 : 128) * 2);
    // more requests may leave max_q to the recurrence, and so their workspace empty, where fewer take chunks
    G.step = d.max_q <= few || (d.max_q <= most_few && room < chunks_bytes);
    if (G.step) return G;
    // not split: a segment holds all T tokens, so any request fits, whatever max_q says
    G.L = std::max(1, (d.T + kDeltaC - 1) / kDeltaC) * kDeltaC;
    // Costs in a chunk's time (some 2 us).  In segments a request's chain is walked twice, a segment's length each time, with
    // a join between (3.3 us a segment) and two more launches.  A compute unit holds two workgroups of 32 columns,
    // which then take a quarter longer; an XCD fills up before all of them do.  8,000 tokens, BF16, whole and in
    // segments: 6 heads of 128 x 128 293 and 124 us, 24 heads 310 and 247, 48 heads 348 whole;
    // of 64 x 64 226 and 85, 245 and 145, 275 and 263.  Near the border the choice may be the slower one: 1,500 tokens
    // of 24 heads of 128 x 128 81 and 90 us, of 48 heads of 64 x 64 70 and 80.
    const int most = std::max(1, std::min(d.max_q, std::max(1, d.T))), chunks = (most + kDeltaC - 1) / kDeltaC;
    const bool even = d.T == int64_t(d.R) * most;  // all requests are as long as the longest
    G.few = heads >= cus && !even ? few : -1;
    const int64_t vs = (d.Dv + 31) / 32, ks = (d.Dk + 31) / 32;
    auto rounds = [&](int64_t wgs) {
        const int64_t n = wgs * d.v_heads * 17 / 16, rest = n % (2 * cus);
        return 1.25 * double(n / (2 * cus)) + (rest == 0 ? 0. : rest <= cus ? 1. : 1.25);
    };
    // whole requests: the longest, or what all give each compute unit to do and a part of the other
    const double share = 0.625 * double(d.T) / kDeltaC * vs * d.v_heads / cus;
    double best = even ? rounds(d.R * vs) * chunks : std::max<double>(chunks, share) + 0.25 * std::min<double>(chunks, share);
    auto seg_bytes = [&](int64_t L) { return (size_t(d.T / L) + d.R + 1) * d.v_heads * d.Dk * (d.Dv + d.Dk) * 4; };
    for (int n = 5; n < chunks && heads < 64 * cus; n += std::max(1, n / 8)) {  // more heads fill the card in any case
        if (chunks_bytes > room || seg_bytes(n * kDeltaC) > room - chunks_bytes) continue;
        const int64_t per = (chunks + n - 1) / n, units = even ? d.R * per : std::max<int64_t>(d.T / (n * kDeltaC) + d.R / 2, d.R);
        const int64_t inner = units > d.R ? units - d.R : 0;  // segments but the last; M of those but the first
        const double cost = (rounds(inner * vs + std::max<int64_t>(0, inner - d.R) * ks) + rounds(units * vs)) * n + 1.8 * per + 1;
        if (cost < best) best = cost, G.split = true, G.L = n * kDeltaC;
    }
    G.images = images;
    G.seg = chunks_bytes;
    G.seg_units = d.T / G.L + d.R + 1;
    G.bytes = chunks_bytes + (G.split ? seg_bytes(G.L) : 0);
    return G;
}

vqmlp_status delta_check(const vqmlp_delta_desc* p, const char* who) {
    OP_REQUIRE(p, "%s: null description", who);
    const vqmlp_delta_desc& d = *p;
    OP_REQUIRE(op_dtype16(d.dtype), "%s: dtype %d is not F16 or BF16", who, d.dtype);
    OP_REQUIRE(d.T >= 0 && d.R >= 1 && d.k_heads >= 1 && d.v_heads >= 1 && d.n_states >= 0 && d.max_q >= 0,
               "%s: a size is out of range", who);
    OP_REQUIRE(d.v_heads % d.k_heads == 0, "%s: v_heads=%d is no multiple of k_heads=%d", who, d.v_heads,
               d.k_heads);
    OP_REQUIRE(d.Dk >= 8 && d.Dk <= 128 && d.Dk % 8 == 0 && d.Dv >= 8 && d.Dv <= 128 && d.Dv % 8 == 0,
               "%s: Dk=%d, Dv=%d are not multiples of 8 up to 128", who, d.Dk, d.Dv);
    if (d.R > 65535 || d.v_heads > 65535 || d.T > 0x3FFFFFFF)
        OP_FAIL(VQMLP_ERR_UNSUPPORTED, "%s: R or v_heads above 65535, or T above 2^30 - 1", who);
    OP_REQUIRE(d.scale - d.scale == 0.f, "%s: scale is not finite", who);
    return VQMLP_OK;
}

template <class E>
void launch_step(DeltaArgs a, int cus, hipStream_t s) {
    const int units = a.p.R + (a.few == INT_MAX);  // and the rows behind the last request, if no chunks follow
    // half the columns and rows a lane where waves of 32 columns are fewer than the chip's SIMDs
    const bool narrow = a.Dk > 64 && int64_t(a.p.R) * a.hv * ((a.Dv + 31) / 32) <= 4 * int64_t(cus);
    const int cols = narrow ? (a.Dv + 15) / 16 : (a.Dv + 31) / 32;
    const int most = int(((int64_t(1) << 25) / units + cols - 1) / cols);  // heads: a launch holds fewer than 2^32 threads
    for (a.h0 = 0; a.h0 < a.hv; a.h0 += most) {
        const dim3 grid(units, std::min(most, a.hv - a.h0), cols);
        if (narrow) k_delta_step<E, 8, 16><<<grid, 64, 0, s>>>(a);
        else if (a.Dk <= 64) k_delta_step<E, 8, 8><<<grid, 64, 0, s>>>(a);
        else k_delta_step<E, 16, 8><<<grid, 64, 0, s>>>(a);
    }
}

template <class E>
void launch_delta(const DeltaArgs& a, bool chunks, int cus, hipStream_t s) {
    if (a.few > 0) launch_step<E>(a, cus, s);
    if (chunks) launch_delta_chunks<E>(a, cus, s);
}

}  // namespace

}  // namespace vqmlp

extern "C" vqmlp_status vqmlp_delta_rule_workspace(const vqmlp_delta_desc* p, size_t* bytes) {
    using namespace vqmlp;
    OP_REQUIRE(bytes, "vqmlp_delta_rule_workspace: null pointer");
    if (const vqmlp_status st = delta_check(p, "vqmlp_delta_rule_workspace")) return st;
    int cus = 0;
    if (const int st = device_cus(&cus)) return static_cast<vqmlp_status>(st);
    *bytes = delta_geom(*p, cus, SIZE_MAX).bytes;
    return op_ok();
}

extern "C" vqmlp_status vqmlp_delta_rule(const vqmlp_delta_desc* p, void* workspace, size_t workspace_bytes,
                                         void* stream) {
    using namespace vqmlp;
    int cus = 0;
    if (const vqmlp_status st = delta_check(p, "vqmlp_delta_rule")) return st;
    const vqmlp_delta_desc& d = *p;
    OP_REQUIRE(d.cu_q && op_aligned(d.cu_q, 4) && op_aligned(d.ctx_len, 4) && op_aligned(d.state_index, 4),
               "vqmlp_delta_rule: null cu_q or an unaligned index array");
    OP_REQUIRE((d.state_in && d.state_out) || d.n_states == 0, "vqmlp_delta_rule: null state");
    OP_REQUIRE(op_aligned(d.state_in, 16) && op_aligned(d.state_out, 16),
               "vqmlp_delta_rule: states have to be 16-byte aligned");
    if (d.T > 0) {
        OP_REQUIRE(d.q && d.k && d.v && d.g && d.beta && d.y, "vqmlp_delta_rule: null pointer");
        OP_REQUIRE(op_aligned(d.q, 16) && op_aligned(d.k, 16) && op_aligned(d.v, 16) && op_aligned(d.y, 16) &&
                       op_aligned(d.g, 4) && op_aligned(d.beta, 4),
                   "vqmlp_delta_rule: q, k, v and y have to be 16-byte aligned, g and beta 4-byte");
        const int64_t rows[] = {int64_t(d.k_heads) * d.Dk, int64_t(d.k_heads) * d.Dk, int64_t(d.v_heads) * d.Dv,
                                int64_t(d.v_heads) * d.Dv, d.v_heads, d.v_heads};
        const int64_t lds[] = {d.ld_q, d.ld_k, d.ld_v, d.ld_y, d.ld_g, d.ld_beta};
        for (int i = 0; i < 6; ++i)
            OP_REQUIRE((d.T == 1 || lds[i] >= rows[i]) && lds[i] >= 0 && lds[i] <= kMaxLd && (i >= 4 || lds[i] % 8 == 0),
                       "vqmlp_delta_rule: token strides have to cover the heads and be at most 2^24, those of q, k, "
                       "v and y be multiples of 8");
    }
    if (const int st = device_cus(&cus)) return static_cast<vqmlp_status>(st);
    const DeltaGeom G = delta_geom(d, cus, workspace ? workspace_bytes : 0);
    if (G.bytes) {
        OP_REQUIRE(workspace && op_aligned(workspace, 256), "vqmlp_delta_rule: the workspace is null or not 256-byte aligned");
        if (workspace_bytes < G.bytes)
            OP_FAIL(VQMLP_ERR_WORKSPACE, "vqmlp_delta_rule: workspace holds %zu bytes, this call needs %zu", workspace_bytes,
                    G.bytes);
    }
    DeltaArgs a{};
    a.q = static_cast<const uint16_t*>(d.q);
    a.k = static_cast<const uint16_t*>(d.k);
    a.v = static_cast<const uint16_t*>(d.v);
    a.g = d.g;
    a.beta = d.beta;
    a.y = static_cast<uint16_t*>(d.y);
    a.sin = d.state_in;
    a.sout = d.state_out;
    a.p = Packed{d.cu_q, d.ctx_len, d.state_index, d.T, d.R, d.n_states};
    a.ld_q = d.ld_q, a.ld_k = d.ld_k, a.ld_v = d.ld_v, a.ld_y = d.ld_y, a.ld_g = d.ld_g, a.ld_b = d.ld_beta;
    a.hk = d.k_heads, a.hv = d.v_heads, a.Dk = d.Dk, a.Dv = d.Dv;
    a.scale = d.scale;
    a.blocks = static_cast<uint8_t*>(workspace);
    a.images = reinterpret_cast<uint16_t*>(a.blocks + G.images);
    a.seg = G.split ? reinterpret_cast<float*>(a.blocks + G.seg) : nullptr;
    a.seg_units = G.seg_units;
    a.L = G.L;
    a.few = G.step ? INT_MAX : G.few;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (d.dtype == VQMLP_F16) launch_delta<F16>(a, !G.step, cus, s);
    else launch_delta<BF16>(a, !G.step, cus, s);
    if (trace_enabled())
        trace_line("delta_rule T=%d R=%d heads=%d/%d: %s%s of %d tokens", d.T, d.R, d.v_heads, d.k_heads,
                   G.few > 0 ? "recurrence of short requests, " : "",
                   G.step ? "recurrence" : G.split ? "segment states, join, then segments" : "chunks, segments", G.step ? 1 : G.L);
    return op_launched("vqmlp_delta_rule");
}
