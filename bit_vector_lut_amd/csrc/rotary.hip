// rotary.hip -- norm and rotation of queries and keys, append of keys and values to the paged cache.
//
//   x' = x / sqrt(mean(x^2) + eps) (offset + w)          each head of q and k, where there are weights
//   (a, b)' = (a cos f - b sin f, b cos f + a sin f)      f = position inv_freq[pair], pairs (a, b) of a head
//
// Roles of the workgroups of one launch: heads of q, heads of k (rows: norm, turn, write), heads of v
// (64 tokens turned through LDS, since values lie transposed in their pages). The angle is a product of
// FP64, brought to one turn before it is rounded: at position 10^6 an FP32 product would be off by 0.06.
// Norm, turn and sums are FP32 and rounded once.
//
// Bound by memory for prompts: 8,192 tokens, 24 + 4 heads of 256 with 64 turned, in 45 us, 268 MB at
// 5.9 TB/s (part of the writes still on the way to memory). One angle a thread, kept in LDS for the heads of
// a workgroup, instead of each lane's own for each head, and four heads on their way at a time: 102 -> 46 us.
// Few tokens: latency. 8 tokens in 3.6 us, 64 requests' single tokens in 5.4 us, 512 tokens of 40 + 8 heads
// of 128 in 6.2 us, where the sines bound.
#include "op.h"

#include <algorithm>

namespace vqmlp {

namespace {

constexpr int kVTok = 64, kVD = 64;  // of a tile of values: two loads a thread
constexpr int kHeads = 4;  // heads on their way at a time
constexpr double kTurns = 0.15915494309189533577;  // 1 / (2 pi)

struct AppendArgs {
    const uint16_t *q, *k, *v;
    uint16_t *q_out, *kc, *vc;
    const uint16_t *qw, *kw;
    const float* freq;
    const int32_t *pos, *slot;
    int64_t ld_q, hs_q, ld_k, hs_k, ld_v, hs_v, ld_qo;
    int64_t slots, id0, row_blocks;
    int T, heads, kv_heads, D, rot, next, shift;
    int lanes;     // of a head: a power of two, 8 elements each
    int rows;      // tokens of a row block
    int per;       // heads of a row block
    int qgroups, groups;
    float eps, off, inv_d;
};

// HB heads at a time of one token for each group of lanes. A lane's eight elements of a head are two runs
// of four: of a half-split rotation four pairs' first and second elements, otherwise eight neighbours.
// The angles' sines and cosines are found once for all heads of the workgroup, one angle a thread at a
// time, while the first heads are on their way.
template <class E, int HB>
__device__ __forceinline__ void rows_role(const AppendArgs& a, int64_t id, float2* trig) {
    const int group = int(id % a.groups);
    const int64_t t0 = id / a.groups * a.rows;
    const bool isk = group >= a.qgroups;
    const int h0 = (isk ? group - a.qgroups : group) * a.per;
    const int h1 = min(h0 + a.per, isk ? a.kv_heads : a.heads);
    const int item = threadIdx.x & (a.lanes - 1), i = threadIdx.x / a.lanes, half = a.rot / 2;
    const bool in = 8 * item < a.D, turn = 8 * item < a.rot;
    // lanes behind the head's end and tokens behind the last read what is there and write nothing
    const int first = in ? item : 0;
    const int e0 = turn && !a.next ? 4 * first : 8 * first, e1 = turn && !a.next ? half + 4 * first : 8 * first + 4;
    const int64_t t = min(t0 + i, int64_t(a.T) - 1);
    const uint16_t* const w = isk ? a.kw : a.qw;
    const int64_t hs = isk ? a.hs_k : a.hs_q;
    const uint16_t* const src = isk ? a.k + t * a.ld_k : a.q + t * a.ld_q;
    struct Raw {
        u32x2 lo, hi;
    };
    auto read = [&](const uint16_t* p) __attribute__((always_inline)) {
        return Raw{*reinterpret_cast<const u32x2*>(p + e0), *reinterpret_cast<const u32x2*>(p + e1)};
    };
    auto unpack = [&](const Raw& r, float* f) __attribute__((always_inline)) {
        f[0] = lo16<E>(r.lo[0]), f[1] = hi16<E>(r.lo[0]), f[2] = lo16<E>(r.lo[1]), f[3] = hi16<E>(r.lo[1]);
        f[4] = lo16<E>(r.hi[0]), f[5] = hi16<E>(r.hi[0]), f[6] = lo16<E>(r.hi[1]), f[7] = hi16<E>(r.hi[1]);
    };
    const int pos = a.pos[t];
    const int64_t s = isk ? a.slot[t] : 0;
    Raw raw[HB], weights{};
#pragma unroll
    for (int b = 0; b < HB; ++b) raw[b] = read(src + min(h0 + b, h1 - 1) * hs);
    if (w) weights = read(w);
    const int pairs = half * a.rows;
    for (int n = threadIdx.x; n < pairs; n += 256) {
        const int64_t tt = min(t0 + n / half, int64_t(a.T) - 1);
        const double f = double(a.pos[tt]) * (double(a.freq[n % half]) * kTurns);
        float2 v;
        sincospif(float(2. * (f - rint(f))), &v.y, &v.x);
        trig[n] = v;
    }
    __syncthreads();
    float wt[8], c[4], sn[4];
    unpack(weights, wt);
#pragma unroll
    for (int j = 0; j < 8; ++j) wt[j] += a.off;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 v = turn ? trig[i * half + 4 * item + j] : float2{1.f, 0.f};
        c[j] = v.x, sn[j] = v.y;
    }
    const bool write = in && t0 + i < a.T && pos >= 0 && s >= 0 && s < a.slots;
    const int64_t page = s >> a.shift, at = s & ((1 << a.shift) - 1);
    uint16_t* const dst = isk ? a.kc + ((page * a.kv_heads << a.shift) + at) * a.D : a.q_out + t * a.ld_qo;
    const int64_t step = isk ? int64_t(a.D) << a.shift : a.D;
    for (int h = h0; h < h1; h += HB) {
        float f[HB][8];
#pragma unroll
        for (int b = 0; b < HB; ++b) {
            unpack(raw[b], f[b]);
            raw[b] = read(src + min(h + HB + b, h1 - 1) * hs);
        }
        if (w) {
            float sum[HB];
#pragma unroll
            for (int b = 0; b < HB; ++b) {
                sum[b] = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[b] = fmaf(f[b][j], f[b][j], sum[b]);
                if (!in) sum[b] = 0.f;
            }
            head_sums(sum, a.lanes);
#pragma unroll
            for (int b = 0; b < HB; ++b) {
                const float by = __builtin_amdgcn_rsqf(fmaf(sum[b], a.inv_d, a.eps));
#pragma unroll
                for (int j = 0; j < 8; ++j) f[b][j] *= by * wt[j];
            }
        }
#pragma unroll
        for (int b = 0; b < HB; ++b) {
            float z[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = a.next ? f[b][2 * j] : f[b][j], y = a.next ? f[b][2 * j + 1] : f[b][j + 4];
                z[j] = x * c[j] - y * sn[j];
                z[j + 4] = y * c[j] + x * sn[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = turn ? z[j] : f[b][j];
            const bool next = a.next && turn;
            if (write && h + b < h1) {
                uint16_t* const p = dst + (h + b) * step;
                *reinterpret_cast<u32x2*>(p + e0) = next ? u32x2{pack16<E>(z[0], z[4]), pack16<E>(z[1], z[5])}
                                                         : u32x2{pack16<E>(z[0], z[1]), pack16<E>(z[2], z[3])};
                *reinterpret_cast<u32x2*>(p + e1) = next ? u32x2{pack16<E>(z[2], z[6]), pack16<E>(z[3], z[7])}
                                                         : u32x2{pack16<E>(z[4], z[5]), pack16<E>(z[6], z[7])};
            }
        }
    }
}

// 64 tokens of one head and up to 64 of its elements: read by rows, written by columns, where
// neighbouring tokens of a prompt are neighbours.
__device__ __forceinline__ void values_role(const AppendArgs& a, int64_t id, uint16_t (*tile)[kVD + 2]) {
    const int parts = (a.D + kVD - 1) / kVD;
    const int d0 = int(id % parts) * kVD, h = int(id / parts % a.kv_heads);
    const int64_t t0 = id / parts / a.kv_heads * kVTok;
    const int P = 1 << a.shift, nd = min(kVD, a.D - d0);
    const int tok = threadIdx.x & 63;
    const int64_t t = min(t0 + tok, int64_t(a.T) - 1);
    const int pos = a.pos[t];
    const int64_t s = a.slot[t];
    u32x4 x[2] = {};
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int i = threadIdx.x + 256 * n;
        const int r = i / (kVD / 8), c = i % (kVD / 8) * 8;
        if (t0 + r < a.T && c < nd) x[n] = *reinterpret_cast<const u32x4*>(a.v + (t0 + r) * a.ld_v + h * a.hs_v + d0 + c);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int i = threadIdx.x + 256 * n;
        uint32_t* const w = reinterpret_cast<uint32_t*>(&tile[i / (kVD / 8)][i % (kVD / 8) * 8]);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = x[n][j];
    }
    __syncthreads();
    if (t0 + tok >= a.T || pos < 0 || s < 0 || s >= a.slots) return;
    const int64_t page = s >> a.shift, off = s & (P - 1);
    uint16_t* const dst = a.vc + ((page * a.kv_heads + h) * a.D + d0) * P + off;
    for (int c = threadIdx.x >> 6; c < nd; c += 4) dst[int64_t(c) * P] = tile[tok][c];
}

template <class E, int HB>
__global__ void __launch_bounds__(256) k_paged_append(AppendArgs a) {
    __shared__ union {
        uint16_t tile[kVTok][kVD + 2];  // a row stride of 33 words
        float2 trig[1024];              // 256 / lanes tokens of up to 4 * lanes pairs
    } lds;
    const int64_t id = a.id0 + blockIdx.x;
    if (id < a.row_blocks) rows_role<E, HB>(a, id, lds.trig);
    else values_role(a, id - a.row_blocks, lds.tile);
}

template <class E>
void launch_append(AppendArgs a, int64_t all, hipStream_t s) {
    constexpr int64_t most = 8 << 20;  // a launch holds fewer than 2^32 threads
    for (a.id0 = 0; a.id0 < all; a.id0 += most) {
        const unsigned grid = unsigned(std::min(most, all - a.id0));
        if (a.per == 1) k_paged_append<E, 1><<<grid, 256, 0, s>>>(a);
        else k_paged_append<E, kHeads><<<grid, 256, 0, s>>>(a);
    }
}

}  // namespace

}  // namespace vqmlp

extern "C" vqmlp_status vqmlp_paged_append(const vqmlp_append_desc* p, void* stream) {
    using namespace vqmlp;
    OP_REQUIRE(p, "vqmlp_paged_append: null description");
    const vqmlp_append_desc& d = *p;
    AppendArgs a{};
    OP_REQUIRE(op_dtype16(d.dtype), "vqmlp_paged_append: dtype %d is not F16 or BF16", d.dtype);
    for (a.shift = 3; a.shift <= 10 && d.page_size != 1 << a.shift; ++a.shift) {}
    OP_REQUIRE(a.shift <= 10, "vqmlp_paged_append: page_size %d is not a power of two in 8..1024", d.page_size);
    OP_REQUIRE(d.T >= 0 && d.heads >= 0 && d.heads <= 65535 && d.kv_heads >= 1 && d.kv_heads <= 65535 && d.D >= 8 &&
                   d.D <= 256 && d.D % 8 == 0 && d.n_pages >= 1,
               "vqmlp_paged_append: T=%d, heads=%d, kv_heads=%d, D=%d, n_pages=%d", d.T, d.heads, d.kv_heads, d.D, d.n_pages);
    OP_REQUIRE(d.rot >= 0 && d.rot <= d.D && d.rot % 8 == 0, "vqmlp_paged_append: rot=%d is not a multiple of 8 up to D", d.rot);
    OP_REQUIRE(d.pairs == VQMLP_PAIRS_HALF || d.pairs == VQMLP_PAIRS_NEXT, "vqmlp_paged_append: pairs %d", d.pairs);
    OP_REQUIRE((int64_t(d.n_pages) << a.shift) <= 0x7FFFFFFF, "vqmlp_paged_append: slots pass 2^31 - 1");
    if (d.T > 0x3FFFFFFF) OP_FAIL(VQMLP_ERR_UNSUPPORTED, "vqmlp_paged_append: T above 2^30 - 1");
    OP_REQUIRE((!d.q_w && !d.k_w) || (d.eps >= 0.f && d.eps - d.eps == 0.f && d.w_offset - d.w_offset == 0.f),
               "vqmlp_paged_append: eps is negative, or eps or w_offset not finite");
    if (d.T == 0) return op_ok();
    OP_REQUIRE(d.k && d.v && d.position && d.slot && d.k_cache && d.v_cache && (d.heads == 0 || (d.q && d.q_out)) &&
                   (d.rot == 0 || d.inv_freq),
               "vqmlp_paged_append: null pointer");
    for (const int64_t ld : {d.heads ? d.ld_q : 0, d.ld_k, d.ld_v})
        OP_REQUIRE(ld >= 0 && ld <= int64_t(1) << 40 && ld % 8 == 0,
                   "vqmlp_paged_append: token strides have to be multiples of 8 up to 2^40");
    for (const int64_t hs : {d.heads ? d.hs_q : 0, d.hs_k, d.hs_v})
        OP_REQUIRE(hs >= 0 && hs <= 1 << 24 && hs % 8 == 0,
                   "vqmlp_paged_append: head strides have to be multiples of 8 up to 2^24");
    if (d.heads)
        OP_REQUIRE((d.T == 1 || d.ld_q_out >= int64_t(d.heads) * d.D) && d.ld_q_out >= 0 &&
                       d.ld_q_out <= int64_t(1) << 40 && d.ld_q_out % 8 == 0,
                   "vqmlp_paged_append: the token stride of q_out has to be a multiple of 8 from heads * D up to 2^40");
    OP_REQUIRE(d.heads == 0 || d.q_out != d.q ||
                   ((d.T == 1 || d.ld_q == d.ld_q_out) && (d.heads == 1 || d.hs_q == d.D)),
               "vqmlp_paged_append: q_out is q with other strides");
    for (const void* x : {d.heads ? d.q : nullptr, d.k, d.v, d.heads ? (const void*)d.q_out : nullptr, (const void*)d.k_cache,
                          (const void*)d.v_cache, d.q_w, d.k_w})
        OP_REQUIRE(op_aligned(x, 16), "vqmlp_paged_append: q, k, v, q_out, weights and caches have to be 16-byte aligned");
    OP_REQUIRE(op_aligned(d.position, 4) && op_aligned(d.slot, 4) && op_aligned(d.inv_freq, 4),
               "vqmlp_paged_append: position, slot and inv_freq have to be 4-byte aligned");
    int cus = 0;
    if (const int st = device_cus(&cus)) return static_cast<vqmlp_status>(st);
    a.q = static_cast<const uint16_t*>(d.q);
    a.k = static_cast<const uint16_t*>(d.k);
    a.v = static_cast<const uint16_t*>(d.v);
    a.q_out = static_cast<uint16_t*>(d.q_out);
    a.kc = static_cast<uint16_t*>(d.k_cache);
    a.vc = static_cast<uint16_t*>(d.v_cache);
    a.qw = static_cast<const uint16_t*>(d.q_w);
    a.kw = static_cast<const uint16_t*>(d.k_w);
    a.freq = d.inv_freq;
    a.pos = d.position;
    a.slot = d.slot;
    a.ld_q = d.ld_q, a.hs_q = d.hs_q, a.ld_k = d.ld_k, a.hs_k = d.hs_k, a.ld_v = d.ld_v, a.hs_v = d.hs_v;
    a.ld_qo = d.ld_q_out;
    a.slots = int64_t(d.n_pages) << a.shift;
    a.T = d.T, a.heads = d.heads, a.kv_heads = d.kv_heads, a.D = d.D, a.rot = d.rot;
    a.next = d.pairs == VQMLP_PAIRS_NEXT;
    a.eps = d.eps, a.off = d.w_offset, a.inv_d = 1.f / float(d.D);
    a.lanes = 1;
    while (a.lanes * 8 < d.D) a.lanes *= 2;
    a.rows = 256 / a.lanes;
    const int64_t heads_each = (d.T + a.rows - 1) / a.rows * int64_t(d.heads + d.kv_heads);
    // Heads that share a workgroup's sines: many once there are workgroups enough (512 tokens, 48 heads of 128:
    // 8.7 us with one, 6.2 with four), one where the card would stand empty (64 tokens: 5.4 us).
    a.per = heads_each < 2 * cus ? 1 : heads_each < 16 * cus ? kHeads : 2 * kHeads;
    a.qgroups = (d.heads + a.per - 1) / a.per;
    a.groups = a.qgroups + (d.kv_heads + a.per - 1) / a.per;
    a.row_blocks = int64_t((d.T + a.rows - 1) / a.rows) * a.groups;
    const int64_t values = int64_t((d.T + kVTok - 1) / kVTok) * d.kv_heads * ((d.D + kVD - 1) / kVD);
    const int64_t all = a.row_blocks + values;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (d.dtype == VQMLP_F16) launch_append<F16>(a, all, s);
    else launch_append<BF16>(a, all, s);
    if (trace_enabled())
        trace_line("paged_append T=%d heads=%d/%d D=%d rot=%d: %lld row workgroups of %d tokens x %d heads, %lld of values", d.T,
                   d.heads, d.kv_heads, d.D, d.rot, (long long)a.row_blocks, a.rows, a.per, (long long)values);
    return op_launched("vqmlp_paged_append");
}
