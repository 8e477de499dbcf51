// rotary.hip -- norm and rotation of queries and keys, append of keys and values to the paged cache.
//
// Roles of the workgroups of one launch: heads of q, heads of k (rows: norm, turn, write), heads of v
// (64 tokens turned through LDS, since values lie transposed in their pages).
#include "op.h"

#include <algorithm>

namespace vqmlp {

namespace {

constexpr int kVTok = 64, kVD = 64;
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
    float eps, off;
};

// A lane's eight elements of a head are two runs of four: of a half-split rotation four pairs' first
// and second elements, otherwise eight neighbours.
template <class E>
__device__ __forceinline__ void rows_role(const AppendArgs& a, int64_t id) {
    const int group = int(id % a.groups);
    const int64_t t0 = id / a.groups * a.rows;
    const bool isk = group >= a.qgroups;
    const int h0 = (isk ? group - a.qgroups : group) * a.per;
    const int h1 = min(h0 + a.per, isk ? a.kv_heads : a.heads);
    const int item = threadIdx.x % a.lanes, half = a.rot / 2;
    const bool in = 8 * item < a.D, turn = 8 * item < a.rot;
    const int e0 = turn && !a.next ? 4 * item : 8 * item, e1 = turn && !a.next ? half + 4 * item : 8 * item + 4;
    const uint16_t* const w = isk ? a.kw : a.qw;
    float wt[8];
    auto read = [&](const uint16_t* p, float* f) __attribute__((always_inline)) {
        const u32x2 x = *reinterpret_cast<const u32x2*>(p + e0), y = *reinterpret_cast<const u32x2*>(p + e1);
        f[0] = lo16<E>(x[0]), f[1] = hi16<E>(x[0]), f[2] = lo16<E>(x[1]), f[3] = hi16<E>(x[1]);
        f[4] = lo16<E>(y[0]), f[5] = hi16<E>(y[0]), f[6] = lo16<E>(y[1]), f[7] = hi16<E>(y[1]);
    };
    if (w && in) {
        read(w, wt);
#pragma unroll
        for (int i = 0; i < 8; ++i) wt[i] += a.off;
    }
    float freq[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) freq[i] = turn ? a.freq[4 * item + i] : 0.f;
    const int step = 256 / a.lanes;
    for (int i = threadIdx.x / a.lanes; i < a.rows; i += step) {
        const int64_t t = t0 + i;
        if (t >= a.T) break;  // a head's lanes leave together
        const int pos = a.pos[t];
        if (pos < 0) continue;
        int64_t s = 0;
        if (isk) {
            s = a.slot[t];
            if (s < 0 || s >= a.slots) continue;
        }
        const int64_t page = s >> a.shift, at = s & ((1 << a.shift) - 1);
        float c[4], sn[4];
        if (turn) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const double f = double(pos) * (double(freq[j]) * kTurns);
                sincospif(float(2. * (f - rint(f))), &sn[j], &c[j]);
            }
        }
        for (int h = h0; h < h1; ++h) {
            const uint16_t* const src = isk ? a.k + t * a.ld_k + h * a.hs_k : a.q + t * a.ld_q + h * a.hs_q;
            uint16_t* const dst = isk ? a.kc + (((page * a.kv_heads + h) << a.shift) + at) * a.D
                                      : a.q_out + t * a.ld_qo + int64_t(h) * a.D;
            float f[8] = {};
            if (in) read(src, f);
            if (w) {
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
                for (int o = 1; o < a.lanes; o <<= 1) sum += __shfl_xor(sum, o);
                const float by = 1.f / sqrtf(sum / float(a.D) + a.eps);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = f[j] * by * wt[j];
            }
            if (turn) {
                float z[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x = a.next ? f[2 * j] : f[j], y = a.next ? f[2 * j + 1] : f[j + 4];
                    z[j] = x * c[j] - y * sn[j];
                    z[j + 4] = y * c[j] + x * sn[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = a.next ? z[j / 2 + (j & 1) * 4] : z[j];
            }
            if (in) {
                *reinterpret_cast<u32x2*>(dst + e0) = u32x2{pack16<E>(f[0], f[1]), pack16<E>(f[2], f[3])};
                *reinterpret_cast<u32x2*>(dst + e1) = u32x2{pack16<E>(f[4], f[5]), pack16<E>(f[6], f[7])};
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
    for (int i = threadIdx.x; i < kVTok * (kVD / 8); i += 256) {
        const int tok = i / (kVD / 8), c = i % (kVD / 8) * 8;
        if (t0 + tok >= a.T || c >= nd) continue;
        const u32x4 x = *reinterpret_cast<const u32x4*>(a.v + (t0 + tok) * a.ld_v + h * a.hs_v + d0 + c);
        uint32_t* const w = reinterpret_cast<uint32_t*>(&tile[tok][c]);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = x[j];
    }
    __syncthreads();
    const int tok = threadIdx.x & 63;
    if (t0 + tok >= a.T || a.pos[t0 + tok] < 0) return;
    const int64_t s = a.slot[t0 + tok];
    if (s < 0 || s >= a.slots) return;
    const int64_t page = s >> a.shift, off = s & (P - 1);
    uint16_t* const dst = a.vc + ((page * a.kv_heads + h) * a.D + d0) * P + off;
    for (int c = threadIdx.x >> 6; c < nd; c += 4) dst[int64_t(c) * P] = tile[tok][c];
}

template <class E>
__global__ void __launch_bounds__(256) k_paged_append(AppendArgs a) {
    __shared__ uint16_t tile[kVTok][kVD + 2];  // a row stride of 33 words
    const int64_t id = a.id0 + blockIdx.x;
    if (id < a.row_blocks) rows_role<E>(a, id);
    else values_role(a, id - a.row_blocks, tile);
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
    a.eps = d.eps, a.off = d.w_offset;
    a.lanes = 1;
    while (a.lanes * 8 < d.D) a.lanes *= 2;
    a.rows = 256 / a.lanes;
    a.per = 1;
    a.qgroups = (d.heads + a.per - 1) / a.per;
    a.groups = a.qgroups + (d.kv_heads + a.per - 1) / a.per;
    a.row_blocks = int64_t((d.T + a.rows - 1) / a.rows) * a.groups;
    const int64_t values = int64_t((d.T + kVTok - 1) / kVTok) * d.kv_heads * ((d.D + kVD - 1) / kVD);
    const int64_t all = a.row_blocks + values, most = 8 << 20;  // a launch holds fewer than 2^32 threads
    const hipStream_t s = static_cast<hipStream_t>(stream);
    for (a.id0 = 0; a.id0 < all; a.id0 += most) {
        const unsigned grid = unsigned(std::min(most, all - a.id0));
        if (d.dtype == VQMLP_F16) k_paged_append<F16><<<grid, 256, 0, s>>>(a);
        else k_paged_append<BF16><<<grid, 256, 0, s>>>(a);
    }
    if (trace_enabled())
        trace_line("paged_append T=%d heads=%d/%d D=%d rot=%d: %lld row workgroups of %d tokens x %d heads, %lld of values", d.T,
                   d.heads, d.kv_heads, d.D, d.rot, (long long)a.row_blocks, a.rows, a.per, (long long)values);
    return op_launched("vqmlp_paged_append");
}
