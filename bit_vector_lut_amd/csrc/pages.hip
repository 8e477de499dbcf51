// pages.hip -- block tables and slot maps from request lengths, and the store of new keys and
// values into the paged cache.
#include "op.h"

#include <algorithm>

namespace vqmlp {

namespace {

// ---------------------------------------------------------------- plan of one step
// With n_r = ceil(seq_r / P) - ceil(ctx_r / P) new pages, request r takes the free pages
// head + sum_{i<r} n_i .. and owns the token rows sum_{i<r} q_i ...  Every workgroup makes both
// prefix sums for itself in LDS (R <= 4096: at most four requests a thread; the lengths come from
// L2), so one launch does what would otherwise be a scan and a fill; then each takes its share of
// the token rows and of the requests' table rows.  A token in a new page takes the page number
// from the free list, not from the table that another workgroup is writing.  Bound by the launch and
// two rounds of memory latency: 3.8 us for 4 requests, 7.0 for 512 with 131,000 token rows.
constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxR = 4096;
constexpr int kPlanPer = kPlanMaxR / kPlanThreads;

// Inclusive prefix sum over the workgroup's threads of a pair of values.
__device__ __forceinline__ void scan2(uint32_t& a, uint32_t& b, uint32_t (*part)[2]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t x = __shfl_up(a, o), y = __shfl_up(b, o);
        if (lane >= o) a += x, b += y;
    }
    if (lane == 63) part[wave][0] = a, part[wave][1] = b;
    __syncthreads();
    uint32_t x = 0, y = 0;
    for (int w = 0; w < wave; ++w) x += part[w][0], y += part[w][1];
    a += x;
    b += y;
}

__global__ void __launch_bounds__(kPlanThreads) k_page_plan(vqmlp_pages_desc d, int shift, int rows) {
    __shared__ uint32_t cu[kPlanMaxR + 1];     // first token row of a request
    __shared__ uint32_t taken[kPlanMaxR];      // new pages of the requests before it
    __shared__ uint32_t part[kPlanThreads / 64][2];
    __shared__ unsigned long long total[2];
    __shared__ uint32_t bad;
    const int tid = threadIdx.x, R = d.R;
    const int64_t cap = int64_t(d.table_width) << shift;
    const int64_t page_up = (int64_t(1) << shift) - 1;
    if (tid == 0) bad = 0, total[0] = total[1] = 0;
    __syncthreads();
    // thread i owns requests per*i .. per*i + per - 1
    const int per = (R + kPlanThreads - 1) / kPlanThreads;
    uint32_t q[kPlanPer], n[kPlanPer], sq = 0, sn = 0;
    unsigned long long lq = 0, ln = 0;
    bool wrong = false;
    for (int j = 0; j < kPlanPer; ++j) {
        const int r = tid * per + j;
        q[j] = n[j] = 0;
        if (j >= per || r >= R) continue;
        const int64_t c = d.ctx_len[r], m = d.q_len[r];
        if (c < 0 || m < 0 || c + m > cap) {
            wrong = true;
        } else {
            q[j] = uint32_t(m);
            n[j] = uint32_t(((c + m + page_up) >> shift) - ((c + page_up) >> shift));
        }
        lq += m > 0 ? m : 0;
        ln += n[j];
        sq += q[j];
        sn += n[j];
    }
    if (wrong) atomicOr(&bad, 1u);
    if (lq) atomicAdd(&total[0], lq);  // integers: the order does not matter
    if (ln) atomicAdd(&total[1], ln);
    uint32_t eq = sq, en = sn;
    scan2(eq, en, part);  // its barrier also orders the totals
    eq -= sq;
    en -= sn;
    for (int j = 0; j < kPlanPer; ++j) {
        const int r = tid * per + j;
        if (j >= per || r >= R) continue;
        cu[r] = eq;
        taken[r] = en;
        eq += q[j];
        en += n[j];
        if (r == R - 1) cu[R] = eq;
    }
    __syncthreads();
    const unsigned long long tokens = total[0], pages = total[1];
    const int64_t head = d.free_head ? *d.free_head : 0;
    uint32_t err = bad;
    if (head < 0 || head > d.n_free || pages > (unsigned long long)(d.n_free - head)) err |= 2;
    if (tokens > (unsigned long long)d.max_tokens) err |= 4;
    if (blockIdx.x == 0) {
        const unsigned long long top = 0x7FFFFFFFull;
        if (tid == 0) {
            d.status[0] = int32_t(err);
            d.status[1] = int32_t(tokens < top ? tokens : top);
            d.status[2] = int32_t(pages < top ? pages : top);
            d.status[3] = 0;
            d.cu_q[R] = err ? 0 : int32_t(cu[R]);
            if (d.free_head_out) *d.free_head_out = int32_t(err ? head : head + int64_t(pages));
        }
        for (int r = tid; r < R; r += kPlanThreads) {
            d.cu_q[r] = err ? 0 : int32_t(cu[r]);
            d.seq_len[r] = err ? d.ctx_len[r] : d.ctx_len[r] + d.q_len[r];
        }
    }
    // token rows: `rows` per workgroup
    const int t0 = blockIdx.x * rows, t1 = min(t0 + rows, d.max_tokens);
    const int live = err ? 0 : int(cu[R]);
    for (int t = t0 + tid; t < t1; t += kPlanThreads) {
        int slot = -1, pos = -1;
        if (t < live) {
            int lo = 0, hi = R;  // the last r with cu[r] <= t: requests without tokens drop out
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= uint32_t(t)) lo = mid; else hi = mid;
            }
            const int c = d.ctx_len[lo];
            pos = c + (t - int(cu[lo]));
            const int held = int((int64_t(c) + page_up) >> shift), at = pos >> shift;
            const int page = at < held ? d.table[lo * d.ld_table + at]
                                       : d.free_pages[head + taken[lo] + (at - held)];
            if (page >= 0 && page < d.n_pages) slot = (page << shift) | (pos & int(page_up));
        }
        d.slot[t] = slot;
        d.position[t] = pos;
    }
    // table rows: a wave per request
    if (err) return;
    const int waves = gridDim.x * (kPlanThreads / 64);
    for (int r = blockIdx.x * (kPlanThreads / 64) + (tid >> 6); r < R; r += waves) {
        const int64_t c = d.ctx_len[r];
        const int held = int((c + page_up) >> shift);
        const int need = int((c + d.q_len[r] + page_up) >> shift);
        for (int i = tid & 63; i < need - held; i += 64)
            d.table[r * d.ld_table + held + i] = d.free_pages[head + taken[r] + i];
    }
}

// ---------------------------------------------------------------- store
// A workgroup owns 64 tokens of one head and up to 64 of its D columns.  Keys go as 16-byte
// chunks; values turn through LDS so that a wave writes one column of 64 tokens: neighbouring
// tokens of a prompt are neighbouring elements there.  Bound by HBM: 8,192 tokens of 4 x 256 in pages of
// 64 take 16.3 us, 4.1 TB/s; 64 tokens 5.6 us, the launch and a load behind a load.
constexpr int kStoreTok = 64, kStoreD = 64;

__global__ void __launch_bounds__(256) k_paged_store(int T, int heads, int D, int shift, int64_t slots,
                                                     const uint16_t* k, int64_t ld_k,
                                                     const uint16_t* v, int64_t ld_v,
                                                     const int32_t* slot, uint16_t* kc, uint16_t* vc) {
    // row stride of 33 words: column reads of 16-bit elements by 64 tokens touch all banks evenly
    __shared__ uint16_t tile[kStoreTok][kStoreD + 2];
    const int t0 = blockIdx.x * kStoreTok, h = blockIdx.y, d0 = blockIdx.z * kStoreD;
    const int P = 1 << shift;
    const int nd = min(kStoreD, D - d0);
    for (int i = threadIdx.x; i < kStoreTok * (kStoreD / 8); i += 256) {
        const int tok = i / (kStoreD / 8), c = (i % (kStoreD / 8)) * 8;
        if (t0 + tok >= T || c >= nd) continue;
        const u32x4 kv = *reinterpret_cast<const u32x4*>(k + (t0 + tok) * ld_k + int64_t(h) * D + d0 + c);
        const u32x4 vv = *reinterpret_cast<const u32x4*>(v + (t0 + tok) * ld_v + int64_t(h) * D + d0 + c);
        uint32_t* w = reinterpret_cast<uint32_t*>(&tile[tok][c]);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = vv[j];
        const int64_t s = slot[t0 + tok];
        if (s < 0 || s >= slots) continue;
        const int64_t page = s >> shift, off = s & (P - 1);
        *reinterpret_cast<u32x4*>(kc + ((page * heads + h) * P + off) * D + d0 + c) = kv;
    }
    __syncthreads();
    const int tok = threadIdx.x & 63;
    if (t0 + tok >= T) return;
    const int64_t s = slot[t0 + tok];
    if (s < 0 || s >= slots) return;
    const int64_t page = s >> shift, off = s & (P - 1);
    uint16_t* dst = vc + ((page * heads + h) * D + d0) * P + off;
    for (int c = threadIdx.x >> 6; c < nd; c += 4) dst[int64_t(c) * P] = tile[tok][c];
}

bool page_shift(int page_size, int* shift) {
    for (int s = 3; s <= 10; ++s)
        if (page_size == 1 << s) return *shift = s, true;
    return false;
}

}  // namespace

}  // namespace vqmlp

extern "C" vqmlp_status vqmlp_page_plan(const vqmlp_pages_desc* p, void* stream) {
    using namespace vqmlp;
    OP_REQUIRE(p, "vqmlp_page_plan: null description");
    const vqmlp_pages_desc& d = *p;
    int shift = 0;
    OP_REQUIRE(page_shift(d.page_size, &shift), "vqmlp_page_plan: page_size %d is not a power of two in 8..1024",
               d.page_size);
    OP_REQUIRE(d.R >= 1 && d.max_tokens >= 0 && d.n_pages >= 1 && d.n_free >= 0 && d.table_width >= 1,
               "vqmlp_page_plan: a size is out of range");
    if (d.R > kPlanMaxR) OP_FAIL(VQMLP_ERR_UNSUPPORTED, "vqmlp_page_plan: R=%d above %d", d.R, kPlanMaxR);
    if (d.max_tokens > 0x3FFFFFFF) OP_FAIL(VQMLP_ERR_UNSUPPORTED, "vqmlp_page_plan: max_tokens above 2^30 - 1");
    OP_REQUIRE((int64_t(d.n_pages) << shift) <= 0x7FFFFFFF && (int64_t(d.table_width) << shift) <= 0x7FFFFFFF,
               "vqmlp_page_plan: positions or slots pass 2^31 - 1");
    OP_REQUIRE(d.ld_table >= d.table_width, "vqmlp_page_plan: ld_table is below table_width");
    OP_REQUIRE(d.ctx_len && d.q_len && d.table && d.seq_len && d.cu_q && d.status,
               "vqmlp_page_plan: null pointer");
    OP_REQUIRE((d.slot && d.position) || d.max_tokens == 0, "vqmlp_page_plan: null slot or position");
    OP_REQUIRE(d.free_pages || d.n_free == 0, "vqmlp_page_plan: null free list");
    OP_REQUIRE(!d.free_head_out || d.free_head_out != d.free_head,
               "vqmlp_page_plan: free_head_out is free_head");
    OP_REQUIRE(d.seq_len != d.ctx_len && d.seq_len != d.q_len, "vqmlp_page_plan: seq_len is an input array");
    for (const void* q : {(const void*)d.ctx_len, (const void*)d.q_len, (const void*)d.free_pages,
                          (const void*)d.free_head, (const void*)d.table, (const void*)d.seq_len,
                          (const void*)d.cu_q, (const void*)d.slot, (const void*)d.position,
                          (const void*)d.status, (const void*)d.free_head_out})
        OP_REQUIRE(op_aligned(q, 4), "vqmlp_page_plan: a pointer is not 4-byte aligned");
    int cus = 0;
    if (const int st = device_cus(&cus)) return static_cast<vqmlp_status>(st);
    // a workgroup per 1024 token rows, at most one per compute unit; table rows fill the rest
    const int want = std::max((d.max_tokens + kPlanThreads - 1) / kPlanThreads, (d.R + 63) / 64);
    const int wgs = std::max(1, std::min(cus, want));
    const int rows = (d.max_tokens + wgs - 1) / wgs;
    k_page_plan<<<wgs, kPlanThreads, 0, static_cast<hipStream_t>(stream)>>>(d, shift, rows);
    if (trace_enabled()) trace_line("page_plan R=%d max_tokens=%d: %d workgroups", d.R, d.max_tokens, wgs);
    return op_launched("vqmlp_page_plan");
}

extern "C" vqmlp_status vqmlp_paged_store(int dtype, int T, int kv_heads, int D, int page_size,
                                          int n_pages, const void* k, int64_t ld_k, const void* v,
                                          int64_t ld_v, const int32_t* slot, void* k_cache,
                                          void* v_cache, void* stream) {
    using namespace vqmlp;
    int shift = 0;
    OP_REQUIRE(op_dtype16(dtype), "vqmlp_paged_store: dtype %d is not F16 or BF16", dtype);
    OP_REQUIRE(page_shift(page_size, &shift), "vqmlp_paged_store: page_size %d is not a power of two in 8..1024",
               page_size);
    OP_REQUIRE(T >= 0 && kv_heads >= 1 && kv_heads <= 65535 && D >= 8 && D <= 256 && D % 8 == 0 && n_pages >= 1,
               "vqmlp_paged_store: T=%d, kv_heads=%d, D=%d, n_pages=%d", T, kv_heads, D, n_pages);
    OP_REQUIRE((int64_t(n_pages) << shift) <= 0x7FFFFFFF, "vqmlp_paged_store: slots pass 2^31 - 1");
    // a launch holds fewer than 2^32 threads
    if (T > 0x3FFFFFFF) OP_FAIL(VQMLP_ERR_UNSUPPORTED, "vqmlp_paged_store: T above 2^30 - 1");
    if (T == 0) return op_ok();
    OP_REQUIRE(k && v && slot && k_cache && v_cache, "vqmlp_paged_store: null pointer");
    const int64_t row = int64_t(kv_heads) * D;
    OP_REQUIRE(T == 1 || (ld_k >= row && ld_v >= row), "vqmlp_paged_store: a token stride is below kv_heads * D");
    OP_REQUIRE(ld_k >= 0 && ld_v >= 0 && ld_k <= (int64_t(1) << 40) && ld_v <= (int64_t(1) << 40) &&
                   ld_k % 8 == 0 && ld_v % 8 == 0,
               "vqmlp_paged_store: token strides have to be multiples of 8");
    OP_REQUIRE(op_aligned(k, 16) && op_aligned(v, 16) && op_aligned(k_cache, 16) && op_aligned(v_cache, 16) &&
                   op_aligned(slot, 4),
               "vqmlp_paged_store: k, v and the caches have to be 16-byte aligned, slot 4-byte");
    int cus = 0;
    if (const int st = device_cus(&cus)) return static_cast<vqmlp_status>(st);
    const dim3 grid((T + kStoreTok - 1) / kStoreTok, kv_heads, (D + kStoreD - 1) / kStoreD);
    k_paged_store<<<grid, 256, 0, static_cast<hipStream_t>(stream)>>>(
        T, kv_heads, D, shift, int64_t(n_pages) << shift, static_cast<const uint16_t*>(k), ld_k,
        static_cast<const uint16_t*>(v), ld_v, slot, static_cast<uint16_t*>(k_cache),
        static_cast<uint16_t*>(v_cache));
    if (trace_enabled()) trace_line("paged_store T=%d: %d x %d x %d workgroups", T, grid.x, grid.y, grid.z);
    return op_launched("vqmlp_paged_store");
}
