// norm.hip -- the norms before and after a block, with its gate, its scale and the residual sum.
//
//   u = N(y; post) . gate,   r = res + res_scale u,   x = N(r; pre),
//   N(z; w, b) = (z - mu) rsqrt(mean((z - mu)^2) + eps) (w + w_offset) + b,  mu = 0 for RMS.
//
// One workgroup owns a row and keeps it in registers in FP32 between the two norms, so every
// input is read once and every output written once: bound by HBM bytes at many rows and by the
// two reductions' latency at few (8,192 rows of 5120, BF16 with gates and an FP32 residual: 120 us, 4.9
// TB/s, the rate of a large copy; 8 rows: 4.6 us).  Mean and centred square sum are two reductions,
// never E[z^2] - E[z]^2, which cancels where the mean is large against the spread.
#include "op.h"

#include <algorithm>

namespace vqmlp {

namespace {

// Sum over the workgroup, in every thread.  Two alternating slots in LDS: a slot is written again
// only two reductions later, with the barrier of the one between them in front of it.
constexpr int kMaxWaves = 16;
struct RowSum {
    float* part;  // [2][kMaxWaves]
    int waves, at = 0;
    __device__ __forceinline__ float operator()(float v) {
        v = wave_sum(v);
        if (waves > 1) {
            float* p = part + at * kMaxWaves;
            if ((threadIdx.x & 63) == 0) p[threadIdx.x >> 6] = v;
            __syncthreads();
            v = 0.f;
            for (int i = 0; i < waves; ++i) v += p[i];
            at ^= 1;
        }
        return v;
    }
};

template <class E>
__device__ __forceinline__ void load8(const void* p, int64_t i, float* f) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = lo16<E>(w[j]);
        f[2 * j + 1] = hi16<E>(w[j]);
    }
}
template <class E>
__device__ __forceinline__ void store8(void* p, int64_t i, const float* f) {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack16<E>(f[2 * j], f[2 * j + 1]);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = w;
}
template <class E, bool RES32>
__device__ __forceinline__ void load_res8(const void* p, int64_t i, float* f) {
    if constexpr (RES32) {
        const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
        const f32x4 a = q[0], b = q[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = a[j], f[4 + j] = b[j];
    } else {
        load8<E>(p, i, f);
    }
}
template <class E, bool RES32>
__device__ __forceinline__ void store_res8(void* p, int64_t i, const float* f) {
    if constexpr (RES32) {
        f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + i);
        q[0] = f32x4{f[0], f[1], f[2], f[3]};
        q[1] = f32x4{f[4], f[5], f[6], f[7]};
    } else {
        store8<E>(p, i, f);
    }
}

// CH chunks of 8 elements a thread: H <= threads * CH * 8.
template <class E, bool RES32, int CH>
__global__ void __launch_bounds__(CH == 1 ? 1024 : 512) k_norm(vqmlp_norm_desc d) {
    __shared__ float part[2 * kMaxWaves];
    const int NT = blockDim.x;
    RowSum row_sum{part, NT / 64};
    const int64_t t = blockIdx.x;
    const int H = d.H;
    const float inv = 1.f / float(H);
    float z[CH][8];
    bool in[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        in[c] = (c * NT + int(threadIdx.x)) * 8 < H;
#pragma unroll
        for (int j = 0; j < 8; ++j) z[c][j] = 0.f;
    }
    auto col = [&](int c) { return int64_t(c * NT + int(threadIdx.x)) * 8; };
    // z := (z - mu) / spread * (w + w_offset) + b
    auto norm = [&](const void* w, const void* b) {
        float mu = 0.f;
        if (d.kind == VQMLP_NORM_LAYER) {
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) s += z[c][j];
            mu = row_sum(s) * inv;
        }
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (in[c]) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    z[c][j] -= mu;
                    s = fmaf(z[c][j], z[c][j], s);
                }
            }
        const float rs = rsqrtf(row_sum(s) * inv + d.eps);
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (in[c]) {
                float f[8];
                load8<E>(w, col(c), f);
#pragma unroll
                for (int j = 0; j < 8; ++j) z[c][j] *= rs * (f[j] + d.w_offset);
                if (b) {
                    load8<E>(b, col(c), f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[c][j] += f[j];
                }
            }
    };
    float rin[CH][8];
    if (d.res) {  // issued before the first norm's reduction
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (in[c]) load_res8<E, RES32>(d.res, t * d.ld_res + col(c), rin[c]);
    }
    if (d.y) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (in[c]) load8<E>(d.y, t * d.ld_y + col(c), z[c]);
        if (d.post_w) norm(d.post_w, d.post_b);
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (in[c]) {
                if (d.gate) {
                    float f[8];
                    load8<E>(d.gate, t * d.ld_gate + col(c), f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[c][j] *= f[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    z[c][j] = d.res ? fmaf(d.res_scale, z[c][j], rin[c][j]) : d.res_scale * z[c][j];
            }
    } else {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (in[c]) {
#pragma unroll
                for (int j = 0; j < 8; ++j) z[c][j] = rin[c][j];
            }
    }
    if (d.res_out) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (in[c]) store_res8<E, RES32>(d.res_out, t * d.ld_res_out + col(c), z[c]);
    }
    if (d.x) {
        norm(d.pre_w, d.pre_b);
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (in[c]) store8<E>(d.x, t * d.ld_x + col(c), z[c]);
    }
}

// Any H, stride and element alignment: the row is not kept, each reduction reads it again (from
// L2 after the first).  Every output element is written by the thread that reads it last.  Bound by its
// 2-byte loads and by making r three times: 8,192 rows of 5121, with gates, biases and an FP32 residual:
// 519 us, 4.3 times what a large copy would take.
template <class E, bool RES32>
__global__ void __launch_bounds__(256) k_norm_any(vqmlp_norm_desc d) {
    __shared__ float part[2 * kMaxWaves];
    RowSum row_sum{part, 4};
    const int64_t t = blockIdx.x;
    const int H = d.H;
    const float inv = 1.f / float(H);
    typedef typename E::T T;
    auto at = [&](const void* p, int64_t i) { return float(static_cast<const T*>(p)[i]); };
    auto stats = [&](auto&& value, float* mu, float* rs) {
        *mu = 0.f;
        if (d.kind == VQMLP_NORM_LAYER) {
            float s = 0.f;
            for (int i = threadIdx.x; i < H; i += 256) s += value(i);
            *mu = row_sum(s) * inv;
        }
        float s = 0.f;
        for (int i = threadIdx.x; i < H; i += 256) {
            const float z = value(i) - *mu;
            s = fmaf(z, z, s);
        }
        *rs = rsqrtf(row_sum(s) * inv + d.eps);
    };
    auto scaled = [&](float z, float mu, float rs, const void* w, const void* b, int i) {
        z = (z - mu) * (rs * (at(w, i) + d.w_offset));
        return b ? z + at(b, i) : z;
    };
    float mu1 = 0.f, rs1 = 1.f, mu2 = 0.f, rs2 = 1.f;
    if (d.y && d.post_w) stats([&](int i) { return at(d.y, t * d.ld_y + i); }, &mu1, &rs1);
    auto r_of = [&](int i) {
        float res = 0.f;
        if (d.res)
            res = RES32 ? static_cast<const float*>(d.res)[t * d.ld_res + i]
                        : at(d.res, t * d.ld_res + i);
        if (!d.y) return res;
        float u = at(d.y, t * d.ld_y + i);
        if (d.post_w) u = scaled(u, mu1, rs1, d.post_w, d.post_b, i);
        if (d.gate) u *= at(d.gate, t * d.ld_gate + i);
        return d.res ? fmaf(d.res_scale, u, res) : d.res_scale * u;
    };
    if (d.x) stats(r_of, &mu2, &rs2);
    for (int i = threadIdx.x; i < H; i += 256) {
        const float r = r_of(i);
        if (d.res_out) {
            if constexpr (RES32)
                static_cast<float*>(d.res_out)[t * d.ld_res_out + i] = r;
            else
                static_cast<T*>(d.res_out)[t * d.ld_res_out + i] = T(r);
        }
        if (d.x)
            static_cast<T*>(d.x)[t * d.ld_x + i] = T(scaled(r, mu2, rs2, d.pre_w, d.pre_b, i));
    }
}

template <class E, bool RES32>
const char* launch_norm(vqmlp_norm_desc d, bool vec, int cus, hipStream_t s) {
    const int chunks = d.H / 8;
    // Few rows: latency, so a chunk a thread (8 rows of 5120: 4.1 us in a graph, 4.9 / 5.7 with 2 / 3
    // chunks).  Many: two (8192 rows of 5120 with gates and an FP32 residual: 120 us, 127 / 126 / 130
    // with 1 / 3 / 4); from 2 chunks a thread on a workgroup has at most 512 threads.
    const int ch = !vec || chunks > 2048 ? 0 : chunks > 1024 ? 4 : chunks <= 64 || d.T <= 2 * cus ? 1 : 2;
    const unsigned nt = ch ? unsigned((chunks + 64 * ch - 1) / (64 * ch)) * 64 : 256;
    // a launch of 2^32 threads or more drops rows without an error
    const int most = int((0xFFFFFFFFull / nt) & ~7ull);
    auto behind = [&](const void* p, int64_t ld, int bytes) {
        return p ? reinterpret_cast<void*>(reinterpret_cast<uintptr_t>(p) + most * ld * bytes) : nullptr;
    };
    const int re = RES32 ? 4 : 2;
    for (int left = d.T; left > 0; left -= most) {
        d.T = std::min(left, most);
        switch (ch) {
            case 0: k_norm_any<E, RES32><<<d.T, nt, 0, s>>>(d); break;
            case 1: k_norm<E, RES32, 1><<<d.T, nt, 0, s>>>(d); break;
            case 2: k_norm<E, RES32, 2><<<d.T, nt, 0, s>>>(d); break;
            default: k_norm<E, RES32, 4><<<d.T, nt, 0, s>>>(d);
        }
        d.y = behind(d.y, d.ld_y, 2);
        d.res = behind(d.res, d.ld_res, re);
        d.gate = behind(d.gate, d.ld_gate, 2);
        d.res_out = behind(d.res_out, d.ld_res_out, re);
        d.x = behind(d.x, d.ld_x, 2);
    }
    return ch == 0   ? "element kernel"
           : ch == 1 ? "vector kernel, 1 chunk a thread"
           : ch == 2 ? "vector kernel, 2 chunks a thread"
                     : "vector kernel, 4 chunks a thread";
}

}  // namespace

}  // namespace vqmlp

extern "C" vqmlp_status vqmlp_block_norm(const vqmlp_norm_desc* p, void* stream) {
    using namespace vqmlp;
    OP_REQUIRE(p, "vqmlp_block_norm: null description");
    const vqmlp_norm_desc& d = *p;
    OP_REQUIRE(op_dtype16(d.dtype), "vqmlp_block_norm: dtype %d is not F16 or BF16", d.dtype);
    OP_REQUIRE(d.res_dtype == d.dtype || d.res_dtype == VQMLP_F32,
               "vqmlp_block_norm: res_dtype %d is neither dtype nor F32", d.res_dtype);
    OP_REQUIRE(d.kind == VQMLP_NORM_RMS || d.kind == VQMLP_NORM_LAYER,
               "vqmlp_block_norm: unknown norm kind %d", d.kind);
    OP_REQUIRE(d.T >= 0 && d.H >= 1 && d.H <= (1 << 20), "vqmlp_block_norm: T=%d, H=%d out of range",
               d.T, d.H);
    if (d.T == 0) return op_ok();
    OP_REQUIRE(d.y || d.res, "vqmlp_block_norm: neither y nor res");
    OP_REQUIRE(d.x || d.res_out, "vqmlp_block_norm: neither x nor res_out");
    OP_REQUIRE(!d.x || d.pre_w, "vqmlp_block_norm: x needs pre_w");
    OP_REQUIRE(d.y || (!d.post_w && !d.gate), "vqmlp_block_norm: post_w or gate without y");
    OP_REQUIRE(d.eps >= 0.f, "vqmlp_block_norm: eps is negative or NaN");
    const size_t re = d.res_dtype == VQMLP_F32 ? 4 : 2;
    const struct { const void* p; int64_t ld; size_t e; const char* name; } rows[] = {
        {d.y, d.ld_y, 2, "y"},           {d.res, d.ld_res, re, "res"},
        {d.gate, d.ld_gate, 2, "gate"},  {d.res_out, d.ld_res_out, re, "res_out"},
        {d.x, d.ld_x, 2, "x"}};
    bool vec = d.H % 8 == 0;
    for (const auto& r : rows) {
        if (!r.p) continue;
        const bool shared = r.p == d.gate && r.ld == 0;
        OP_REQUIRE(shared || r.ld >= d.H || d.T == 1, "vqmlp_block_norm: row stride of %s is below H",
                   r.name);
        OP_REQUIRE(r.ld >= 0 && r.ld <= (int64_t(1) << 40), "vqmlp_block_norm: row stride of %s", r.name);
        OP_REQUIRE(op_aligned(r.p, r.e), "vqmlp_block_norm: %s is not aligned to its type", r.name);
        vec = vec && r.ld % 8 == 0 && op_aligned(r.p, 16);
    }
    for (const void* w : {d.post_w, d.post_b, d.pre_w, d.pre_b}) {
        OP_REQUIRE(op_aligned(w, 2), "vqmlp_block_norm: a weight is not aligned to its type");
        vec = vec && op_aligned(w, 16);
    }
    int cus = 0;
    if (const int st = device_cus(&cus)) return static_cast<vqmlp_status>(st);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool r32 = d.res_dtype == VQMLP_F32;
    const char* what =
        d.dtype == VQMLP_F16 ? (r32 ? launch_norm<F16, true>(d, vec, cus, s) : launch_norm<F16, false>(d, vec, cus, s))
                             : (r32 ? launch_norm<BF16, true>(d, vec, cus, s) : launch_norm<BF16, false>(d, vec, cus, s));
    if (trace_enabled()) trace_line("block_norm T=%d H=%d: %s", d.T, d.H, what);
    return op_launched("vqmlp_block_norm");
}
