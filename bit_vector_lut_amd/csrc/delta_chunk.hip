// delta_chunk.hip -- gated delta rule over chunks of 64 tokens on the matrix cores (gfx950).
//
// With b_t = g_1 + .. + g_t inside a chunk and S the state before it,
//   A_tj = beta_t e^{b_t - b_j} k_t . k_j  (j < t),   T = (I + A)^-1 diag(beta)
//   U  = T (V - diag(e^b) K S)
//   y  = scale (diag(e^b) Q S + P U),  P_tj = e^{b_t - b_j} q_t . k_j  (j <= t)
//   S' = e^{b_64} S + K^T diag(e^{b_64 - b}) U.
// T and P do not depend on the state: k_delta_prep makes them for all chunks at once.  k_delta_scan goes
// through a request's chunks in order.  There a wave owns 16 value columns of the state and all that
// follows from them, so that the chain S -> K S -> U -> S' stays in its registers: each product's result
// lies, per lane, as eight neighbouring rows of one column, which is the next product's operand.
//
// Precision.  What reaches the state keeps FP32 accuracy: matrix-core operands made here (S, V - K S, T, U)
// are sums of two binary16 parts (22 bits) in units of 2^-e that put a column's (of T, a row's) largest
// element into the upper range of binary16.  The state and U may be smaller than the values by the sizes of
// the keys and of beta: their units are 2^-(e + lift) and 2^-(e + ulift), lift and ulift the same for all columns
// of a chunk.  Keys and queries are binary16 as they are; bfloat16 ones become binary16 by a power of two for
// each row, which leaves out at most 2^-40 of a query's largest element (brought to 2^14), 2^-25 of a key's (brought
// to 1: K^T U is added to the state as it comes).  The outputs are made of two parts of P, U and S too, so that
// their one rounding is at the end, as in the recurrence: 2.1e-4 of their norm off (binary16), where one part of
// each gives 3.4e-4 and one of P alone 2.7e-4 (three prompts: 282, 257 and 268 us).  The second parts of U and S
// go to the outputs' waves in the place of T, which they load again.  The triangular system is solved in FP32.
//
// Bound: not by memory or the matrix cores (three prompts of 8,073 tokens, 48 heads of 128 x 128: 282 us a call, where
// the bytes take 58 and the products 39), but by the chain.  A chunk's products depend on each other and on conversions
// between them: 2.2 us alone on a compute unit, 2.7 beside another workgroup, of which the matrix cores work 0.6.
// k_delta_prep (75 us of it) writes 188 MB and reads 57: 67% of a copy's rate, with LDS and the triangular solve.
// The scan with outputs has no register left for heads of 128: it takes all 256 and keeps 8 (binary16) or 31 (bfloat16)
// in memory, some of them from chunk to chunk.
#include "delta.h"

#include <algorithm>

namespace vqmlp {

namespace {

constexpr int kC = kDeltaC;
constexpr int kIdle = 1 << 16;

// A block of the workspace: parts of T and P as the lanes of the matrix cores take them (1 KB each) and
// factors for each token; what the state's chain takes, then what the outputs take.
struct StateBlock {
    u32x4 th[6][64], tl[6][64];
    float xf[kC];  // e^b 2^(kexp - lift): of K S
    float uf[kC];  // the unit of T's row, and 2^ulift
    float tf[kC];  // e^(b_64 - b) 2^(kexp + lift - ulift): of U where it joins the state
    float etot;    // e^b_64
    int bad;       // first token with something not finite in k, g or beta, or 64
    int lift;      // the state is in units of 2^-lift of the values' here; kIdle: of 1, and no token changes it
    int pad[61];
};
struct OutBlock {
    u32x4 ph[6][64], pl[6][64];
    float qf[kC];  // e^b in the units of P's row and U: of Q S
    int pe[kC];    // exponent of the scale and of the units of P's row, of U and of the query
    int pad[128];
};
struct DeltaBlock {
    StateBlock s;
    OutBlock o;
};
static_assert(sizeof(StateBlock) == 13 * 1024 && sizeof(DeltaBlock) == kDeltaBlock, "block");

__device__ uint32_t kZeros[4] = {0, 0, 0, 0};  // where rows and columns that do not exist are read

// Rows of K in LDS: 16-byte chunks, their order within a row changed by an exclusive or so that both ways
// of reading an operand (16 rows 8 (m / 4) + m % 4 of one chunk; four neighbouring rows of four chunks,
// transposed) touch all banks evenly.
template <int DKP>
__device__ __forceinline__ int kkey(int r) {
    return DKP == 64 ? (r & 2) << 1 | (r >> 3 & 1) | (r >> 3 & 2) : (r & 3) << 2 | (r >> 3 & 3);
}
// Row m of tile b of a pair of row tiles: a lane's four results of both are eight neighbours.
__device__ __forceinline__ int pair_row(int m, int b) { return 8 * (m >> 2) + 4 * b + (m & 3); }

// e^x of a log in base 2
__device__ __forceinline__ float exp_b(double b) {
    const float h = float(b), r = float(b - double(h));
    return __builtin_amdgcn_exp2f(h) * fmaf(r, kLn2, 1.f);
}

// Parts of eight values: hi + lo, the latter of what rounding left.
__device__ __forceinline__ u32x4 pack_hi(const float* x) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t z = pack16<F16>(x[2 * i], x[2 * i + 1]);
        // one rounded value for the operand and for what is left of x
        asm("" : "+v"(z));
        w[i] = z;
    }
    return w;
}
// By mixed multiply-adds, which round to binary16 themselves: half the instructions of what the compiler makes.
// The halves of a word are written four instructions apart and read by a matrix-core step two or more behind;
// what they read has been read by pack_hi, which waited for it.
__device__ __forceinline__ u32x4 pack_lo(const float* x, u32x4 hi) {
    uint32_t a, b, c, d;
    asm("v_fma_mixlo_f16 %0, %4, -1.0, %8 op_sel_hi:[1,0,0]\n\t"
        "v_fma_mixlo_f16 %1, %5, -1.0, %10 op_sel_hi:[1,0,0]\n\t"
        "v_fma_mixlo_f16 %2, %6, -1.0, %12 op_sel_hi:[1,0,0]\n\t"
        "v_fma_mixlo_f16 %3, %7, -1.0, %14 op_sel_hi:[1,0,0]\n\t"
        "v_fma_mixhi_f16 %0, %4, -1.0, %9 op_sel:[1,0,0] op_sel_hi:[1,0,0]\n\t"
        "v_fma_mixhi_f16 %1, %5, -1.0, %11 op_sel:[1,0,0] op_sel_hi:[1,0,0]\n\t"
        "v_fma_mixhi_f16 %2, %6, -1.0, %13 op_sel:[1,0,0] op_sel_hi:[1,0,0]\n\t"
        "v_fma_mixhi_f16 %3, %7, -1.0, %15 op_sel:[1,0,0] op_sel_hi:[1,0,0]\n\t"
        "s_nop 1"
        : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d)
        : "v"(hi[0]), "v"(hi[1]), "v"(hi[2]), "v"(hi[3]), "v"(x[0]), "v"(x[1]), "v"(x[2]), "v"(x[3]), "v"(x[4]), "v"(x[5]),
          "v"(x[6]), "v"(x[7]));
    return u32x4{a, b, c, d};
}

// Largest bits of eight 16-bit magnitudes
__device__ __forceinline__ uint32_t top8(u32x4 x) {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) t = max(t, max(x[i] & 0x7FFFu, x[i] >> 16 & 0x7FFFu));
    return t;
}
// ... of a lane's values of a chunk
__device__ __forceinline__ uint32_t largest(const u32x2 (&x)[2][2]) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 t = {0, 0};
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2, x[p][b][i] & 0x7FFF7FFFu));
    return max(t[0], t[1]);
}
template <class E>
constexpr uint32_t kInf16 = __is_same(E, F16) ? 0x7C00u : 0x7F80u;

// bfloat16 to binary16 in units of 2^e
__device__ __forceinline__ u32x4 to_half(u32x4 x, float by) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = lo16<BF16>(x[i]) * by, f[2 * i + 1] = hi16<BF16>(x[i]) * by;
    return pack_hi(f);
}
// The exponent of a key's largest element, of these bits; kNoKey of a key of zeros.
constexpr int kNoKey = -200;
__device__ __forceinline__ int key_expo(uint32_t top) {
    return top == 0 ? kNoKey : top >= 0x7F80u ? 0 : min(max(int(top >> 7) - 127, -126), 126);
}
// The power of two that brings the largest of a row, of these bits, to 2^14 or as near as FP32 holds the factor.
__device__ __forceinline__ int query_unit(uint32_t top) {
    return top == 0 || top >= 0x7F80u ? 0 : min(14 + 127 - max(int(top >> 7), 1), 126);
}

template <int DKP>
struct PrepSmem {
    union {
        __attribute__((aligned(256))) uint16_t k[kC * DKP];
        __attribute__((aligned(256))) float AT[2][kC][kC + 4];  // A and T of a value head
    };
    float b[kC], lo[kC];  // b log2 e and what it lost in rounding
    float beta[kC];
    int kexp[kC];
    int lift, ulift;
    int kbad, bad;  // first token with something not finite in k; or in g or beta
};

// c ? v : 0 without a branch around what made v
__device__ __forceinline__ float only(bool c, float v) {
    asm("" : "+v"(v));
    return c ? v : 0.f;
}

// 2^(b_t - b_j) from the two parts of the b's
__device__ __forceinline__ float decayed(float bt, float lt, float bj, float lj) {
    return __builtin_amdgcn_exp2f((bt - bj) + (lt - lj));
}

// Where 2^top in a band of 8 powers has to go to end up between 2^-4 and 2^4
__device__ __forceinline__ int band(int top) { return -((top + 4) & ~7); }

// A workgroup makes the blocks of `per` value heads that share a key head: K K^T and Q K^T are theirs together.
// Tiles of 16 x 16: each wave has one on the diagonal of A and one or two of the six below.
template <class E, int DKP>
__global__ void __launch_bounds__(256, 4) k_delta_prep(DeltaArgs a, int per) {
    constexpr int KS = DKP / 32;
    constexpr bool HALF = __is_same(E, F16);
    __shared__ PrepSmem<DKP> sm;
    float (*const A)[kC + 4] = sm.AT[0], (*const T)[kC + 4] = sm.AT[1];
    const int heads = a.hv / a.hk, parts = heads / per;
    const int64_t id = a.id0 + blockIdx.x, pair = id / (8 * parts) * 8 + id % 8;
    const int hk = int(pair % a.hk), h0 = hk * heads + int(id / 8 % parts) * per;
    const int x = int(pair / a.hk);
    PackedUnit u;
    if (!packed_unit(a.p, kC, x, u)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int lr = lane & 15, g4 = lane >> 4;
    const int64_t t0 = u.c0 + int64_t(u.seg) * kC;
    const int m = min(kC, u.n - u.seg * kC);
    if (u.r == a.p.R) {  // rows behind the last request
        const int row = per * a.Dv / 8;
        for (int i = tid; i < m * row; i += 256)
            *reinterpret_cast<u32x4*>(a.y + (t0 + i / row) * a.ld_y + int64_t(h0) * a.Dv + i % row * 8) = u32x4{0, 0, 0, 0};
        return;
    }
    if (m <= 0 || u.n <= a.few) return;
    uint16_t* const image = a.image(x, hk, DKP, HALF);
    const bool first = h0 % heads == 0;
    const u32x4 none = {0, 0, 0, 0};

    // keys
    constexpr int LPR = DKP / 8, RPP = 256 / LPR;
    u32x4 kr[kC / RPP];
    const int kc = tid % LPR;
#pragma unroll
    for (int i = 0; i < kC / RPP; ++i) {
        const int r = i * RPP + tid / LPR;
        kr[i] = none;
        if (r < m && 8 * kc < a.Dk) kr[i] = *reinterpret_cast<const u32x4*>(a.k + (t0 + r) * a.ld_k + int64_t(hk) * a.Dk + 8 * kc);
    }
    // this wave's 16 queries
    u32x4 qf[KS];
    uint32_t qtop = 0;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        qf[s] = none;
        if (16 * wave + lr < m && 32 * s + 8 * g4 < a.Dk)
            qf[s] = *reinterpret_cast<const u32x4*>(a.q + (t0 + 16 * wave + lr) * a.ld_q + int64_t(hk) * a.Dk + 32 * s + 8 * g4);
    }
    float gv = 0.f, bv = 0.f;  // of token `lane` of the next head (wave 0)
    auto gates = [&](int h) __attribute__((always_inline)) {
        if (wave == 0 && lane < m) {
            gv = a.g[(t0 + lane) * a.ld_g + h];
            bv = a.beta[(t0 + lane) * a.ld_b + h];
        }
    };
    gates(h0);
    if (tid == 0) sm.kbad = kC;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kC / RPP; ++i) {
        const int r = i * RPP + tid / LPR;
        uint32_t top = top8(kr[i]);
        if constexpr (!HALF) {
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1) top = max(top, uint32_t(__shfl_xor(int(top), o)));
            const int e = key_expo(top);
            kr[i] = to_half(kr[i], e == kNoKey ? 1.f : pow2(-e));
            if (kc == 0) sm.kexp[r] = e;
            if (first) *reinterpret_cast<u32x4*>(image + kC * DKP + r * DKP + 8 * kc) = kr[i];
        }
        if (top >= kInf16<E>) atomicMin(&sm.kbad, r);
        *reinterpret_cast<u32x4*>(&sm.k[r * DKP + 8 * (kc ^ kkey<DKP>(r))]) = kr[i];
    }
    int qe = 0;  // the row of queries is in units of 2^-qe
    if constexpr (!HALF) {
#pragma unroll
        for (int s = 0; s < KS; ++s) qtop = max(qtop, top8(qf[s]));
        // the lanes of a row are 16 apart
        qtop = max(qtop, uint32_t(__shfl_xor(int(qtop), 16)));
        qtop = max(qtop, uint32_t(__shfl_xor(int(qtop), 32)));
        qe = query_unit(qtop);
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[s] = to_half(qf[s], pow2(qe));
    }
    if (first) {
#pragma unroll
        for (int s = 0; s < KS; ++s) *reinterpret_cast<u32x4*>(image + ((wave * KS + s) * 64 + lane) * 8) = qf[s];
    }
    __syncthreads();
    const int kbad = sm.kbad;
    int kmax = 0;  // of the chunk's keys: P is made in its units
    if constexpr (!HALF) {
        kmax = __builtin_amdgcn_readlane(lane_scan(sm.kexp[lane], kNoKey, [](int p, int q) { return max(p, q); }), 63);
        if (kmax == kNoKey) kmax = 0;
    }
    auto k_read = [&](int r, int s) {
        return *reinterpret_cast<const u32x4*>(&sm.k[r * DKP + 8 * ((4 * s + g4) ^ kkey<DKP>(r))]);
    };
    // K K^T: tile (wave, wave), then (1, 0) and (3, 1); (2, 0) and (3, 2); (2, 1); (3, 0)
    const int bi[3] = {wave, wave == 0 ? 1 : wave == 3 ? 3 : 2, 3}, bj[3] = {wave, wave == 2 ? 1 : 0, wave + 1};
    f32x4 kk[3];
#pragma unroll
    for (int z = 0; z < 3; ++z) {
        kk[z] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (z == 2 && wave > 1) continue;
#pragma unroll
        for (int s = 0; s < KS; ++s) kk[z] = F16::mfma16(k_read(16 * bi[z] + lr, s), k_read(16 * bj[z] + lr, s), kk[z]);
    }
    // K Q^T of this wave's queries: a lane has eight neighbouring keys of one query
    f32x4 qk[2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            qk[c][b] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (c > wave / 2) continue;
#pragma unroll
            for (int s = 0; s < KS; ++s) qk[c][b] = F16::mfma16(k_read(32 * c + pair_row(lr, b), s), qf[s], qk[c][b]);
        }
    __syncthreads();  // K is done with: A and T stand in its place

#pragma unroll 1
    for (int h = h0; h < h0 + per; ++h) {
        const int lane = fresh(tid & 63), lr = lane & 15, g4 = lane >> 4;  // no addresses kept over the loop
        DeltaBlock& blk = reinterpret_cast<DeltaBlock*>(a.blocks)[int64_t(x) * a.hv + h];
        if (wave == 0) {
            const float g = lane < m ? bounded(gv) : 0.f, beta = lane < m ? bv : 0.f;
            const uint64_t odd = __ballot(!(fabsf(g) < __builtin_inff() && fabsf(beta) < __builtin_inff()));
            const int bad = min(kbad, odd ? __builtin_ctzll(odd) : kC);
            // sums in FP64: behind strong decays b reaches thousands, and T and P take differences of neighbours
            const double b = lane_scan(double(g) * 1.4426950408889634, 0., [](double p, double q) { return p + q; });
            const int ke = HALF ? 0 : sm.kexp[lane];
            const double all = __shfl(b, 63);
            // The state and U in units of their own, which follow the largest |k| beta and beta: from a state of zeros
            // they are as much smaller than the values.  Bands keep the units the same from chunk to chunk.  The state's is
            // bounded, since it may hold what other chunks left.
            constexpr int none = -1000;
            struct Two {
                int key, beta;
            };
            const int be = lane < bad && beta != 0.f && ke != kNoKey ? expo(beta) : none;
            const Two top = lane_scan(Two{be == none ? none : ke + be, be}, Two{none, none}, [](Two p, Two q) {
                return Two{max(p.key, q.key), max(p.beta, q.beta)};
            });
            const int tk = __builtin_amdgcn_readlane(top.key, 63), tb = __builtin_amdgcn_readlane(top.beta, 63);
            const int far = min(64, 126 - kmax);
            const int lift = tk == none ? 0 : min(max(band(tk), max(-64, kmax - 126)), far);
            const int ulift = tb == none ? 0 : min(max(band(tb), -64), 120);
            sm.b[lane] = float(b);
            sm.lo[lane] = float(b - double(float(b)));
            sm.beta[lane] = beta;
            blk.s.xf[lane] = exp_b(b + double(ke - lift));
            blk.s.tf[lane] = exp_b(all - b + double(ke + lift - ulift));
            if (lane == 0) {
                sm.bad = bad, sm.lift = lift, sm.ulift = ulift;
                blk.s.etot = exp_b(all), blk.s.bad = bad, blk.s.lift = tb == none ? kIdle : lift;
            }
        }
        __syncthreads();
        if (h + 1 < h0 + per) gates(h + 1);
        const int bad = sm.bad;
        // A
#pragma unroll
        for (int z = 0; z < 3; ++z) {
            if (z == 2 && wave > 1) break;
            const int cj = 16 * bj[z] + lr, r0 = 16 * bi[z] + 4 * g4;
            const float bjv = sm.b[cj], lj = sm.lo[cj];
            const f32x4 bt = *reinterpret_cast<const f32x4*>(&sm.b[r0]), lt = *reinterpret_cast<const f32x4*>(&sm.lo[r0]);
            const f32x4 be = *reinterpret_cast<const f32x4*>(&sm.beta[r0]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = r0 + i;
                float v = kk[z][i] * be[i] * decayed(bt[i], lt[i], bjv, lj);
                if constexpr (!HALF) v = __builtin_ldexpf(v, sm.kexp[cj] + sm.kexp[t]);
                A[t][cj] = only(cj < t && t < bad, v);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        // (I + A)^-1 of this wave's diagonal tile: of its 4 x 4 blocks by substitution, then twice blocks of double
        // size, D - D O D with O the blocks of A between two that D has.  A step of the FP32 products takes one row of
        // each lane group's four, so that a result is the next product's operand.
        {
            f32x4 d, row[3];
#pragma unroll
            for (int i = 0; i < 3; ++i) row[i] = *reinterpret_cast<const f32x4*>(&A[16 * wave + 4 * g4 + i + 1][16 * wave + 4 * g4]);
            const f32x4 ar = *reinterpret_cast<const f32x4*>(&A[16 * wave + lr][16 * wave + 4 * g4]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                d[i] = (lr & 3) == i ? 1.f : 0.f;
#pragma unroll
                for (int j = 0; j < i; ++j) d[i] = fmaf(-row[i - 1][j], d[j], d[i]);
            }
            d *= lr / 4 == g4 ? 1.f : 0.f;
            auto keep = [&]() __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) T[16 * wave + 4 * g4 + i][16 * wave + lr] = d[i];
            };
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                keep();
                const f32x4 dr = *reinterpret_cast<const f32x4*>(&T[16 * wave + lr][16 * wave + 4 * g4]);
                const bool between = z == 0 ? (lr & 4) && g4 == (lr >> 2) - 1 : lr >= 8 && g4 < 2;
                f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = x;
#pragma unroll
                for (int i = 0; i < 4; ++i) x = __builtin_amdgcn_mfma_f32_16x16x4f32(between ? ar[i] : 0.f, d[i], x, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) y = __builtin_amdgcn_mfma_f32_16x16x4f32(dr[i], x[i], y, 0, 0, 0);
                d -= y;
            }
            keep();
        }
        __builtin_amdgcn_sched_barrier(0);
        // P, of the queries in their units
        {
            const int t = 16 * wave + lr;
            const float bt = sm.b[t], lt = sm.lo[t];
            float p[2][8], top = 0.f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (c > wave / 2) break;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int j0 = 32 * c + 8 * g4 + 4 * b;
                    const f32x4 bjv = *reinterpret_cast<const f32x4*>(&sm.b[j0]), lj = *reinterpret_cast<const f32x4*>(&sm.lo[j0]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = j0 + i;
                        float v = qk[c][b][i] * decayed(bt, lt, bjv[i], lj[i]);
                        if constexpr (!HALF) v = __builtin_ldexpf(v, sm.kexp[j] - kmax);
                        p[c][4 * b + i] = only(j <= t && j < bad, v);
                        top = fmaxf(top, fabsf(p[c][4 * b + i]));
                    }
                }
            }
            top = column_max(top);
            // Q S, which is below 2^34 in its units, takes 2^(e + more) too
            const int more = sm.ulift - sm.lift - kmax;
            const int e = min(top > 0.f ? max(14 - expo(top), -60) : 0, 60 - max(more, 0));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (c > wave / 2) break;
#pragma unroll
                for (int i = 0; i < 8; ++i) p[c][i] *= pow2(e);
                const u32x4 hi = pack_hi(p[c]);
                const int at = wave < 2 ? wave : 2 * wave - 2 + c;
                blk.o.ph[at][lane] = hi;
                blk.o.pl[at][lane] = pack_lo(p[c], hi);
            }
            if (g4 == 0) {
                blk.o.qf[t] = __builtin_ldexpf(decayed(bt, lt, 0.f, 0.f), e + more);
                blk.o.pe[t] = __builtin_amdgcn_frexp_expf(a.scale) - e - qe + kmax - sm.ulift;
            }
        }
        __syncthreads();
        // the tiles below: T_ij = -T_ii sum_m A_im T_mj, a column of tiles a wave
        {
            f32x4 tc[4];
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                if (j != wave) continue;
#pragma unroll
                for (int i = 0; i < 4; ++i) tc[j][i] = T[16 * j + 4 * g4 + i][16 * j + lr];
#pragma unroll
                for (int i = j + 1; i < 4; ++i) {
                    f32x4 y = {0.f, 0.f, 0.f, 0.f}, z = y;
#pragma unroll
                    for (int k = j; k < i; ++k) {
                        const f32x4 r = *reinterpret_cast<const f32x4*>(&A[16 * i + lr][16 * k + 4 * g4]);
#pragma unroll
                        for (int s = 0; s < 4; ++s) y = __builtin_amdgcn_mfma_f32_16x16x4f32(r[s], tc[k][s], y, 0, 0, 0);
                    }
                    const f32x4 r = *reinterpret_cast<const f32x4*>(&T[16 * i + lr][16 * i + 4 * g4]);
#pragma unroll
                    for (int s = 0; s < 4; ++s) z = __builtin_amdgcn_mfma_f32_16x16x4f32(r[s], -y[s], z, 0, 0, 0);
                    tc[i] = z;
#pragma unroll
                    for (int s = 0; s < 4; ++s) T[16 * i + 4 * g4 + s][16 * j + lr] = z[s];
                }
            }
        }
        __syncthreads();
        // T as operands
        {
            const int c1 = wave / 2, t = 32 * c1 + pair_row(lr, wave & 1);
            float v[2][8], top = 0.f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (c > c1) break;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int j = 32 * c + 8 * g4 + i;
                    v[c][i] = only(j <= t && j < bad, T[t][j] * sm.beta[j]);
                    top = fmaxf(top, fabsf(v[c][i]));
                }
            }
            top = column_max(top);
            const int e = top > 0.f ? min(max(13 - expo(top), -120), 126) : 0;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (c > c1) break;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[c][i] *= pow2(e);
                const u32x4 hi = pack_hi(v[c]);
                const int at = wave < 2 ? wave : 2 * wave - 2 + c;
                blk.s.th[at][lane] = hi;
                blk.s.tl[at][lane] = pack_lo(v[c], hi);
            }
            if (g4 == 0) blk.s.uf[t] = __builtin_ldexpf(1.f, sm.ulift - e);
        }
        __syncthreads();  // b and beta are read
    }
}

// ---------------------------------------------------------------- the chunks in order
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Maximum over the lanes with the same lane % 16, in all of them
__device__ __forceinline__ int column_max(int v) {
    const auto x = __builtin_amdgcn_permlane32_swap(uint32_t(v), uint32_t(fresh(v)), false, false);
    v = max(int(x[0]), int(x[1]));
    const auto y = __builtin_amdgcn_permlane16_swap(uint32_t(v), uint32_t(fresh(v)), false, false);
    return max(int(y[0]), int(y[1]));
}

constexpr int kPairs = 2, kCols = 16 * kPairs;  // pairs of waves, value columns of a workgroup

// What the state's chain reads of a chunk, what the outputs read, and what the chain hands to the outputs.
template <int DKP>
struct ChainStage {
    __attribute__((aligned(1024))) uint16_t k[kC * DKP], v[kC * kCols];
    StateBlock d;
};
template <int DKP>
struct ScanSmem {
    ChainStage<DKP> chain[2];  // of this chunk and the next
    u32x4 sh[kPairs][DKP / 32][64], uo[kPairs][2][64];  // of each wave: the state before the chunk, U
    __attribute__((aligned(16))) int unit[kCols], from[kCols];  // of a column: e, first token without a number
};

// Whole requests: the longest first, or a long one starts when the others are done.  Up to 64 requests; of more the
// x-th that the recurrence leaves, -1 where there is none.
__device__ __forceinline__ int nth_request(const Packed& p, int few, int x) {
    const int lane = threadIdx.x & 63;
    auto length = [&](int r) { return r < p.R ? packed_row(p, r + 1) - packed_row(p, r) : -1; };
    if (p.R <= 64) {
        const int n = length(lane);
        int rank = 0;
        for (int j = 0; j < p.R; ++j) {
            const int m = __builtin_amdgcn_readlane(n, j);
            rank += m > n || (m == n && j < lane);
        }
        return __builtin_ctzll(__ballot(rank == x && lane < p.R) | 1ull << 63);
    }
    if (few < 0) return x;
    for (int r = 0; r < p.R; r += 64) {
        const bool mine = length(r + lane) > few;
        const uint64_t mask = __ballot(mine);
        const int count = __builtin_popcountll(mask);
        if (x < count) return r + __builtin_ctzll(__ballot(mine && __builtin_popcountll(mask & ((1ull << lane) - 1)) == x) | 1ull << 63);
        x -= count;
    }
    return -1;
}

// Two waves for each 16 columns of the state: one has the chain from state to state, the other the
// outputs of the chunk before it and all loads.  A wave issues an instruction every four cycles at most: in one
// wave outputs and loads took longer than the chain, with little under the matrix cores' steps.
//
// Segments.  Few heads and few requests leave most compute units idle, so the chunks of a request may go through
// in segments at once.  U and the state are linear in the state before a segment, S -> M S + B: a first launch
// (OUT false) makes of each segment but the last B, from a state of zeros and with the values, and M, from
// a state of ones on the diagonal and without (of the first segment its end from the request's own state); then
// k_delta_join goes through the segments, and the second launch makes the outputs of all from their states.
template <class E, int DKP, bool OUT>
__global__ void __launch_bounds__(128 * kPairs, 2) k_delta_scan(DeltaArgs a) {
    constexpr int KS = DKP / 32;
    constexpr bool HALF = __is_same(E, F16);
    __shared__ ScanSmem<DKP> sm;
    const int slices = (a.Dv + kCols - 1) / kCols, all = slices + (OUT ? 0 : (a.Dk + kCols - 1) / kCols);
    // The slices of a head are 8 apart, on one XCD, one after another.  (Not all heads of a key head: with few units
    // that gave some XCDs more workgroups than compute units, and the launch twice the time.)
    const int64_t id = a.id0 + blockIdx.x, pair = id / (8 * all) * 8 + id % 8;
    const int h = int(pair % a.hv), hk = h / (a.hv / a.hk), j0 = int(id / 8 % all), x = int(pair / a.hv);
    const int v0 = j0 % slices * kCols;
    const bool ones = !OUT && j0 >= slices;  // columns of M
    const int i0 = ones ? (j0 - slices) * kCols : v0;
    PackedUnit u;
    const int number = a.seg || x >= a.p.R ? x : nth_request(a.p, a.few, x);
    if (number < 0 || !packed_unit(a.p, a.L, number, u) || u.r >= a.p.R || u.n <= a.few) return;
    if (!OUT && (u.seg == u.nseg - 1 || (ones && u.seg == 0))) return;
    const int tid = threadIdx.x, lane = tid & 63, both = uniform(tid >> 6), wave = both % kPairs;
    const int lr = lane & 15, g4 = lane >> 4;
    const int c0 = u.c0 + u.seg * a.L, n = min(u.n - u.seg * a.L, a.L);
    const int nch = (n + kC - 1) / kC;

    if (both >= kPairs) {
        // ---- loads and outputs.  Loads straight to LDS, 1 KB each: bases that the wave shares plus 32-bit offsets of the
        // lanes, which stay the same from chunk to chunk.
        constexpr int LPR = DKP / 8, RPI = 64 / LPR, NI = kC / RPI / kPairs, NV = kC * kCols / 512 / kPairs;
        const int64_t ldk = 2 * (HALF ? a.ld_k : DKP), ldv = 2 * a.ld_v;  // bytes
        const int64_t unit0 = u.c0 / kC + u.r + u.seg * (a.L / kC);  // number of the first chunk's block
        const uint8_t* qp = reinterpret_cast<const uint8_t*>(a.image(unit0, hk, DKP, HALF));
        const uint8_t* kp = HALF ? reinterpret_cast<const uint8_t*>(a.k + int64_t(hk) * a.Dk) + c0 * ldk : qp + kC * DKP * 2;
        const uint8_t* vp = reinterpret_cast<const uint8_t*>(a.v + int64_t(h) * a.Dv + v0) + c0 * ldv;
        const uint8_t *dp = a.blocks + (unit0 * a.hv + h) * kDeltaBlock, *pp = dp + sizeof(StateBlock);
        const int64_t qstep = int64_t(a.hk) * (HALF ? 1 : 2) * (kC * DKP * 2), kstep = HALF ? kC * ldk : qstep;
        const int64_t vstep = kC * ldv, dstep = int64_t(a.hv) * kDeltaBlock;
        uint32_t koff[NI], voff[NV];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int row = (wave * NI + i) * RPI + lane / LPR;
            koff[i] = uint32_t(row) * uint32_t(ldk) + 16 * uint32_t(lane % LPR ^ kkey<DKP>(row));
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = (wave * NV + i) * 64 + lane;
            voff[i] = uint32_t(at / (kCols / 8)) * uint32_t(ldv) + 16 * uint32_t(at % (kCols / 8));
        }
        const uint8_t* const zeros = reinterpret_cast<const uint8_t*>(kZeros);  // rows and columns that are not there
        const bool kwide = !HALF || a.Dk == DKP, vwide = !ones && v0 + kCols <= a.Dv;
        auto load_chain = [&](int c) __attribute__((always_inline)) {
            const int m = min(kC, n - c * kC);
            const uint32_t at = lds_byte(&sm.chain[c & 1]);
            if (__builtin_expect(kwide && m == kC, 1)) {
#pragma unroll
                for (int i = 0; i < NI; ++i) load_lds16(kp, koff[i], at + (wave * NI + i) * 1024);
            } else {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int row = (wave * NI + i) * RPI + lane / LPR, ch = lane % LPR ^ kkey<DKP>(row);
                    load_lds16(row < m && (!HALF || 8 * ch < a.Dk) ? kp + koff[i] : zeros, at + (wave * NI + i) * 1024);
                }
            }
            const uint32_t vto = at + int(offsetof(ChainStage<DKP>, v)) + wave * NV * 1024;
            if (__builtin_expect(vwide && m == kC, 1)) {
#pragma unroll
                for (int i = 0; i < NV; ++i) load_lds16(vp, voff[i], vto + i * 1024);
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int j = (wave * NV + i) * 64 + lane;
                    const bool there = !ones && j / (kCols / 8) < m && v0 + j % (kCols / 8) * 8 < a.Dv;
                    load_lds16(there ? vp + voff[i] : zeros, vto + i * 1024);
                }
            }
#pragma unroll
            for (int i = 0; i < (12 + kPairs) / kPairs; ++i) {
                const int j = wave + kPairs * i;
                // the second parts of the chunk before lie there, in the place of the wave's own pieces
                if (OUT && i == 0) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                if (j < 13) load_lds16(dp + j * 1024, lane * 16, at + int(offsetof(ChainStage<DKP>, d)) + j * 1024);
            }
            kp += kstep, vp += vstep, dp += dstep;
        };
        // queries and P straight to registers, as the matrix cores take them
        u32x4 q[4][KS], ph[6], pl[6];
        float qf[4];
        int pe[4];
        auto load_out = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int s = 0; s < KS; ++s) q[x][s] = *reinterpret_cast<const u32x4*>(qp + ((x * KS + s) * 1024 + lane * 16));
#pragma unroll
            for (int i = 0; i < 6; ++i) {
                ph[i] = *reinterpret_cast<const u32x4*>(pp + (i * 1024 + lane * 16));
                pl[i] = *reinterpret_cast<const u32x4*>(pp + ((6 + i) * 1024 + lane * 16));
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                qf[x] = *reinterpret_cast<const float*>(pp + (int(offsetof(OutBlock, qf)) + (16 * x + lr) * 4));
                pe[x] = *reinterpret_cast<const int*>(pp + (int(offsetof(OutBlock, pe)) + (16 * x + lr) * 4));
            }
            qp += qstep, pp += dstep;
        };
        uint8_t* yp = reinterpret_cast<uint8_t*>(a.y + c0 * a.ld_y + int64_t(h) * a.Dv + v0);
        const uint32_t yoff = uint32_t(lr) * uint32_t(2 * a.ld_y) + 2 * (16 * wave + 4 * g4);
        const bool inside = v0 + 16 * wave + 4 * g4 < a.Dv;
        if (nch > 0) {
            load_chain(0);
            wait_loads();
        }
        __syncthreads();
        if constexpr (!OUT) {
            for (int c = 0; c < nch; ++c) {
                if (c + 1 < nch) load_chain(c + 1);
                wait_loads();
                __syncthreads();
                __syncthreads();
            }
            return;
        }
        const float scale = __builtin_amdgcn_frexp_mantf(a.scale);
        u32x2 y[4];
        u32x4 low[KS + 2];  // second parts of the state and of U
        auto take = [&](int c) __attribute__((always_inline)) {
            const u32x4(*const at)[64] = reinterpret_cast<const u32x4(*)[64]>(&sm.chain[c & 1].d);
#pragma unroll
            for (int s = 0; s < KS + 2; ++s) low[s] = at[wave + kPairs * s][lane];
        };
        auto outputs = [&]() __attribute__((always_inline)) {
            // what the chain has handed over of the chunk before, which stands until the next barrier
            u32x4 sh[KS], uo[2];
#pragma unroll
            for (int s = 0; s < KS; ++s) sh[s] = sm.sh[wave][s][lane];
#pragma unroll
            for (int k = 0; k < 2; ++k) uo[k] = sm.uo[wave][k][lane];
            typedef int i32x4 __attribute__((ext_vector_type(4)));
            const i32x4 unit = *reinterpret_cast<const i32x4*>(&sm.unit[16 * wave + 4 * g4]);
            const i32x4 from = *reinterpret_cast<const i32x4*>(&sm.from[16 * wave + 4 * g4]);
            // queries 16 x + lr of columns 4 g4 + i
            f32x4 o[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) o[x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[x] = F16::mfma16(z ? low[s] : sh[s], q[x][s], o[x]);
#pragma unroll
            for (int x = 0; x < 4; ++x) o[x] *= qf[x];
#pragma unroll
            for (int z = 0; z < 3; ++z)
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int k = 0; k <= x / 2; ++k) {
                        const int at = x < 2 ? x : 2 * x - 2 + k;
                        o[x] = F16::mfma16(z == 1 ? low[KS + k] : uo[k], z == 2 ? pl[at] : ph[at], o[x]);
                    }
            bool all = true;
#pragma unroll
            for (int i = 0; i < 4; ++i) all &= from[i] >= kC;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                float z[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = __builtin_ldexpf(o[x][i] * scale, pe[x] - unit[i]);
                if (__builtin_expect(__any(!all), 0)) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[i] = 16 * x + lr >= from[i] ? __builtin_nanf("") : z[i];
                }
                y[x] = u32x2{pack16<E>(z[0], z[1]), pack16<E>(z[2], z[3])};
            }
        };
        auto store = [&](int m) __attribute__((always_inline)) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (16 * x + lr < m && inside) *reinterpret_cast<u32x2*>(yp + 32 * x * a.ld_y + yoff) = y[x];
            yp += 2 * kC * a.ld_y;
        };
        // Phase c: the chain's loads of chunk c + 1, which it waits for in the middle of chunk c; outputs of chunk c - 1;
        // loads for those of chunk c.
        for (int c = 0; c < nch; ++c) {
            take(c + 1);  // of chunk c - 1, if there is one
            if (c + 1 < nch) load_chain(c + 1);
            if (c > 0) outputs();
            load_out();
            // the chain's loads, which are older than those: 16-byte loads of one wave cannot be made fewer
            asm volatile("s_waitcnt vmcnt(%0)" :: "n"(4 * KS + 12) : "memory");
            __syncthreads();  // the next chunk is there for the chain; what it handed over is read
            if (c > 0) store(kC);
            __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0), known to the compiler: later it would wait for the chain's loads too
            __syncthreads();  // the chain is done with chunk c
        }
        if (nch > 0) {
            take(nch - 1);
            outputs();
            store(n - (nch - 1) * kC);
        }
        return;
    }

    // ---- the chain
    bool old;
    const int slot = packed_slot(a.p, u.r, &old);
    const int dv = i0 + 16 * wave + lr, width = ones ? a.Dk : a.Dv;
    const bool cin = dv < width;
    const int64_t own = (int64_t(max(slot, 0)) * a.hv + h) * a.Dk * a.Dv;
    const float* from = nullptr;  // where the columns start
    float* to = nullptr;          // and end
    if (!OUT) {
        to = ones ? a.factor(u.first + u.seg, h) : a.ends(u.first + u.seg, h);
        if (u.seg == 0 && old) from = a.sin + own;
    } else {
        if (u.nseg > 1) from = a.ends(u.first + (u.seg ? u.seg : u.nseg) - 1, h);
        else if (old) from = a.sin + own;
        if (u.seg == u.nseg - 1 && slot >= 0) to = a.sout + own;
    }
    // state element (p, b, i): dk = 32 p + 8 g4 + 4 b + i of column dv, in units of 2^-(e + lift), the values' being 2^-e
    f32x4 S[KS][2];
    int e = 0, lift = 0;
#pragma unroll
    for (int p = 0; p < KS; ++p)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int dk = 32 * p + 8 * g4 + 4 * b + i;
                S[p][b][i] = ones && dk == dv ? 1.f : 0.f;
                if (from && cin && dk < a.Dk) S[p][b][i] = from[int64_t(dk) * width + dv];
            }
    auto scale_state = [&](float by) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < KS; ++p)
#pragma unroll
            for (int b = 0; b < 2; ++b) S[p][b] *= by;
    };
    // four tokens of one column: lanes 4 i .. 4 i + 3 of 16 give the addresses of 16 columns of token i
    auto tr_read = [](const uint8_t* p) __attribute__((always_inline)) {
        return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)const_cast<uint8_t*>(p)));
    };
    // Where a lane reads K by rows (pair_row of a tile), K by columns and V: the swizzles do not depend on the tile,
    // so that tiles are constants away, or an exclusive or with a multiple of 64.
    const int krow = pair_row(lr, 0), trow = 8 * g4 + lr / 4;
    const int kat = krow * 2 * DKP + 16 * (g4 ^ kkey<DKP>(krow));
    const int tat = trow * 2 * DKP + 16 * (lr % 4 ^ kkey<DKP>(trow));
    const int vat = trow * 2 * kCols + 32 * wave + lr % 4 * 8;
    bool lost = false;  // the column has met something that is not finite
    // values (token 32 p + 8 g4 + 4 b + i of the lane's column) and keys of the next chunk to be worked on
    u32x2 vb[2][2];
    u32x4 kf[KS][2][2];
    auto read_next = [&](const ChainStage<DKP>& st) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int b = 0; b < 2; ++b) vb[p][b] = tr_read(reinterpret_cast<const uint8_t*>(st.v) + vat + (32 * p + 4 * b) * 2 * kCols);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    kf[s][p][b] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(st.k) + (kat ^ 64 * s) + (32 * p + 4 * b) * 2 * DKP);
    };
    __syncthreads();
    if (nch > 0) read_next(sm.chain[0]);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // as behind a chunk's last barrier: the compiler then knows of no read in flight
    for (int c = 0; c < nch; ++c) {
        const ChainStage<DKP>& st = sm.chain[c & 1];
        const uint8_t* const kb = reinterpret_cast<const uint8_t*>(st.k);
        int late = st.d.bad;  // first token that the column gets no number from
        const float etot = st.d.etot;
        const int next_lift = uniform(st.d.lift);
        uint32_t vtop = largest(vb);
        if (__builtin_expect(__any(vtop >= kInf16<E>), 0)) {
            // of the finite ones, and the first of the others
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int t = 32 * p + 8 * g4 + 4 * b + 2 * i;
                        uint32_t w = vb[p][b][i];
                        if ((w >> 16 & 0x7FFFu) >= kInf16<E>) late = min(late, t + 1), w &= 0xFFFFu;
                        if ((w & 0x7FFFu) >= kInf16<E>) late = min(late, t), w &= 0xFFFF0000u;
                        vb[p][b][i] = w;
                    }
            late = min(late, __shfl_xor(late, 16));
            late = min(late, __shfl_xor(late, 32));
            vtop = largest(vb);
        }
        if (__builtin_expect(next_lift != lift, 0)) {
            const bool idle = next_lift == kIdle;
            const int by = (idle ? 0 : next_lift) - lift;
            scale_state(pow2(by / 2));  // up to 2^128 in two steps
            scale_state(pow2(by - by / 2));
            lift += by;
            if (idle) {  // the values count for nothing: the unit follows the state alone
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int b = 0; b < 2; ++b) vb[p][b] = u32x2{0, 0};
                vtop = 0;
            }
        }
        // the column's unit: S and V below 2^11 in it, the larger of them from 2^5 on
        float big = 0.f;
#pragma unroll
        for (int p = 0; p < KS; ++p)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) big = fmaxf(big, fabsf(S[p][b][i]));
        const float top = lo16<E>(vtop);
        const bool any_late = __any(late < kC);
        const int none = -1000;
        int level = max(top > 0.f ? expo(top) + e : none, big > 0.f ? expo(big) : none);
        level = column_max(level);
        bool move = level >= 11 || (level < 5 && level != none);
        int aim = min(max(e + 10 - level, -120), 100);
        f32x4 U[2][2];
        u32x4 sh[KS], sl[KS], uh[2], ul[2], uo[2], uq[2];
        float unit, most;
        for (int again = 0;; ++again) {
            if (__builtin_expect(__any(move), 0)) {
                const int by = min(max(move ? aim - e : 0, -126), 126);
                scale_state(pow2(by));
                e += by;
            }
            unit = pow2(e);
            most = 0.f;
            // K S, each step's parts of S made between the steps in front of it
            auto split = [&](int s) __attribute__((always_inline)) {
                const float x[8] = {S[s][0][0], S[s][0][1], S[s][0][2], S[s][0][3], S[s][1][0], S[s][1][1], S[s][1][2], S[s][1][3]};
                sh[s] = pack_hi(x);
                sl[s] = pack_lo(x, sh[s]);
            };
            f32x4 acc[2][2], xf[2][2];
            u32x4 th[6], tl[6];
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int b = 0; b < 2; ++b) acc[p][b] = f32x4{0.f, 0.f, 0.f, 0.f};
            split(0);
            __builtin_amdgcn_sched_barrier(0);
            each([&](auto sc) __attribute__((always_inline)) {
                constexpr int s = decltype(sc)::value;
                if constexpr (s + 1 < KS) split(s + 1);
                // T is read meanwhile
#pragma unroll
                for (int i = 6 * s / KS; i < 6 * (s + 1) / KS; ++i) th[i] = st.d.th[i][lane], tl[i] = st.d.tl[i][lane];
                if constexpr (s + 1 == KS) {
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int b = 0; b < 2; ++b) xf[p][b] = *reinterpret_cast<const f32x4*>(&st.d.xf[32 * p + 8 * g4 + 4 * b]);
                }
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int b = 0; b < 2; ++b) acc[p][b] = F16::mfma16(kf[s][p][b], z ? sh[s] : sl[s], acc[p][b]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x2, 3, 0);
                    __builtin_amdgcn_sched_group_barrier(0x80, 1, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }, std::make_integer_sequence<int, KS>{});
            u32x4 rh[2], rl[2];
            auto rest = [&](int p) __attribute__((always_inline)) {  // V - e^b K S of the tokens 32 p ..
                float x[8];
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t w = uint32_t(fresh(int(vb[p][b][i])));  // or all conversions would be kept
                        x[4 * b + 2 * i] = fmaf(lo16<E>(w), unit, -xf[p][b][2 * i] * acc[p][b][2 * i]);
                        x[4 * b + 2 * i + 1] = fmaf(hi16<E>(w), unit, -xf[p][b][2 * i + 1] * acc[p][b][2 * i + 1]);
                    }
                if (__builtin_expect(any_late, 0)) {
                    const int to = fresh(late) - 32 * p - 8 * g4;  // here, not ahead of the branch
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = i >= to ? 0.f : x[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(x[i]));
                rh[p] = pack_hi(x);
                rl[p] = pack_lo(x, rh[p]);
            };
            auto updates = [&](int k, int p0, int p1) __attribute__((always_inline)) {  // T times those
#pragma unroll
                for (int z = 0; z < 3; ++z)
#pragma unroll
                    for (int p = p0; p < p1; ++p)
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const int at = p ? 2 + 2 * b + k : b;
                            U[p][b] = F16::mfma16(z == 0 ? tl[at] : th[at], z == 1 ? rl[k] : rh[k], U[p][b]);
                        }
            };
            auto scaled = [&](int p) __attribute__((always_inline)) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    U[p][b] *= *reinterpret_cast<const f32x4*>(&st.d.uf[32 * p + 8 * g4 + 4 * b]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) most = fmaxf(most, fabsf(U[p][b][i]));
                }
            };
            auto parts = [&](int p) __attribute__((always_inline)) {
                float x[8] = {U[p][0][0], U[p][0][1], U[p][0][2], U[p][0][3], U[p][1][0], U[p][1][1], U[p][1][2], U[p][1][3]};
                uo[p] = pack_hi(x);
                if constexpr (OUT) uq[p] = pack_lo(x, uo[p]);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const f32x4 tf = *reinterpret_cast<const f32x4*>(&st.d.tf[32 * p + 8 * g4 + 4 * b]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[4 * b + i] *= tf[i];
                        most = fmaxf(most, fabsf(x[4 * b + i]));
                    }
                }
                uh[p] = pack_hi(x);
                ul[p] = pack_lo(x, uh[p]);
            };
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int b = 0; b < 2; ++b) U[p][b] = f32x4{0.f, 0.f, 0.f, 0.f};
            rest(0);
            __builtin_amdgcn_sched_barrier(0);
            rest(1);
            updates(0, 0, 2);
#pragma unroll
            for (int i = 0; i < 12; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 1);
                __builtin_amdgcn_sched_group_barrier(0x2, 4, 1);
            }
            __builtin_amdgcn_sched_barrier(0);
            scaled(0);
            parts(0);
            updates(1, 1, 2);
#pragma unroll
            for (int i = 0; i < 6; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 2);
                __builtin_amdgcn_sched_group_barrier(0x2, 6, 2);
            }
            __builtin_amdgcn_sched_barrier(0);
            scaled(1);
            parts(1);
            // beyond binary16: once more in larger units
            move = most >= 32768.f && e > -120;
            if (__builtin_expect(!__any(move), 1) || again == 12) break;
            move = column_max(move);
            aim = max(e - 10, -120);
            // the keys are still there
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        kf[s][p][b] = *reinterpret_cast<const u32x4*>(kb + (kat ^ 64 * s) + (32 * p + 4 * b) * 2 * DKP);
        }
        // K^T by columns
        u32x4 kt[2 * KS * 2];
        auto read_kt = [&](int z) __attribute__((always_inline)) {
            const int k = z / (2 * KS), p = z / 2 % KS, b = z & 1;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const u32x2 w = tr_read(kb + (tat ^ 64 * p) + (32 * k + 4 * y) * 2 * DKP + 8 * b);
                kt[z][2 * y] = w[0], kt[z][2 * y + 1] = w[1];
            }
        };
#pragma unroll
        for (int z = 0; z < 2 * KS; ++z) read_kt(z);
        __syncthreads();  // the next chunk is there; the outputs' waves have taken what was handed over
        if constexpr (OUT) {
#pragma unroll
            for (int s = 0; s < KS; ++s) sm.sh[wave][s][lane] = sh[s];
#pragma unroll
            for (int k = 0; k < 2; ++k) sm.uo[wave][k][lane] = uo[k];
            // T is read; the outputs' wave loads these pieces of the next but one
            u32x4(*const to)[64] = reinterpret_cast<u32x4(*)[64]>(&sm.chain[c & 1].d);
#pragma unroll
            for (int s = 0; s < KS + 2; ++s) to[wave + kPairs * s][lane] = s < KS ? sl[s] : uq[s - KS];
            if (g4 == 0) sm.unit[16 * wave + lr] = e, sm.from[16 * wave + lr] = lost ? 0 : late;
        }
        lost |= late < kC;
        const float keep = lost ? __builtin_nanf("") : etot;
#pragma unroll
        for (int z = 2 * KS; z < 4 * KS; ++z) read_kt(z);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int z = 0; z < 2 * KS; ++z) S[z / 2][z & 1] *= keep;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k == 1) {
                __builtin_amdgcn_sched_barrier(0);
                if (c + 1 < nch) read_next(sm.chain[c + 1 & 1]);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int z = 0; z < 2 * KS; ++z)
                    S[z / 2][z & 1] = F16::mfma16(kt[2 * KS * k + z], y ? uh[k] : ul[k], S[z / 2][z & 1]);
        }
        __syncthreads();  // K is read
    }
    if (to && cin) {
#pragma unroll
        for (int p = 0; p < KS; ++p)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int dk = 32 * p + 8 * g4 + 4 * b + i;
                    if (dk < a.Dk) to[int64_t(dk) * width + dv] = __builtin_ldexpf(S[p][b][i], -e - lift);
                }
    }
}

// The states in front of a request's segments, S_{g+1} = M_g S_g + B_g, in FP32.  A workgroup owns 16 columns, a wave
// two tiles of 16 rows; a step of the products takes one row of each lane group's four, so that a result goes to
// the next product as it stands, through LDS to the other waves.   S_{g+1} takes
// the place of B_g; the place of the last segment, which has no B, gets the first state, since the second
// launch may write the request's slot before a segment would read it.  A step takes 3.3 us, of which the matrix cores
// 1: a compute unit gets 64 KB of M at some 16 bytes a cycle.  The next M but one read ahead, and the slices of
// a head on one XCD, gave 2 of 30 us.
template <int DKP>
__global__ void __launch_bounds__(32 * (DKP / 16)) k_delta_join(DeltaArgs a) {
    constexpr int NT = DKP / 16;
    __shared__ f32x4 sm[2][NT][64];  // S_g by tiles
    const int r = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int lr = lane & 15, g4 = lane >> 4;
    const int c0 = packed_row(a.p, r), n = max(0, packed_row(a.p, r + 1) - c0), nseg = (n + a.L - 1) / a.L;
    if (nseg <= 1) return;
    const int64_t first = c0 / a.L + r;
    const int dv = blockIdx.z * 16 + lr;
    bool old;
    const int slot = packed_slot(a.p, r, &old);
    f32x4 m[2][NT], B[2];
    auto rows = [&](auto&& f) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int dk = 16 * (2 * wave + t) + 4 * g4 + i;
                f(t, i, int64_t(dk) * a.Dv + dv, dv < a.Dv && dk < a.Dk);
            }
    };
    auto load = [&](int g) __attribute__((always_inline)) {
        const float *const src = a.ends(first + g, h), *const M = a.factor(first + g, h);
        rows([&](int t, int i, int64_t at, bool in) { B[t][i] = in ? src[at] : 0.f; });
        if (g == 0) return;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < NT; ++k) {
                const int row = 16 * (2 * wave + t) + lr, col = 16 * k + 4 * g4;
                m[t][k] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (row < a.Dk && col < a.Dk) m[t][k] = *reinterpret_cast<const f32x4*>(M + int64_t(row) * a.Dk + col);
            }
    };
    load(0);
    const float* const src = a.sin + (int64_t(max(slot, 0)) * a.hv + h) * a.Dk * a.Dv;
    float* const last = a.ends(first + nseg - 1, h);
    rows([&](int, int, int64_t at, bool in) { if (in) last[at] = old ? src[at] : 0.f; });
    for (int g = 0; g + 2 < nseg; ++g) {
#pragma unroll
        for (int t = 0; t < 2; ++t) sm[g & 1][2 * wave + t][lane] = B[t];
        load(g + 1);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            const f32x4 s = sm[g & 1][k][lane];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int t = 0; t < 2; ++t) B[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(m[t][k][i], s[i], B[t], 0, 0, 0);
        }
        float* const dst = a.ends(first + g + 1, h);
        rows([&](int t, int i, int64_t at, bool in) { if (in) dst[at] = B[t][i]; });
    }
}

template <class E, int DKP>
void launch(DeltaArgs a, int cus, hipStream_t s) {
    constexpr int64_t most = 8 << 20;  // a launch holds fewer than 2^32 threads
    const int64_t units = int64_t(a.p.T) / kC + a.p.R + 1, heads = a.hv / a.hk, slices = (a.Dv + kCols - 1) / kCols;
    // all value heads of a key head in one workgroup where there are enough of those
    const int per = units * a.hk >= 2 * cus ? int(heads) : 1;
    const int64_t prep = (units * a.hk + 7) / 8 * 8 * (heads / per);
    for (a.id0 = 0; a.id0 < prep; a.id0 += most)
        k_delta_prep<E, DKP><<<unsigned(std::min(most, prep - a.id0)), 256, 0, s>>>(a, per);
    // beside the recurrence: no more requests than can be long enough
    const int64_t segs = a.seg || a.few < 0 ? int64_t(a.p.T) / a.L + a.p.R + 1 : std::min<int64_t>(a.p.R, a.p.T / (a.few + 1));
    const int64_t scans = (segs * a.hv + 7) / 8 * 8;
    if (a.seg) {
        const int64_t most1 = scans * (slices + (a.Dk + kCols - 1) / kCols);
        for (a.id0 = 0; a.id0 < most1; a.id0 += most)
            k_delta_scan<E, DKP, false><<<unsigned(std::min(most, most1 - a.id0)), 128 * kPairs, 0, s>>>(a);
        k_delta_join<DKP><<<dim3(a.p.R, a.hv, (a.Dv + 15) / 16), 32 * (DKP / 16), 0, s>>>(a);
    }
    for (a.id0 = 0; a.id0 < scans * slices; a.id0 += most)
        k_delta_scan<E, DKP, true><<<unsigned(std::min(most, scans * slices - a.id0)), 128 * kPairs, 0, s>>>(a);
}

}  // namespace

template <class E>
void launch_delta_chunks(const DeltaArgs& a, int cus, hipStream_t s) {
    if (a.Dk <= 64) launch<E, 64>(a, cus, s);
    else launch<E, 128>(a, cus, s);
}
template void launch_delta_chunks<F16>(const DeltaArgs&, int, hipStream_t);
template void launch_delta_chunks<BF16>(const DeltaArgs&, int, hipStream_t);

}  // namespace vqmlp
