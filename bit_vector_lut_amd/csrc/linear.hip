// linear.hip -- linear attention with a decay per head and token (gfx950).
//
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   y_t = scale S_t^T q_t.
//
// Few tokens: the recurrence itself, state in registers (k_lin_step), bound by reading and
// writing the FP32 states.  Many: chunks of 64 tokens.  With b_t = g_1 + .. + g_t inside a chunk
// and S the state before it,
//   y_t = scale (e^{b_t} S^T q_t + sum_{j <= t} e^{b_t - b_j} (q_t . k_j) v_j)
//   S'  = e^{b_64} S + sum_j k_j (e^{b_64 - b_j} v_j)^T
// all four products on the matrix cores (k_lin_chunk).
#include "op.h"

#include <algorithm>

namespace vqmlp {

namespace {

constexpr int kC = 64;          // tokens per chunk
constexpr int kStepMaxQ = 16;
constexpr int64_t kMaxLd = 1 << 24;  // 63 tokens apart still is a 32-bit number of bytes

struct LinArgs {
    const uint16_t *q, *k, *v;
    const float* g;
    uint16_t* y;
    const float* sin;
    float* sout;
    const int32_t *cu, *ctx, *index;
    float* seg;   // [unit][v_heads] states of segments, padded and in pieces (split launches only)
    float* dec;   // [unit][v_heads] decay over a segment
    int64_t ld_q, ld_k, ld_v, ld_y, ld_g;
    int T, R, hk, hv, Dk, Dv, n_states, L;
    int id0;      // number of the launch's first workgroup
    float scale;
};

__device__ __forceinline__ int lin_row(const LinArgs& a, int r) { return min(max(a.cu[r], 0), a.T); }

// The state slot of a request, or -1, and whether it starts from what the slot holds.
__device__ __forceinline__ int lin_slot(const LinArgs& a, int r, bool* old) {
    int s = a.index ? a.index[r] : r;
    if (uint32_t(s) >= uint32_t(a.n_states)) s = -1;
    *old = s >= 0 && (!a.ctx || a.ctx[r] > 0);
    return s;
}

// ---------------------------------------------------------------- the recurrence
// A wave owns a head's Dk x 32 (or 16) columns of the state: lane = (row block, four columns), the eight
// (or sixteen) row blocks' rows contiguous so that a token's q and k come as 16-byte chunks.  The sum
// over rows is a lane's own rows, then lane swaps; no LDS and no barrier, so that a wave's loads are
// all that is in flight.
// Two tokens are on their way while one is in work (8 tokens of 48 heads of 128 x 128, 32 columns a
// wave: 10.9 us in a graph, 11.7 with four, which leave two waves a SIMD; with single tokens one is as
// good).  64 requests of one token: 88 us, 4.6 TB/s, the rate of a large copy.
template <class E, int RPL, int RB>  // rows per lane, row blocks: Dk <= RPL RB
__global__ void __launch_bounds__(64) k_lin_step(LinArgs a) {
    constexpr int CB = 64 / RB;
    const int r = blockIdx.x, h = blockIdx.y;
    const int lane = threadIdx.x, cb = lane % CB, rb = lane / CB;
    const int col = (blockIdx.z * CB + cb) * 4, row0 = rb * RPL;
    if (r == a.R) {  // rows behind the last request
        for (int64_t t = lin_row(a, a.R) + rb; t < a.T; t += RB)
            if (col < a.Dv) *reinterpret_cast<u32x2*>(a.y + t * a.ld_y + int64_t(h) * a.Dv + col) = u32x2{0, 0};
        return;
    }
    const int c0 = lin_row(a, r), n = lin_row(a, r + 1) - c0;
    bool old;
    const int slot = lin_slot(a, r, &old);
    const int64_t base = (int64_t(max(slot, 0)) * a.hv + h) * a.Dk * a.Dv;
    f32x4 s[RPL];
    const bool cin = col < a.Dv;
    const int hk = h / (a.hv / a.hk);
    constexpr int CH = RPL / 8, AHEAD = 2;
    struct Token {
        u32x4 k[CH], q[CH];
        u32x2 v;
        float g;
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
        x.v = u32x2{0, 0};
        if (cin) x.v = *reinterpret_cast<const u32x2*>(a.v + t * a.ld_v + int64_t(h) * a.Dv + col);
        x.g = a.g[t * a.ld_g + h];
    };
    auto token = [&](int t, const Token& x) __attribute__((always_inline)) {
        const f32x4 v = {lo16<E>(x.v[0]), hi16<E>(x.v[0]), lo16<E>(x.v[1]), hi16<E>(x.v[1])};
        const float e = exp_f32(bounded(x.g));
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float kk = j & 1 ? hi16<E>(x.k[c][j / 2]) : lo16<E>(x.k[c][j / 2]);
                const float qq = j & 1 ? hi16<E>(x.q[c][j / 2]) : lo16<E>(x.q[c][j / 2]);
                f32x4& z = s[8 * c + j];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    z[i] = fmaf(kk, v[i], z[i] * e);
                    acc[i] = fmaf(qq, z[i], acc[i]);
                }
            }
        // Sums over the row blocks, four columns at once: a swap of halves (then of rows of 16
        // lanes) puts the two parts of one sum side by side with those of another.
        auto pair = [](float x, float y, auto&& swap) __attribute__((always_inline)) {
            const auto z = swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y));
            const uint32_t z0 = z[0], z1 = z[1];
            return __builtin_bit_cast(float, z0) + __builtin_bit_cast(float, z1);
        };
        auto half = [](uint32_t x, uint32_t y) { return __builtin_amdgcn_permlane32_swap(x, y, false, false); };
        auto row = [](uint32_t x, uint32_t y) { return __builtin_amdgcn_permlane16_swap(x, y, false, false); };
        float sum = pair(pair(acc[0], acc[1], half), pair(acc[2], acc[3], half), row);
        sum += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, sum), 0x128, 0xF, 0xF, false));
        if constexpr (RB == 16)
            sum += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, sum), 0x124, 0xF, 0xF, false));
        // 16-lane row 0, 1, 2, 3 has column 0, 2, 1, 3 of the lane's four, RB / 4 times
        if ((lane & 15) < CB && cin)
            a.y[int64_t(t) * a.ld_y + int64_t(h) * a.Dv + col + (lane >> 4 & 1) * 2 + (lane >> 5)] =
                uint16_t(bits16<E>(sum * a.scale));
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

// ---------------------------------------------------------------- chunks on the matrix cores
// A workgroup of four waves owns one head of one segment (a.L tokens at most) and goes through its
// chunks in order; wave w owns NTV tiles of 16 value columns and the whole Dk of their state, which
// stays in matrix-core accumulators (FP32) from chunk to chunk.
//
// Orders chosen so that nothing but the token axis has to be transposed:
//   - the state product S += K^T V leaves, per lane, rows (dk) of one column (dv); the product
//     S^T Q wants, per lane, eight dk of one dv.  The two row tiles of a pair take dk 8(m/4) + m%4
//     and the same + 4, so a lane holds dk 8g .. 8g+7 and packs them where they are;
//   - K^T and V^T (token runs per column) are what both token-axis products want; each thread turns
//     an 8 x 8 block in registers on the way to LDS;
//   - the scores are made as K Q^T, 16 keys per wave, and pass through LDS once, since every wave
//     needs them all.
//
// Precision.  The state and its decays are FP32.  What joins the state is e^{..} v in FP32, handed
// to the matrix cores as a sum of parts of the 16-bit type, three for bfloat16 and two for binary16 (its 22 bits:
// off by 2^-23 of the value or 2^-39 of the column's sum, whichever is more).  The scores times their decays, and
// the state as an operand of S^T Q, are rounded once to the 16-bit type: the outputs are rounded to it as well.
// In binary16 the parts and the state of each value column share a power of two 2^e, so that columns of any sizes
// stand side by side.  It puts the sum over the chunk's tokens of e^{..} |v|, decays included, into [2^14, 2^15);
// the matrix cores make that sum, of 2^15 e^{..} in binary16 and |v| (a maximum by vector instructions took 57
// instead of 53 us for the states of three packed prompts).  The state is taken up or down where its largest
// element leaves [2^-2, 2^15).  One unit for all of a wave's columns is 3% faster, but where columns lie 2^20 apart
// it cost the smaller ones' states 12 bits.
// Binary16 scores have a power of two of their own, 2^su, which the outputs give back with their rounding: su is the
// chunk's before as long as the largest score stays in [2^5, 2^15), so that scores down to 2^-19 of it keep all
// bits; otherwise the chunk's scores are made once more (2% of the time; without a unit scores below 2^-14 lose
// bits and those beyond 65504 are infinite).
//
// Bound by the latencies of a chunk: two workgroups a compute unit (registers), each 64 x 64 scores,
// 118 matrix-core steps and about 900 vector instructions a wave and chunk, which keep the matrix cores
// busy 18% of the time, the vector unit 36%, LDS 25%.  Eight waves of 16 columns, four a SIMD, read twice
// as much LDS and took 193 us instead of 160.  Three prompts of 5003, 1021 and 2049 tokens, 48 value and
// 16 key heads of 128 x 128: 51 us for the segments' states, 106 for the outputs; 152 us back to back,
// 208 TFLOP/s of the recurrence's operations.
constexpr int kTok = kC + 8;  // LDS row stride of the scores: 144 bytes, 16-byte chunks spread over banks

// K^T and V^T in LDS: rows of 64 tokens, the eight 16-byte chunks of a row permuted by an exclusive or
// with bits 1, 3 and 2 ^ 4 of the row number.  An operand read takes one chunk number from sixteen
// rows, either m = 0 .. 15 or 8 (m / 4) + m % 4; two rows fill the 64 banks, and rows of one parity get
// eight different chunks either way.  In bytes; the permutation is linear, so a constant row or chunk
// is an exclusive or with tok_bits of it, and a multiple of 32 rows an offset.
__device__ __forceinline__ constexpr int tok_bits(int row, int chunk) {
    return 16 * (chunk ^ ((row >> 1 & 1) | (row >> 2 & 2) | ((row ^ (row >> 2)) & 4)));
}
__device__ __forceinline__ constexpr int tok_at(int row, int chunk) { return row * kC * 2 + tok_bits(row, chunk); }

struct alignas(16) LinDecay {  // of one chunk; b = sum of g up to a token
    float eb[kC];            // e^b
    float bl[kC], lo[kC];    // b log2 e and what it lost in rounding
    float tail[kC];          // e^(sum behind the token)
    uint16_t weight[kC];     // 2^15 tail in binary16 (of binary16 values)
    float etot;              // e^(sum of the chunk)
};
template <int DKP, int DVP>
struct LinSmem {
    __attribute__((aligned(256))) uint8_t kt[DKP * kC * 2];  // [dk][token], tok_at
    __attribute__((aligned(256))) uint8_t vt[DVP * kC * 2];  // [dv][token]
    LinDecay d[2];           // of this chunk and the next
    __attribute__((aligned(16))) uint32_t top[4];  // largest score of each wave's keys
    // Values that are not finite: whether a wave that stages V met one, and for its columns 64 - the first token.
    uint32_t odd[4], late[DVP];
    __attribute__((aligned(16))) float unit[DVP];  // 2^-e of a column
};
template <int DKP>
struct LinOutSmem {
    uint16_t p[kC][kTok];                        // [query][key] scores
    __attribute__((aligned(1024))) uint16_t q[kC * DKP], k[kC * DKP];  // rows of tokens, chunks permuted
};

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = lane_scan(v, 0u, [](uint32_t a, uint32_t b) { return max(a, b); });
    return uint32_t(__builtin_amdgcn_readlane(int(v), 63));
}

struct LinUnit {
    int r, c0, n, seg, nseg, first;  // request, its first row and tokens; segment; unit of segment 0
};

// Units of all requests in one launch without their lengths on the host: request r owns unit
// numbers floor(cu[r] / L) + r and on (enough for ceil(n / L), and one where n is 0).
__device__ __forceinline__ bool lin_unit(const LinArgs& a, int x, LinUnit& u) {
    const int lane = threadIdx.x & 63;
    int count = 0;
    for (int r0 = 0; r0 <= a.R; r0 += 64) {
        const int r = r0 + lane;
        count += __popcll(__ballot(r <= a.R && lin_row(a, min(r, a.R)) / a.L + r <= x));
    }
    u.r = max(0, count - 1);
    u.c0 = lin_row(a, u.r);
    const int c1 = u.r < a.R ? lin_row(a, u.r + 1) : a.T;
    u.n = max(0, c1 - u.c0);
    u.first = u.c0 / a.L + u.r;
    u.seg = x - u.first;
    u.nseg = max(1, (u.n + a.L - 1) / a.L);
    return u.seg >= 0 && u.seg < u.nseg;
}

// Workgroups a compute unit holds: three where LDS and registers allow it.  48 heads of 64 x 64, 12,000 tokens:
// 116 us with two, 98 with three.  64 x 128, 12,000 tokens: 168 and 171 in bfloat16, 177 and 185 in binary16, since
// three put 16 registers into memory.
__host__ __device__ constexpr int lin_resident(int dkp, int ntv) { return dkp == 64 && ntv == 1 ? 3 : 2; }

// OUT: outputs and the final state; otherwise the states of the segments, for a later OUT launch.
template <class E, int DKP, int NTV, bool OUT>
__global__ void __launch_bounds__(256, lin_resident(DKP, NTV)) k_lin_chunk(LinArgs a) {
    constexpr int KS = DKP / 32;       // steps over dk, pairs of state row tiles
    constexpr int DVP = 64 * NTV;
    constexpr bool HALF = __is_same(E, F16);
    constexpr int PARTS = HALF ? 2 : 3;
    __shared__ LinSmem<DKP, DVP> sm;
    __shared__ __attribute__((aligned(1024))) std::conditional_t<OUT, LinOutSmem<DKP>, char> so;
    // Workgroups go round the eight XCDs; those of the value heads that read the same queries and keys
    // are 8 apart, on one XCD, one after another.
    const int heads = a.hv / a.hk;
    const int id = a.id0 + blockIdx.x, pair = id / (8 * heads) * 8 + id % 8;  // (unit, key head)
    const int hk = pair % a.hk, h = hk * heads + id / 8 % heads;
    LinUnit u;
    if (!lin_unit(a, pair / a.hk, u)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int lr = lane & 15, g4 = lane >> 4;
    const int t0 = u.seg * a.L, t1 = min(u.n, t0 + a.L);
    if (u.r == a.R) {  // rows behind the last request
        if (OUT)
            for (int i = tid; i < (t1 - t0) * (a.Dv / 8); i += 256) {
                const int64_t t = u.c0 + t0 + i / (a.Dv / 8);
                *reinterpret_cast<u32x4*>(a.y + t * a.ld_y + int64_t(h) * a.Dv + (i % (a.Dv / 8)) * 8) =
                    u32x4{0, 0, 0, 0};
            }
        return;
    }
    if (!OUT && u.nseg == 1) return;
    bool old;
    const int slot = lin_slot(a, u.r, &old);
    const int64_t ss = int64_t(a.Dk) * a.Dv;
    const int64_t sbase = (int64_t(max(slot, 0)) * a.hv + h) * ss;
    // A segment's state: what a lane holds as 16-byte pieces, a wave's 1 KB pieces one after another.
    const uint32_t seg_off = (wave * KS * 2 * NTV * 64 + lane) * 16;
    auto seg_state = [&](int unit) {
        return reinterpret_cast<uint8_t*>(a.seg) + (int64_t(unit) * a.hv + h) * (DKP * 64 * NTV * 4);
    };

    // state element (pair p, tile b, column tile v, i): dk = 32 p + 8 g4 + 4 b + i, dv = dvc(v)
    auto dvc = [&](int v, int m) {
        return NTV == 1 ? 16 * wave + m : 32 * wave + 8 * (m >> 2) + (m & 3) + 4 * v;
    };
    f32x4 S[KS][2][NTV];
    auto each_state = [&](auto&& f) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < KS; ++p)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int v = 0; v < NTV; ++v) {
                    const int dk = 32 * p + 8 * g4 + 4 * b, dv = dvc(v, lr);
                    if (dk < a.Dk && dv < a.Dv) f(S[p][b][v], int64_t(dk) * a.Dv + dv);
                }
    };
    auto each_piece = [&](auto&& f) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < KS; ++p)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int v = 0; v < NTV; ++v) f(S[p][b][v], ((p * 2 + b) * NTV + v) * 1024);
    };
    auto store_seg = [&](int unit) __attribute__((always_inline)) {
        uint8_t* const dst = seg_state(unit);
        each_piece([&](f32x4& x, int at) { *reinterpret_cast<f32x4*>(dst + at + seg_off) = x; });
    };
    auto load_seg = [&](int unit) __attribute__((always_inline)) {
        const uint8_t* const src = seg_state(unit);
        each_piece([&](f32x4& x, int at) { x = *reinterpret_cast<const f32x4*>(src + at + seg_off); });
    };
    auto load_state = [&](const float* src) __attribute__((always_inline)) {
        each_state([&](f32x4& x, int64_t at) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = src[at + int64_t(i) * a.Dv];
        });
    };
    auto store_state = [&](float* dst) __attribute__((always_inline)) {
        each_state([&](f32x4& x, int64_t at) {
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[at + int64_t(i) * a.Dv] = x[i];
        });
    };
#pragma unroll
    for (int p = 0; p < KS; ++p)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int v = 0; v < NTV; ++v) S[p][b][v] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (!OUT) {
        // the last segment's own state is not needed before the outputs: its place keeps the
        // start state, which an in-place OUT launch could not read safely for segment 0
        if (u.seg == 0 || u.seg == u.nseg - 1) {
            if (old) load_state(a.sin + sbase);
            if (u.seg == u.nseg - 1) {
                store_seg(u.first + u.seg);
                return;
            }
        }
    } else if (u.nseg == 1) {
        if (old) load_state(a.sin + sbase);
    } else if (u.seg == 0) {
        load_seg(u.first + u.nseg - 1);
    } else {
        load_seg(u.first);
        for (int j = 1; j < u.seg; ++j) {
            const float dj = a.dec[int64_t(u.first + j) * a.hv + h];
            const uint8_t* const src = seg_state(u.first + j);
            each_piece([&](f32x4& x, int at) {
                const f32x4 z = *reinterpret_cast<const f32x4*>(src + at + seg_off);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = fmaf(x[i], dj, z[i]);
            });
        }
    }

    // Addresses: a base that the wave shares plus 32-bit offsets of the lanes.
    // staging: thread = one 8 x 8 block (tokens 8 bi .., columns 8 bj ..) of K or V; a wave has one of
    // them, eight neighbouring lanes 128 bytes of a token
    const int bi = lane >> 3, bj = 8 * wave + (lane & 7);
    const bool isk = 8 * wave < DKP / 8;
    const int cj = isk ? bj : bj - DKP / 8;
    const bool stage = isk || 8 * wave - DKP / 8 < DVP / 8;
    const bool inside = isk ? 8 * cj < a.Dk : stage && 8 * cj < a.Dv;
    const bool dense = stage && (isk ? a.Dk == DKP : a.Dv == DVP);  // all lanes of the wave load
    const int64_t ld = 2 * (isk ? a.ld_k : a.ld_v);  // bytes
    const uint8_t* const src =
        reinterpret_cast<const uint8_t*>(isk ? a.k + int64_t(hk) * a.Dk : a.v + int64_t(h) * a.Dv) + u.c0 * ld;
    const uint32_t src_off = uint32_t(8 * bi) * uint32_t(ld) + 16 * cj;
    const int kget = tok_at(8 * (lr >> 2) + (lr & 3), g4), vget = tok_at(dvc(0, lr), g4);
    const int put = tok_at(8 * cj, bi);
    u32x4 blk[8];
    // of the chunk after the one in work: g of token `lane` (wave 2), of token 63 - `lane` (wave 3)
    float gv = 0.f;
    // One of the eight loads of the chunk at token t.  A wave's loads go out one by one between its
    // matrix-core steps: eight in a row keep it from issuing anything else for over a thousand cycles.
    auto fetch = [&](int t, int i) __attribute__((always_inline)) {
        const uint8_t* const base = src + t * ld + i * ld;
        if (dense && t + kC <= t1) {
            blk[i] = *reinterpret_cast<const u32x4*>(base + src_off);
        } else {
            blk[i] = u32x4{0, 0, 0, 0};
            if (inside && t + 8 * bi + i < t1) blk[i] = *reinterpret_cast<const u32x4*>(base + src_off);
        }
    };
    auto fetch_g = [&](int t) __attribute__((always_inline)) {
        if (wave < 2) return;
        const uint8_t* const base = reinterpret_cast<const uint8_t*>(a.g + (u.c0 + t) * a.ld_g + h);
        const int i = wave == 3 ? 63 - lane : lane;
        gv = t + i < t1 ? *reinterpret_cast<const float*>(base + uint32_t(i) * uint32_t(a.ld_g) * 4) : 0.f;
    };
    // Sums from the front for e^{b}, from the back for the tails, in FP64: behind strong decays b reaches thousands,
    // and the scores take differences of neighbours (in FP32 they kept 3e-4, less than binary16 holds).
    auto decays = [&](LinDecay& d) __attribute__((always_inline)) {
        if (wave < 2) return;
        // the bound here, not where g is loaded: it would wait for the load
        const double b = lane_scan(double(bounded(gv)) * 1.4426950408889634, 0., [](double x, double y) { return x + y; });
        const float bl = float(b), lo = float(b - bl);
        const float eb = __builtin_amdgcn_exp2f(bl) * fmaf(lo, kLn2, 1.f);
        if (wave == 2) {
            d.eb[lane] = eb;
            d.bl[lane] = bl;
            d.lo[lane] = lo;
            if (lane == 63) d.etot = eb;
        } else {
            // from the back b reaches to token 63 - lane: what lies behind token 62 - lane
            const int at = lane == 63 ? 63 : 62 - lane;
            const float tail = lane == 63 ? 1.f : eb;
            d.tail[at] = tail;
            if constexpr (HALF) d.weight[at] = uint16_t(bits16<F16>(fminf(tail * 32768.f, 65504.f)));
        }
    };
    // Q rows of a chunk, token by token, straight to LDS; behind the last token the last again
    constexpr int RPI = 512 / DKP, NI = kC / RPI / 4;  // rows per load, loads per wave
    auto swz = [](int row) { return DKP == 64 ? (row >> 1) & 7 : row & 15; };
    auto stage_q = [&](int t, int j) __attribute__((always_inline)) {  // load j of NI
        if constexpr (OUT) {
            const uint32_t ql = lds_byte(so.q) + (wave * NI + j) * 1024;
            const uint8_t* const q = reinterpret_cast<const uint8_t*>(a.q + (u.c0 + t) * a.ld_q + int64_t(hk) * a.Dk);
            const uint32_t lq = uint32_t(a.ld_q) * 2;
            const int r0 = lane / (DKP / 8);
            const int first = (wave * NI + j) * RPI;  // a multiple of RPI: its low bits are j's
            int chunk = (lane % (DKP / 8)) ^ swz(r0) ^ swz(j * RPI);
            if (8 * chunk >= a.Dk) chunk = 0;  // meets zeros of K
            if (t + kC <= t1) {
                load_lds16(q + int64_t(first) * lq, r0 * lq + 16 * chunk, ql);
            } else {
                const int r = min(first + r0, t1 - 1 - t);
                load_lds16(q, r * lq + 16 * chunk, ql);
            }
        }
    };
    // 8 chunk columns 32 s + 8 g4 of token row r
    auto qk_read = [&](const uint16_t* p, int r, int s) {
        return *reinterpret_cast<const u32x4*>(p + r * DKP + 8 * ((4 * s + g4) ^ swz(r)));
    };
    const bool last = uniform(u.seg == u.nseg - 1 && slot >= 0);  // has the request's final state to write
    float decay = 1.f;  // over the segment so far (!OUT)
    int e[NTV] = {};    // a lane's columns of S are kept in units of 2^-e
    if constexpr (HALF && OUT) {  // no other wave reads its columns
#pragma unroll
        for (int v = 0; v < NTV; ++v) sm.unit[dvc(v, lr)] = 1.f;
    }
    auto scale_state = [&](const float* by) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < KS; ++p)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int v = 0; v < NTV; ++v) S[p][b][v] *= by[v];
    };
    // Scores are kept in units of 2^-su (binary16), the same in all waves: first those of queries and keys
    // of length one, then the chunk's before.
    auto clip = [](int x) { return min(max(x, -60), 60); };
    int su = HALF ? clip(11 - expo(a.scale)) : 0;
    // This wave's 16 keys with queries 16 x .., times their decays; the lane's largest so far.
    auto scores = [&](const LinDecay& dc, int x, const u32x4* kf, const u32x4* qf, float unit, float& top) __attribute__((always_inline)) {
        if constexpr (OUT) {
            if (x < (wave & 2)) return;
            float p[4] = {0.f, 0.f, 0.f, 0.f};  // keys behind the queries' block
            if (x >= wave) {
                f32x4 sc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < KS; ++s) sc = E::mfma16(kf[s], qf[s], sc);
                const float bt = dc.bl[16 * x + lr], one = unit * fmaf(dc.lo[16 * x + lr], kLn2, 1.f);
                const f32x4 bj = *reinterpret_cast<const f32x4*>(&dc.bl[16 * wave + 4 * g4]);
                const f32x4 lj = *reinterpret_cast<const f32x4*>(&dc.lo[16 * wave + 4 * g4]);
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = sc[i] * one * __builtin_amdgcn_exp2f((bt - bj[i]) - lj[i]);
                if (x == wave) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = 4 * g4 + i <= lr ? p[i] : 0.f;
                }
                if constexpr (HALF) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(p[i]));
                }
            }
            *reinterpret_cast<u32x2*>(&so.p[16 * x + lr][16 * wave + 4 * g4]) =
                u32x2{pack16<E>(p[0], p[1]), pack16<E>(p[2], p[3])};
        }
    };
    if (t0 < t1) {
        fetch_g(t0);
#pragma unroll
        for (int i = 0; i < 8; ++i) fetch(t0, i);
#pragma unroll
        for (int j = 0; j < NI; ++j) stage_q(t0, j);
        decays(sm.d[0]);
        fetch_g(t0 + kC);
    }
    // A value that is not finite would reach its block's tokens before it, as zero times itself.  Where outputs
    // are made it is taken out of LDS, and its column gets no number from its token on.  Zero times all values
    // finds one: 32 vector instructions of the waves that stage V, which have fewer scores to make than wave 0.
    auto take_out = [&]() __attribute__((always_inline)) {
        float z[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j & 1] = E::dot2(blk[i][j], 0u, z[j & 1]);
        const bool odd = __any(!(z[0] + z[1] == 0.f));
        if (lane == 0) sm.odd[wave] = odd;
        if (__builtin_expect(!odd, 1)) return;
        constexpr uint32_t top = HALF ? 0x7C00u : 0x7F80u;
#pragma unroll 1
        for (int cc = 0; cc < 8; ++cc) {  // the lane's eight tokens of a column
            u32x4* const at = reinterpret_cast<u32x4*>(&sm.vt[(put ^ tok_bits(cc, 0)) + cc * kC * 2]);
            u32x4 w = *at;
            int late = 0;
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                if ((w[i] >> 16 & 0x7FFFu) >= top) w[i] &= 0xFFFFu, late = 63 - (8 * bi + 2 * i);
                if ((w[i] & 0x7FFFu) >= top) w[i] &= 0xFFFF0000u, late = 64 - (8 * bi + 2 * i);
            }
            *at = w;
#pragma unroll
            for (int by = 8; by < 64; by *= 2) late = max(late, __shfl_xor(late, by));
            if (bi == 0) sm.late[8 * cj + cc] = uint32_t(late);
        }
    };
    const int vwave = DKP / 64 + (NTV == 2 ? wave / 2 : 0);  // that stages the columns of this wave
    for (int t = t0; t < t1; t += kC) {
        const LinDecay& dc = sm.d[(t - t0) / kC & 1];
        if (stage) {
#pragma unroll
            for (int cc = 0; cc < 8; ++cc) {
                const uint32_t sel = cc & 1 ? 0x07060302u : 0x05040100u;
                u32x4 w;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = __builtin_amdgcn_perm(blk[2 * i + 1][cc / 2], blk[2 * i][cc / 2], sel);
                *reinterpret_cast<u32x4*>(&(isk ? sm.kt : sm.vt)[(put ^ tok_bits(cc, 0)) + cc * kC * 2]) = w;
            }
            if constexpr (OUT) {
                if (isk) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<u32x4*>(so.k + (8 * bi + i) * DKP + 8 * (cj ^ swz(8 * bi + i))) = blk[i];
                }
            }
        }
        wait_loads();  // this wave's part of Q is in LDS
        __syncthreads();
        if (OUT && stage && !isk) take_out();  // V is read behind the next barrier
        f32x4 o[NTV][4];
        int odd = 0;
        u32x4 vf[NTV][2];
        auto read_v = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int v = 0; v < NTV; ++v)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    vf[v][c] = *reinterpret_cast<const u32x4*>(&sm.vt[(vget ^ tok_bits(4 * v, 4 * c)) + 4 * v * kC * 2]);
        };
        if constexpr (OUT) {
            u32x4 qf[4][KS], kf[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                kf[s] = qk_read(so.k, 16 * wave + lr, s);
#pragma unroll
                for (int x = 0; x < 4; ++x) qf[x][s] = qk_read(so.q, 16 * x + lr, s);
            }
            __builtin_amdgcn_sched_barrier(0);  // all reads on their way before the first product waits
            const float unit = a.scale * pow2(su);
            float top = 0.f;
#pragma unroll
            for (int x = 0; x < 4; ++x) scores(dc, x, kf, qf[x], unit, top);
            if constexpr (HALF) {
                // an infinite score is no measure of the others; of values that are not negative, the bits are
                // in the values' order
                const uint32_t w = wave_max(__builtin_bit_cast(uint32_t, top < __builtin_inff() ? top : 0.f));
                if (lane == 0) sm.top[wave] = w;
            }
            // the next chunk's decays, by the waves with the fewest scores
            decays(sm.d[((t - t0) / kC + 1) & 1]);
            fetch_g(t + 2 * kC);
            // e^{b} S^T Q
            if constexpr (HALF) {
                float mx[NTV], up[NTV];
                bool out = false;
#pragma unroll
                for (int v = 0; v < NTV; ++v) {
                    mx[v] = 0.f;
#pragma unroll
                    for (int p = 0; p < KS; ++p)
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int i = 0; i < 4; ++i) mx[v] = fmaxf(mx[v], fabsf(S[p][b][v][i]));
                    out |= mx[v] >= 32768.f || (mx[v] < 0.25f && mx[v] > 0.f);
                }
                // outside the range in which binary16 holds all that matters of a column: other units
                if (__builtin_expect(__any(out), 0)) {
#pragma unroll
                    for (int v = 0; v < NTV; ++v) {
                        mx[v] = column_max(mx[v]);
                        const bool mine = mx[v] >= 32768.f || (mx[v] < 0.25f && mx[v] > 0.f);
                        const int f = mine ? min(max(min(max(10 - expo(mx[v]), -100 - e[v]), 100 - e[v]), -126), 126) : 0;
                        up[v] = pow2(f);
                        e[v] += f;
                        sm.unit[dvc(v, lr)] = pow2(-e[v]);
                    }
                    scale_state(up);
                }
            }
#pragma unroll
            for (int v = 0; v < NTV; ++v)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[v][x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int p = 0; p < KS; ++p)
#pragma unroll
                for (int v = 0; v < NTV; ++v) {
                    const f32x4 s0 = S[p][0][v], s1 = S[p][1][v];
                    const u32x4 sf = {pack16<E>(s0[0], s0[1]), pack16<E>(s0[2], s0[3]),
                                      pack16<E>(s1[0], s1[1]), pack16<E>(s1[2], s1[3])};
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[v][x] = E::mfma16(sf, qf[x][p], o[v][x]);
                    constexpr int N = 8 / (KS * NTV);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < N; ++i) fetch(t + kC, (p * NTV + v) * N + i);
                    __builtin_amdgcn_sched_barrier(0);
                }
            float eb[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) eb[x] = dc.eb[16 * x + lr] * unit;
#pragma unroll
            for (int v = 0; v < NTV; ++v) {
                if constexpr (HALF) {
                    // of the columns whose outputs the lane holds
                    const f32x4 down = *reinterpret_cast<const f32x4*>(&sm.unit[dvc(v, 4 * g4)]);
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[v][x] *= down * eb[x];
                } else {
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[v][x] *= eb[x];
                }
            }
            __syncthreads();
            // every wave is done with this chunk's queries and keys
            const u32x4 w = *reinterpret_cast<const u32x4*>(sm.top);
            const uint32_t found = sm.odd[vwave];
            read_v();
            __builtin_amdgcn_sched_barrier(0);  // all on their way before the first is waited for
            odd = uniform(int(found));
            if constexpr (HALF) {
                // The largest score has to lie where binary16 holds it and those 2^-15 of it with all bits: else
                // once more, in units that put it into [2^10, 2^11).
                const float mx = __builtin_bit_cast(float, uniform(int(max(max(w[0], w[1]), max(w[2], w[3])))));
                const int to = clip(su + 10 - expo(mx));
                if (__builtin_expect((mx >= 32768.f || (mx < 32.f && mx > 0.f)) && to != su, 0)) {
                    const float by = pow2(to - su);
#pragma unroll
                    for (int v = 0; v < NTV; ++v)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[v][x] *= by;
                    su = to;
                    u32x4 qf[KS], kf[KS];
#pragma unroll
                    for (int s = 0; s < KS; ++s) kf[s] = qk_read(so.k, 16 * wave + lr, s);
                    float top = 0.f;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
#pragma unroll
                        for (int s = 0; s < KS; ++s) qf[s] = qk_read(so.q, 16 * x + lr, s);
                        scores(dc, x, kf, qf, a.scale * pow2(su), top);
                        __builtin_amdgcn_sched_barrier(0);  // few registers: S, o and the next chunk's loads stay
                    }
                    __syncthreads();
                }
            }
        }
        if constexpr (!OUT) read_v();
        // sum over the tokens of e^{..} |v| of the lane's columns, times 2^15
        f32x4 sum[NTV];
        if constexpr (HALF) {
#pragma unroll
            for (int v = 0; v < NTV; ++v) sum[v] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const u32x4 w = *reinterpret_cast<const u32x4*>(&dc.weight[32 * c + 8 * g4]);
#pragma unroll
                for (int v = 0; v < NTV; ++v) sum[v] = E::mfma16(w, vf[v][c] & 0x7FFF7FFFu, sum[v]);
            }
        }
        int en[NTV];
        auto new_units = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int v = 0; v < NTV; ++v) {
                // bounds: states of up to 2^97 stay finite, parts keep what is above 2^-55
                const float z = sum[v][0];
                en[v] = z > 0.f ? min(max(14 + 15 - expo(z), max(e[v] - 126, -100)), min(e[v] + 126, 30)) : e[v];
            }
        };
        if (HALF && !OUT) new_units();
        if constexpr (OUT) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if (HALF && x == 1) new_units();
                if (x < NI && t + kC < t1) stage_q(t + kC, x);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int c = 0; c <= x / 2; ++c) {
                    const u32x4 pf = *reinterpret_cast<const u32x4*>(&so.p[16 * x + lr][32 * c + 8 * g4]);
#pragma unroll
                    for (int v = 0; v < NTV; ++v) o[v][x] = E::mfma16(vf[v][c], pf, o[v][x]);
                }
            }
            if (__builtin_expect(odd, 0)) {
#pragma unroll
                for (int v = 0; v < NTV; ++v)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int from = 64 - int(sm.late[dvc(v, 4 * g4 + i)]);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            o[v][x][i] = 16 * x + lr >= from ? __builtin_nanf("") : o[v][x][i];
                    }
            }
            const float by = pow2(-su);  // one rounding of the product
            auto out16 = [&](const f32x4& z, int i) __attribute__((always_inline)) {
                if constexpr (HALF) return pack16<E>(fmaf(z[i], by, -0.f), fmaf(z[i + 1], by, -0.f));
                else return pack16<E>(z[i], z[i + 1]);
            };
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if (t + 16 * x + lr >= t1) continue;
                uint8_t* const dst = reinterpret_cast<uint8_t*>(a.y + (u.c0 + t + 16 * x) * a.ld_y + int64_t(h) * a.Dv);
                const uint32_t off = uint32_t(lr) * uint32_t(a.ld_y) * 2;
                if constexpr (NTV == 2) {
                    const int dv = 32 * wave + 8 * g4;
                    const u32x4 w = {out16(o[0][x], 0), out16(o[0][x], 2), out16(o[NTV - 1][x], 0), out16(o[NTV - 1][x], 2)};
                    if (dv < a.Dv) *reinterpret_cast<u32x4*>(dst + (off + 2 * dv)) = w;
                } else {
                    const int dv = 16 * wave + 4 * g4;
                    const u32x2 w = {out16(o[0][x], 0), out16(o[0][x], 2)};
                    if (dv < a.Dv) *reinterpret_cast<u32x2*>(dst + (off + 2 * dv)) = w;
                }
            }
        }
        // the state after the chunk, which nobody needs behind a segment's last unless it is the request's
        if (OUT && t + kC >= t1 && !last) continue;
        // What joins it: e^{..} v, in units that put a column's sum of magnitudes into [2^14, 2^15).
        auto tail = [&](int c, float* w) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f32x4 z = *reinterpret_cast<const f32x4*>(&dc.tail[32 * c + 8 * g4 + 4 * j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) w[4 * j + i] = z[i];
            }
        };
        float lift[NTV], keep[NTV];
#pragma unroll
        for (int v = 0; v < NTV; ++v) {
            lift[v] = 1.f;
            keep[v] = dc.etot;
            if (__builtin_expect(odd, 0)) keep[v] = sm.late[dvc(v, lr)] ? __builtin_nanf("") : keep[v];
        }
        if constexpr (HALF) {
#pragma unroll
            for (int v = 0; v < NTV; ++v) {
                lift[v] = pow2(en[v]);
                keep[v] *= pow2(en[v] - e[v]);
                e[v] = en[v];
                if (OUT) sm.unit[dvc(v, lr)] = pow2(-en[v]);
            }
        }
        decay *= dc.etot;
        scale_state(keep);
        // K^T operands are read two steps (of four products and more) ahead; the parts of the second 32
        // tokens are made between the products of the first
        u32x4 part[2][NTV][PARTS], kk[2][2];
        auto parts = [&](int c, int v) __attribute__((always_inline)) {
            float x[8];
            tail(c, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = fmaf(lo16<E>(vf[v][c][i]), x[2 * i] * lift[v], 0.f);
                x[2 * i + 1] = fmaf(hi16<E>(vf[v][c][i]), x[2 * i + 1] * lift[v], 0.f);
            }
#pragma unroll
            for (int q = 0; q < PARTS; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w = pack16<E>(x[2 * i], x[2 * i + 1]);
                    // one rounded value for the operand and for what is left of x: otherwise
                    // the compiler rounds x twice, once fused with its product, and the two
                    // may differ by a step
                    asm("" : "+v"(w));
                    part[c][v][q][i] = w;
                    if (q + 1 < PARTS) {
                        x[2 * i] = fmaf(lo16<E>(w), -1.f, x[2 * i]);
                        x[2 * i + 1] = fmaf(hi16<E>(w), -1.f, x[2 * i + 1]);
                    }
                }
        };
        constexpr int STEPS = 4 * KS;  // (c, p, b)
        auto k_read = [&](int z) {
            const int c = z / (2 * KS), p = z / 2 % KS, b = z & 1;
            return *reinterpret_cast<const u32x4*>(
                &sm.kt[(kget ^ tok_bits(4 * b, 4 * c)) + (32 * p + 4 * b) * kC * 2]);
        };
#pragma unroll
        for (int y = 0; y < 2; ++y) kk[0][y] = k_read(y);
#pragma unroll
        for (int v = 0; v < NTV; ++v) parts(0, v);
        each([&](auto zc) __attribute__((always_inline)) {
            constexpr int z = decltype(zc)::value;
            constexpr int c = z / (2 * KS), p = z / 2 % KS, b = z & 1;
            if constexpr (z % 2 == 0 && z + 2 < STEPS) {
#pragma unroll
                for (int y = 0; y < 2; ++y) kk[(z / 2 + 1) & 1][y] = k_read(z + 2 + y);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int q = PARTS - 1; q >= 0; --q)
#pragma unroll
                for (int v = 0; v < NTV; ++v)
                    S[p][b][v] = E::mfma16(kk[z / 2 & 1][z & 1], part[c][v][q], S[p][b][v]);
            if constexpr (z < 2 * KS && z % KS == 0 && z / KS < NTV) parts(1, z / KS);
            // Behind products, which hide the lane moves' waits, and before this chunk's first load: which of
            // those were made the compiler does not know, so behind them it would wait for all.
            if constexpr (!OUT && z == 0) {
                decays(sm.d[((t - t0) / kC + 1) & 1]);
                fetch_g(t + 2 * kC);
            }
            if constexpr (!OUT && z < 8) {
                __builtin_amdgcn_sched_barrier(0);
                fetch(t + kC, z);
            }
        }, std::make_integer_sequence<int, STEPS>{});
        __syncthreads();
    }
    // no load to LDS is in flight here: each was waited for in the chunk that it was made for
    if (HALF && (!OUT || last)) {
        float by[NTV];
#pragma unroll
        for (int v = 0; v < NTV; ++v) by[v] = pow2(-e[v]);
        scale_state(by);
    }
    if (!OUT) {
        store_seg(u.first + u.seg);
        if (tid == 0) a.dec[int64_t(u.first + u.seg) * a.hv + h] = decay;
    } else if (last) {
        store_state(a.sout + sbase);
    }
}

// ---------------------------------------------------------------- host half

struct LinGeom {
    bool step, narrow;  // recurrence; of it, 16 columns a wave
    int L, units;  // tokens per segment (the whole request when not split), unit numbers
    bool split;
    size_t dec, bytes;
};

LinGeom lin_geom(const vqmlp_linear_desc& d, int cus) {
    LinGeom G{};
    G.step = d.max_q <= kStepMaxQ;
    if (G.step) {
        // Half the columns and rows a lane where waves of 32 columns are fewer than the chip's SIMDs: one
        // request of 8 tokens, 48 heads of 128 x 128: 11.0 -> 9.5 us in a graph, of 16: 16.7 -> 13.0, four of
        // one: 8.0 -> 7.5; beyond, half lines of the state cost more: 16 of one 18.8 -> 21.2, 64: 88 -> 126.
        G.narrow = d.Dk > 64 && int64_t(d.R) * d.v_heads * ((d.Dv + 31) / 32) <= 4 * int64_t(cus);
        return G;
    }
    // Segments of a request go through at once, at the price of a pass for their states first (0.6 of
    // the time of the outputs' pass), of three chunks' worth of time to start and end each, and of 0.13
    // for each earlier segment whose state an output segment takes in.  The unit is a chunk in a round
    // that fills every compute unit; one workgroup alone on a unit gets through it in 3/4 of the time of
    // two together.  8,000 tokens of heads of 128 x 128, 48 heads: 159 us with the 13 chunks that this
    // chooses, 172 / 188 / 173 / 187 with 8 / 10 / 15 / 18; 4 heads: 56 with 4, 61 / 69 / 89 with 6 / 8 / 12.
    const int most = std::max(1, std::min(d.max_q, std::max(1, d.T)));
    const int chunks = (most + kC - 1) / kC, held = lin_resident(d.Dk <= 64 ? 64 : 128, d.Dv <= 64 ? 1 : 2);
    const int64_t slots = held * int64_t(cus);
    auto rounds = [&](int64_t units) {
        const int64_t n = units * d.v_heads, rest = n % slots, per = (5 * rest + 4 * cus - 1) / (4 * cus);
        return double(n / slots) + (rest ? 0.5 + 0.5 * double(std::min<int64_t>(per, held)) / held : 0.0);
    };
    // not split: a segment holds all T tokens, so any request fits, whatever max_q says
    G.L = std::max(1, (d.T + kC - 1) / kC) * kC;
    double best = rounds(d.R) * (chunks + 3);
    const bool even = d.T == int64_t(d.R) * most;  // all requests are as long as the longest
    for (int n = 4; n < chunks; ++n) {
        const int64_t units = even ? int64_t(d.R) * ((chunks + n - 1) / n) : d.T / (n * kC) + d.R / 2;
        const double cost = rounds(std::max<int64_t>(units, d.R)) * (1.6 * n + 6 + 0.13 * ((chunks - 1) / n));
        if (cost < best) best = cost, G.split = true, G.L = n * kC;
    }
    G.units = d.T / G.L + d.R + 1;
    if (G.split) {
        G.dec = align256(size_t(G.units) * d.v_heads * (d.Dk <= 64 ? 64 : 128) * (d.Dv <= 64 ? 64 : 128) * 4);
        G.bytes = G.dec + align256(size_t(G.units) * d.v_heads * 4);
    }
    return G;
}

vqmlp_status lin_check(const vqmlp_linear_desc* p, const char* who) {
    OP_REQUIRE(p, "%s: null description", who);
    const vqmlp_linear_desc& d = *p;
    OP_REQUIRE(op_dtype16(d.dtype), "%s: dtype %d is not F16 or BF16", who, d.dtype);
    OP_REQUIRE(d.T >= 0 && d.R >= 1 && d.k_heads >= 1 && d.v_heads >= 1 && d.n_states >= 0 && d.max_q >= 0,
               "%s: a size is out of range", who);
    OP_REQUIRE(d.v_heads % d.k_heads == 0, "%s: v_heads=%d is no multiple of k_heads=%d", who, d.v_heads,
               d.k_heads);
    OP_REQUIRE(d.Dk >= 8 && d.Dk <= 128 && d.Dk % 8 == 0 && d.Dv >= 8 && d.Dv <= 128 && d.Dv % 8 == 0,
               "%s: Dk=%d, Dv=%d are not multiples of 8 up to 128", who, d.Dk, d.Dv);
    if (d.R > 65535 || d.v_heads > 65535 || d.T > 0x3FFFFFFF)
        OP_FAIL(VQMLP_ERR_UNSUPPORTED, "%s: R or v_heads above 65535, or T above 2^30 - 1", who);
    // workgroup numbers are 32-bit (segments have four chunks or more; rounded up to whole rounds of XCDs)
    if ((int64_t(d.T) / (4 * kC) + d.R + 1 + 8) * d.v_heads > 0x7FFFFFFF)
        OP_FAIL(VQMLP_ERR_UNSUPPORTED, "%s: (T / 256 + R + 9) * v_heads above 2^31 - 1", who);
    OP_REQUIRE(d.scale == d.scale && d.scale - d.scale == 0.f, "%s: scale is not finite", who);
    return VQMLP_OK;
}

template <class E>
void launch_step(const LinArgs& a, bool narrow, hipStream_t s) {
    const dim3 grid(a.R + 1, a.hv, (a.Dv + 31) / 32);
    if (a.Dk <= 64) k_lin_step<E, 8, 8><<<grid, 64, 0, s>>>(a);
    else if (narrow) k_lin_step<E, 8, 16><<<dim3(a.R + 1, a.hv, (a.Dv + 15) / 16), 64, 0, s>>>(a);
    else k_lin_step<E, 16, 8><<<grid, 64, 0, s>>>(a);
}

template <class E, bool OUT>
void launch_chunk(LinArgs a, int units, hipStream_t s) {
    const int64_t all = (int64_t(units) * a.hk + 7) / 8 * 8 * (a.hv / a.hk), most = 8 << 20;
    for (int64_t at = 0; at < all; at += most) {  // a launch holds fewer than 2^32 threads
        const unsigned grid = unsigned(std::min(most, all - at));
        a.id0 = int(at);
        if (a.Dk <= 64) {
            if (a.Dv <= 64) k_lin_chunk<E, 64, 1, OUT><<<grid, 256, 0, s>>>(a);
            else k_lin_chunk<E, 64, 2, OUT><<<grid, 256, 0, s>>>(a);
        } else {
            if (a.Dv <= 64) k_lin_chunk<E, 128, 1, OUT><<<grid, 256, 0, s>>>(a);
            else k_lin_chunk<E, 128, 2, OUT><<<grid, 256, 0, s>>>(a);
        }
    }
}

template <class E>
void launch_linear(const LinArgs& a, const LinGeom& G, hipStream_t s) {
    if (G.step) return launch_step<E>(a, G.narrow, s);
    if (G.split) launch_chunk<E, false>(a, G.units, s);
    launch_chunk<E, true>(a, G.units, s);
}

}  // namespace

}  // namespace vqmlp

extern "C" vqmlp_status vqmlp_linear_attn_workspace(const vqmlp_linear_desc* p, size_t* bytes) {
    using namespace vqmlp;
    OP_REQUIRE(bytes, "vqmlp_linear_attn_workspace: null pointer");
    int cus = 0;
    if (const vqmlp_status st = lin_check(p, "vqmlp_linear_attn_workspace")) return st;
    if (const int st = device_cus(&cus)) return static_cast<vqmlp_status>(st);
    *bytes = lin_geom(*p, cus).bytes;
    return op_ok();
}

extern "C" vqmlp_status vqmlp_linear_attn(const vqmlp_linear_desc* p, void* workspace,
                                          size_t workspace_bytes, void* stream) {
    using namespace vqmlp;
    int cus = 0;
    if (const vqmlp_status st = lin_check(p, "vqmlp_linear_attn")) return st;
    const vqmlp_linear_desc& d = *p;
    OP_REQUIRE(d.cu_q && op_aligned(d.cu_q, 4) && op_aligned(d.ctx_len, 4) && op_aligned(d.state_index, 4),
               "vqmlp_linear_attn: null cu_q or an unaligned index array");
    OP_REQUIRE((d.state_in && d.state_out) || d.n_states == 0, "vqmlp_linear_attn: null state");
    OP_REQUIRE(op_aligned(d.state_in, 16) && op_aligned(d.state_out, 16),
               "vqmlp_linear_attn: states have to be 16-byte aligned");
    if (d.T > 0) {
        OP_REQUIRE(d.q && d.k && d.v && d.g && d.y, "vqmlp_linear_attn: null pointer");
        OP_REQUIRE(op_aligned(d.q, 16) && op_aligned(d.k, 16) && op_aligned(d.v, 16) && op_aligned(d.y, 16) &&
                       op_aligned(d.g, 4),
                   "vqmlp_linear_attn: q, k, v and y have to be 16-byte aligned, g 4-byte");
        const int64_t rows[] = {int64_t(d.k_heads) * d.Dk, int64_t(d.k_heads) * d.Dk,
                                int64_t(d.v_heads) * d.Dv, int64_t(d.v_heads) * d.Dv, d.v_heads};
        const int64_t lds[] = {d.ld_q, d.ld_k, d.ld_v, d.ld_y, d.ld_g};
        for (int i = 0; i < 5; ++i)
            OP_REQUIRE((d.T == 1 || lds[i] >= rows[i]) && lds[i] >= 0 && lds[i] <= kMaxLd &&
                           (i == 4 || lds[i] % 8 == 0),
                       "vqmlp_linear_attn: token strides have to cover the heads and be at most 2^24, those of q, k, "
                       "v and y be multiples of 8");
    }
    if (const int st = device_cus(&cus)) return static_cast<vqmlp_status>(st);
    const LinGeom G = lin_geom(d, cus);
    if (G.bytes) {
        OP_REQUIRE(workspace && op_aligned(workspace, 256),
                   "vqmlp_linear_attn: the workspace is null or not 256-byte aligned");
        if (workspace_bytes < G.bytes)
            OP_FAIL(VQMLP_ERR_WORKSPACE, "vqmlp_linear_attn: workspace holds %zu bytes, this call needs %zu",
                    workspace_bytes, G.bytes);
    }
    LinArgs a;
    a.q = static_cast<const uint16_t*>(d.q);
    a.k = static_cast<const uint16_t*>(d.k);
    a.v = static_cast<const uint16_t*>(d.v);
    a.g = d.g;
    a.y = static_cast<uint16_t*>(d.y);
    a.sin = d.state_in;
    a.sout = d.state_out;
    a.cu = d.cu_q;
    a.ctx = d.ctx_len;
    a.index = d.state_index;
    a.seg = static_cast<float*>(workspace);
    a.dec = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + G.dec);
    a.ld_q = d.ld_q;
    a.ld_k = d.ld_k;
    a.ld_v = d.ld_v;
    a.ld_y = d.ld_y;
    a.ld_g = d.ld_g;
    a.T = d.T;
    a.R = d.R;
    a.hk = d.k_heads;
    a.hv = d.v_heads;
    a.Dk = d.Dk;
    a.Dv = d.Dv;
    a.n_states = d.n_states;
    a.L = G.L;
    a.scale = d.scale;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (d.dtype == VQMLP_F16) launch_linear<F16>(a, G, s);
    else launch_linear<BF16>(a, G, s);
    if (trace_enabled()) {
        if (G.step)
            trace_line("linear_attn T=%d R=%d heads=%d/%d: recurrence", d.T, d.R, d.v_heads, d.k_heads);
        else
            trace_line("linear_attn T=%d R=%d heads=%d/%d: %schunks, segments of %d tokens", d.T, d.R,
                       d.v_heads, d.k_heads, G.split ? "segment states, then " : "", G.L);
    }
    return op_launched("vqmlp_linear_attn");
}
