// attn_tile.hip -- paged attention with the keys in LDS: anything but up to 16 rows of D > 128 (gfx950).
//
// The mathematics, the packing of rows and the transposed products are those of attn.hip; here four
// waves share a tile of 64 keys in LDS and each has 32 rows of its own, 32x32x16 matrix-core steps.
// Every tile goes straight from the cache to LDS, one ahead (keys two ahead), and while the matrix
// cores make the scores of tile i + 1, the vector unit makes the exponentials of tile i.
//
// 128 rows a workgroup and two workgroups a compute unit (one for D > 128): 64 rows a wave would
// halve the LDS reads, but leave one wave a SIMD and its scores in registers that the vector unit
// cannot read (630 against 788 TFLOP/s).  512 rows over 33,001 keys, 40/8 heads of 128, FP16: 376 to
// 425 us with the join on different cards, 808 to 912 TFLOP/s, 74 to 83% of a large library product; bound by the clock that
// the power leaves (1.8 GHz of 2.4) and by exponentials beside the matrix cores, which are busy 45% of the
// time.  64 requests of one token and up to 16,252 keys, BF16: 391 us, 5.5 TB/s, bound by the cache.
#include "attn.h"

namespace vqmlp {

namespace {

constexpr int kKT = 64;   // keys of a tile

// Places for the splits of a row tile: with several requests an odd number, so that the splits that have
// keys in every request do not all meet on the same engines as workgroups go round them (four prompts of
// 37 to 1,000 rows: 197 us with four places, 98 with three).  A single request fills all of its splits.
__host__ __device__ inline int split_slots(int nsplit, int requests) { return requests == 1 ? nsplit : nsplit | 1; }

// DP: a row of keys in LDS, DM: the part of it that the products take in (D <= DM).  FEW: few rows a request,
// so that the time goes into reading keys and values.
template <class E, int DP, int DM, bool FULL, bool FEW>
__global__ void __launch_bounds__(256, DP > 128 ? 1 : 2) k_attn_tile(AttnArgs a) {
    constexpr int KS = DM / 16, DB = DM / 32, NI = DP / 32, NV = DM / 32;  // loads of K and V a wave and tile
    constexpr int RPI = 512 / DP;        // key rows per load instruction
    constexpr int TILE = kKT * DP * 2;   // bytes
    __shared__ __attribute__((aligned(1024))) uint8_t kbuf[2 * TILE];
    __shared__ __attribute__((aligned(1024))) uint8_t vbuf[2 * TILE];
    // The last tiles of a prompt, which see the most keys, come first; but one tile of one request stands in
    // front of those that turn out to be empty, so that each of its splits finds a compute unit of its own.
    const int groups = a.kv_heads * split_slots(a.nsplit, a.R), gi = blockIdx.x % groups;
    const bool single = a.R == 1 && a.T * a.g <= kAttnTileRows;
    const int x = (single ? blockIdx.x : gridDim.x - 1 - blockIdx.x) / groups;
    const int hk = gi % a.kv_heads, split = gi / a.kv_heads;
    Tile t;
    if (!find_tile<kAttnTileRows>(a, x, t)) return;
    const Split ks = key_split(a, t, split, 6);
    const int begin = ks.begin, end = ks.end;
    if (split >= ks.used) return;
    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int lr = lane & 31, lh = lane >> 5;
    const int D = FULL ? DP : a.D;
    const int P1 = (1 << a.shift) - 1;

    // this lane's query row: its token in the request (from t.n on: none) and its head
    auto query = [&](int lane32, int* head) {
        const int rho = t.rho0 + 32 * wave + lane32;
        const int i = rho / a.g;
        *head = hk * a.g + rho - i * a.g;
        return i;
    };
    int head;
    int qi = query(lr, &head);
    const bool real = qi < t.n;
    const int pos = t.kv - t.n + qi;
    const int hi = real && t.r < a.R ? min(pos, (a.width << a.shift) - 1) : -1;
    const int lo = a.window ? max(0, pos - a.window + 1) : 0;
    u32x4 qf[KS];
    {
        const uint16_t* src = a.q + (t.c0 + qi) * a.ld_q + int64_t(head) * a.D + 8 * lh;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            qf[s] = u32x4{0, 0, 0, 0};
            if (real && (FULL || 16 * s + 8 * lh < D)) qf[s] = *reinterpret_cast<const u32x4*>(src + 16 * s);
        }
    }
    const float c = a.scale * 1.4426950408889634f;
    float m = kNegInf, l = 0.f;
    f32x16 o[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.f;

    const int32_t* row = a.table + (t.r < a.R ? t.r : 0) * a.ld_table;
    auto page_of = [&](int key) { return row[min(key >> a.shift, a.width - 1)]; };
    auto in_cache = [&](int page) { return uint32_t(page) < uint32_t(a.n_pages); };

    // Staging.  A load instruction writes 1 KB of LDS, 16 bytes a lane in order.  K lies there as
    // [key][D] and V as [d][64 keys], the 16-byte chunks of a row permuted by an exclusive or, so
    // that sixteen neighbouring lanes of an operand read touch all 64 banks.
    auto kf = [](int key) { return DP == 64 ? (key >> 1) & 7 : key & 15; };
    const uint32_t klds = lds_byte(kbuf) + wave * NI * 1024, vlds = lds_byte(vbuf) + wave * NV * 1024;
    const int vrow = lane >> 3;
    // of a wave's even loads; odd ones are four chunks away, as are rows that are eight apart
    const int vchunk = (lane & 7) ^ (vrow >> 1) ^ (wave * NV & 1) * 4;
    int kp[2] = {0, 0}, vp[2] = {0, 0};
    auto pages_k = [&](int kt) {
        kp[0] = page_of(kt * kKT + 16 * wave);
        kp[1] = page_of(kt * kKT + 16 * wave + 8);
    };
    auto pages_v = [&](int kt) {
        vp[0] = page_of(kt * kKT + 8 * vchunk);
        vp[1] = page_of(kt * kKT + 8 * (vchunk ^ 4));
    };
    struct Source {
        const uint8_t* k[2];   // of the first of a page's eight keys
        const uint16_t* v[2];  // this lane's eight keys in row vrow of V, in even and odd loads
    };
    auto find_k = [&](int kt, Source& x) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int page = uniform(in_cache(kp[h]) ? kp[h] : 0);
            const int key = kt * kKT + 16 * wave + 8 * h;
            x.k[h] = reinterpret_cast<const uint8_t*>(
                a.kc + (((int64_t(page) * a.kv_heads + hk) << a.shift) + (key & P1)) * D);
        }
    };
    // row j * RPI + krow of the wave's sixteen; its permutation is that of j * RPI or-ed with krow's
    const int krow = lane / (DP / 8), kchunk = (lane % (DP / 8)) ^ kf(krow);
    const int koff = krow * DP * 2 + kchunk * 16;
    auto load_k = [&](int j, const Source& x, int buf) __attribute__((always_inline)) {
        int off;
        if constexpr (FULL) {
            off = (koff ^ (kf(j * RPI) * 16)) + (j * RPI & 7) * DP * 2;
        } else {
            int chunk = kchunk ^ kf(j * RPI);
            if (8 * chunk >= D) chunk = 0;  // meets zeros of the query
            off = ((j * RPI + krow) & 7) * D * 2 + chunk * 16;
        }
        load_lds16(x.k[j * 2 / NI], off, klds + buf * TILE + j * 1024);
    };
    auto find_v = [&](int kt, Source& x) __attribute__((always_inline)) -> bool {  // true: a page is outside the cache
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int page = in_cache(vp[h]) ? vp[h] : 0;
            x.v[h] = a.vc + ((int64_t(page) * a.kv_heads + hk) * D << a.shift) +
                     ((kt * kKT + 8 * (vchunk ^ (4 * h))) & P1);
        }
        return __any(!in_cache(vp[0]));
    };
    auto load_v = [&](int j, const Source& x, int buf) __attribute__((always_inline)) {
        int d = (wave * NV + j) * 8 + vrow;
        if (!FULL) d = min(d, D - 1);
        load_lds16(x.v[j & 1] + (int64_t(d) << a.shift), vlds + buf * TILE + j * 1024);
    };
    auto stage_k = [&](int kt, int buf) {
        Source x;
        find_k(kt, x);
#pragma unroll
        for (int j = 0; j < NI; ++j) load_k(j, x, buf);
    };
    auto stage_v = [&](int kt, int buf) {
        Source x;
        const bool bad = find_v(kt, x);
#pragma unroll
        for (int j = 0; j < NV; ++j) load_v(j, x, buf);
        return bad;
    };

    // Operand addresses.  Row m = 8a + 4h + b of the K operand takes key 16(a/2) + 8h + 4(a%2) + b,
    // so that a lane's sixteen scores are keys 8 lh .. 8 lh + 7 of both 16-key steps.
    const int key_m = 16 * (lr >> 4) + 8 * ((lr >> 2) & 1) + 4 * ((lr >> 3) & 1) + (lr & 3);
    const int kbase = key_m * DP * 2 + (lh ^ kf(key_m)) * 16;  // step st: its chunk number gains 2 st
    const int vbase = lr * 128 + (lh ^ (lr >> 1 & 7)) * 16;
    constexpr int KA = DP == 64 ? 4 : 8;  // steps that the exclusive or reaches
    auto kread = [&](int base, int sb, int st) {
        return *reinterpret_cast<const u32x4*>(&kbuf[(base ^ (st % KA * 32)) + st / KA * (KA * 32) + sb * 32 * DP * 2]);
    };
    auto vread = [&](int base, int d, int q) {
        return *reinterpret_cast<const u32x4*>(&vbuf[(base ^ (q * 32)) + d * 4096]);
    };

    auto edge = [&](int kt, bool bad) { return kt * kKT < t.full_lo || kt * kKT + kKT - 1 > t.full_hi || bad; };
    // masks and the running maximum, before the tile's exponentials
    auto maximum = [&](int kt, bool cut, f32x16* s, float mx) {
        if (cut) {
            mx = kNegInf;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int key = kt * kKT + 16 * q + 8 * lh;
                const bool gone = !in_cache(page_of(key));
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float z = s[q >> 1][8 * (q & 1) + j];
                    s[q >> 1][8 * (q & 1) + j] = (gone | (key + j > hi) | (key + j < lo)) ? kNegInf : z;
                    mx = fmaxf(mx, s[q >> 1][8 * (q & 1) + j]);
                }
            }
        }
        {
            // the other half's maximum; the operands are two values to the compiler, which takes both
            // results for one otherwise
            const auto z = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, mx),
                                                            uint32_t(fresh(__builtin_bit_cast(int, mx))), false, false);
            const uint32_t z0 = z[0], z1 = z[1];
            mx = fmaxf(__builtin_bit_cast(float, z0), __builtin_bit_cast(float, z1));
        }
        // the sums shrink only when a score outgrows the maximum by 2^3: probabilities then stay
        // below 2^3 (2^15 with binary16's factor), and most tiles leave the outputs alone
        if (__any((mx - m) * c > 3.f)) {
            const float mn = fmaxf(m, mx);
            const float alpha = __builtin_amdgcn_exp2f((m - (mn == kNegInf ? 0.f : mn)) * c);
            m = mn;
            l *= alpha;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[d][i] *= alpha;
        }
    };

    // Iteration i: the exponentials of tile i (scores `s`) on the vector unit while the matrix cores
    // make the scores of tile i + 1 (`sn`), then the value product of tile i.  K of i + 2 and V of
    // i + 1 are on their way meanwhile.
    const bool idle = t.rho0 + 32 * wave >= t.n * a.g;
    bool bad_v = false;  // a page of the tile staged last is outside the cache
    auto iteration = [&](int i, int buf, f32x16* s, f32x16* sn) {
        wait_loads();  // this wave's loads are in LDS
        __syncthreads();
        if (edge(i, bad_v)) {
            // values that no row may see can be anything in memory: make them zero
            for (int e = threadIdx.x; e < DM * 8; e += 256) {
                const int d = e >> 3, key = i * kKT + 8 * ((e & 7) ^ (d >> 1 & 7));
                const bool there = in_cache(page_of(key));
                u32x4* at = reinterpret_cast<u32x4*>(&vbuf[buf * TILE + e * 16]);
                u32x4 v = *at;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool x0 = there & (key + 2 * j >= t.kmin) & (key + 2 * j <= t.kmax);
                    const bool x1 = there & (key + 2 * j + 1 >= t.kmin) & (key + 2 * j + 1 <= t.kmax);
                    v[j] &= (x0 ? 0xFFFFu : 0u) | (x1 ? 0xFFFF0000u : 0u);
                }
                *at = v;
            }
            __syncthreads();
        }
        if (idle) {  // no rows: only its share of the loads
            stage_k(min(i + 2, end - 1), buf);
            bad_v = stage_v(min(i + 1, end - 1), buf ^ 1);
            pages_k(min(i + 3, end - 1)), pages_v(min(i + 2, end - 1));
            return;
        }
        const float mc = (m == kNegInf ? 0.f : m * c) - kBias<E>;
        // One straight run of matrix-core steps, the scores' (of what the buffer held, unused, behind
        // the last tile) and then the value product's.  Their operands are read from LDS four steps
        // ahead, since a read takes longer than a step, and the vector work stands between them: the
        // exponentials of keys 16 q .. 16 q + 15 before the value product of those keys.  The barriers
        // keep the compiler from gathering the reads right in front of their steps.
        constexpr int QK = 2 * KS, STEPS = QK + 4 * DB, SPREAD = QK + DB, MAX = (32 + 2 * DB - 1) / (2 * DB);
        u32x4 pf[4], fr[2][4];
        Source where;
        float sum[2] = {0.f, 0.f}, p[2];
        float mx[2] = {kNegInf, kNegInf};
        const int kb = DP == 128 ? fresh(kbase) : kbase, vb = DP == 128 ? fresh(vbase) : vbase;
        auto operand = [&](int z) {
            return z < QK ? kread(kb + (buf ^ 1) * TILE, z & 1, z >> 1)
                          : vread(vb + buf * TILE, (z - QK) % DB, (z - QK) / DB);
        };
#pragma unroll
        for (int e = 0; e < 16; ++e) sn[0][e] = sn[1][e] = 0.f;
#pragma unroll
        for (int y = 0; y < 4; ++y) fr[0][y] = operand(y);
        each([&](auto zc) __attribute__((always_inline)) {
            constexpr int z = decltype(zc)::value;
            if constexpr (z % 4 == 0 && z + 4 < STEPS) {
#pragma unroll
                for (int y = 0; y < 4; ++y) fr[(z / 4 + 1) & 1][y] = operand(z + 4 + y);
                __builtin_amdgcn_sched_barrier(0);
            }
            const u32x4 f = fr[z / 4 & 1][z % 4];
            if constexpr (z < QK) sn[z & 1] = E::mfma32(f, qf[z >> 1], sn[z & 1]);
            else o[(z - QK) % DB] = E::mfma32(f, pf[(z - QK) / DB], o[(z - QK) % DB]);
            constexpr int e0 = (z * 32 + SPREAD - 1) / SPREAD, e1 = ((z + 1) * 32 + SPREAD - 1) / SPREAD;
#pragma unroll
            for (int e = e0; e < e1 && e < 32; ++e) {
                p[e & 1] = __builtin_amdgcn_exp2f(fmaf(s[e >> 4][e & 15], c, -mc));
                sum[e & 1] += p[e & 1];
                if (e & 1) pf[e >> 3][(e & 7) >> 1] = pack16<E>(p[0], p[1]);
            }
            if constexpr (z >= SPREAD && z < SPREAD + 2 * DB) {
#pragma unroll
                for (int e = (z - SPREAD) * MAX; e < (z - SPREAD + 1) * MAX && e < 32; ++e)
                    mx[e & 1] = fmaxf(mx[e & 1], sn[e >> 4][e & 15]);
            }
            // The loads one by one: together they would hold up the steps behind them.  With FEW it is the
            // loads that take the time, and they go first.  Tiles behind the last one are the last again:
            // their buffers are not read.
            constexpr int GAP = FEW ? 0 : (STEPS - 2) / (NI + NV), at = z - 1;
            if constexpr (at == 0) find_k(min(i + 2, end - 1), where), pages_k(min(i + 3, end - 1));
            if constexpr (at == NI * GAP) bad_v = find_v(min(i + 1, end - 1), where), pages_v(min(i + 2, end - 1));
#pragma unroll
            for (int j = 0; j < NI; ++j)
                if (at == j * GAP) load_k(j, where, buf);
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (at == (NI + j) * GAP) load_v(j, where, buf ^ 1);
            __builtin_amdgcn_sched_barrier(0);
        }, std::make_integer_sequence<int, STEPS>{});
        asm volatile("" : "+v"(mx[0]), "+v"(mx[1]));  // made above, not where it turns out to be needed
        l += sum[0] + sum[1];
        if (i + 1 < end) maximum(i + 1, edge(i + 1, bad_v), sn, fmaxf(mx[0], mx[1]));
    };

    if (begin < end) {
        f32x16 s0[2], s1[2];
        pages_k(begin);
        pages_v(begin);
        stage_k(begin, 0);
        bad_v = stage_v(begin, 0);
        pages_k(min(begin + 1, end - 1));
        stage_k(min(begin + 1, end - 1), 1);
        pages_k(min(begin + 2, end - 1));
        pages_v(min(begin + 1, end - 1));
        wait_loads();
        __syncthreads();
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
#pragma unroll
            for (int e = 0; e < 16; ++e) s0[sb][e] = 0.f;
#pragma unroll
            for (int st = 0; st < KS; ++st)
                s0[sb] = E::mfma32(kread(kbase, sb, st), qf[st], s0[sb]);
        }
        float mx = kNegInf;
#pragma unroll
        for (int e = 0; e < 32; ++e) mx = fmaxf(mx, s0[e >> 4][e & 15]);
        maximum(begin, edge(begin, bad_v), s0, mx);
        for (int i = begin; i < end; i += 2) {
            iteration(i, 0, s0, s1);
            if (i + 1 < end) iteration(i + 1, 1, s1, s0);
        }
        // no load may still be writing LDS when the workgroup ends
        wait_loads();
    }

    l += __shfl_xor(l, 32);
    qi = query(fresh(lr), &head);
    if (qi >= t.n) return;
    const int64_t rowi = int64_t(t.c0 + qi) * a.heads + head;
    if (a.nsplit > 1 && lh == 0) put_ml(a, rowi, split, ks, m, l);
    if (ks.used > 1) {
        float* dst = a.opart + (rowi * a.nsplit + split) * D;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = 32 * d + 8 * j + 4 * lh;
                if (FULL || at < D)
                    *reinterpret_cast<f32x4*>(dst + at) =
                        f32x4{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
            }
    } else {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN stays NaN
        uint16_t* dst = a.y + (t.c0 + qi) * a.ld_y + int64_t(head) * D;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = 32 * d + 8 * j + 4 * lh;
                if (FULL || at < D)
                    *reinterpret_cast<u32x2*>(dst + at) =
                        u32x2{pack16<E>(o[d][4 * j] * inv, o[d][4 * j + 1] * inv),
                              pack16<E>(o[d][4 * j + 2] * inv, o[d][4 * j + 3] * inv)};
            }
        if (lh == 0 && a.lse)
            a.lse[rowi] = l == 0.f ? kNegInf : fmaf(m, a.scale, logf(l) - kBias<E> * 0.6931471805599453f);
    }
}

template <class E, int DP, bool FEW>
void launch_dp(const AttnArgs& a, unsigned blocks, hipStream_t s) {
    // Heads of up to three quarters of the LDS row leave the last quarter's products and values out: 512 rows
    // over 16,001 keys, 24/4 heads of 192: 293 -> 247 us, of 96: 137 -> 114; 64 requests of 8 tokens and up to
    // 16,252 keys, 40/8 heads of 192: 834 -> 762.
    constexpr int DM = DP > 64 ? DP / 4 * 3 : DP;
    if (a.D == DP) k_attn_tile<E, DP, DP, true, FEW><<<blocks, 256, 0, s>>>(a);
    else if (a.D <= DM) k_attn_tile<E, DP, DM, false, FEW><<<blocks, 256, 0, s>>>(a);
    else k_attn_tile<E, DP, DP, false, FEW><<<blocks, 256, 0, s>>>(a);
}

template <class E, bool FEW>
void launch_e(const AttnArgs& a, unsigned blocks, hipStream_t s) {
    if (a.D <= 64) launch_dp<E, 64, FEW>(a, blocks, s);
    else if (a.D <= 128) launch_dp<E, 128, FEW>(a, blocks, s);
    else launch_dp<E, 256, FEW>(a, blocks, s);
}

}  // namespace

void launch_attn_tile(const AttnArgs& a, int dtype, bool few, int tiles, hipStream_t s) {
    const unsigned blocks = unsigned(tiles) * a.kv_heads * split_slots(a.nsplit, a.R);
    if (dtype == VQMLP_F16) few ? launch_e<F16, true>(a, blocks, s) : launch_e<F16, false>(a, blocks, s);
    else few ? launch_e<BF16, true>(a, blocks, s) : launch_e<BF16, false>(a, blocks, s);
}

}  // namespace vqmlp
