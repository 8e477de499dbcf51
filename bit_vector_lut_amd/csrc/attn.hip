// attn.hip -- attention of a chunk of new tokens over the paged key/value cache (gfx950).
//
//   y[t][h] = sum_j softmax_j(scale q . k_j) v_j over the positions j that row t sees.
//
// One pass over the keys with the running maximum m and sum l of the softmax: a tile of scores s
// gives m' = max(m, s), the sums so far shrink by 2^((m - m') c), and p = 2^((s - m') c) joins them
// (c = scale log2 e).  The query heads that share a key head are rows of one tile, row = token *
// group + head in group, so a key is read once for all of them.
//
// Operands without a transpose.  Scores are computed as S^T = K Q^T and outputs as O^T = V^T P^T,
// 16x16 matrix-core steps.  A result of the first holds, per lane, four scores of one query row;
// the second wants, per lane, eight keys of one query row.  The order of the keys along an
// operand is free as long as both operands agree, so the two key sub-tiles of a 32-key tile take
// keys 8(m/4) + m%4 and the same + 4: a lane then holds keys 8g .. 8g+7 (g = lane / 16), packs
// them to 16 bits in place, and the matching operand of V^T is one 16-byte load because the cache
// keeps values as [D][page_size].  Neither product goes through LDS.
#include "attn.h"

#include <algorithm>

namespace vqmlp {

namespace {

// ---------------------------------------------------------------- few rows: keys over the waves
// D in 129 .. 256.  Four waves share 16 rows of one key head and a split of the keys, tile by tile in
// turn, each straight from the cache into its registers; their sums join in LDS at the end.  Bound by
// reading the cache.  A tile ahead in registers measured the same, 256 registers for two waves a SIMD
// spill (177 against 123 us at 32 requests of up to 8,000 keys, 24/4 heads of 256).
template <class E, bool FULL>
__global__ void __launch_bounds__(256) k_attn_wave(AttnArgs a) {
    constexpr int DP = 256, NW = 4, MT = 16, KS = DP / 32, DT = DP / 16;
    constexpr int DC = 128;  // columns joined per round
    __shared__ float obuf[NW][MT][DC + 4];
    __shared__ float mlbuf[NW][MT][2];
    Tile t;
    const int hk = blockIdx.y, split = blockIdx.z;
    if (!find_tile<MT>(a, blockIdx.x, t)) return;
    const Split ks = key_split(a, t, split, 5);
    const int begin = ks.begin, end = ks.end;
    if (split >= ks.used) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lr = lane & 15, g = lane >> 4;
    const int D = FULL ? DP : a.D;
    const int P1 = (1 << a.shift) - 1;

    const int rho = t.rho0 + lr;
    const int qi = rho / a.g, hh = rho - qi * a.g;
    const bool real = qi < t.n;
    const int pos = t.kv - t.n + qi;
    const int hi = real && t.r < a.R ? min(pos, (a.width << a.shift) - 1) : -1;
    const int lo = a.window ? max(0, pos - a.window + 1) : 0;
    const uint16_t* src = a.q + (t.c0 + qi) * a.ld_q + int64_t(hk * a.g + hh) * a.D + 8 * g;
    u32x4 qf[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        qf[s] = u32x4{0, 0, 0, 0};
        if (real && (FULL || 32 * s + 8 * g < D)) qf[s] = *reinterpret_cast<const u32x4*>(src + 32 * s);
    }
    float m = kNegInf, l = 0.f;
    f32x4 o[DT];
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) o[dt] = f32x4{0.f, 0.f, 0.f, 0.f};
    const float c = a.scale * 1.4426950408889634f;

    const int32_t* row = a.table + (t.r < a.R ? t.r : 0) * a.ld_table;
    // page numbers of the lane's two K rows and of its eight V columns in a tile
    const int krow = 8 * (lr >> 2), vcol = 8 * g;
    auto page_of = [&](int key) { return row[min(key >> a.shift, a.width - 1)]; };
    struct Keys {
        u32x4 a[KS], b[KS], v[DT];
        bool bad;
    } cur;
    int kp = 0, vp = 0;  // pages of the tile loaded next
    auto pages = [&](int kt) {
        kp = page_of(kt * 32 + krow);
        vp = page_of(kt * 32 + vcol);
    };
    auto load = [&](int kt, Keys& x) __attribute__((always_inline)) {
        const int k0 = kt * 32;
        x.bad = uint32_t(vp) >= uint32_t(a.n_pages);
        const int kq = uint32_t(kp) >= uint32_t(a.n_pages) ? 0 : kp, vq = x.bad ? 0 : vp;
        const uint16_t* kr = a.kc +
            (((int64_t(kq) * a.kv_heads + hk) << a.shift) + ((k0 + krow) & P1) + (lr & 3)) * D;
        const uint16_t* vr = a.vc + ((int64_t(vq) * a.kv_heads + hk) * D << a.shift) + ((k0 + vcol) & P1);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            // columns behind D meet zeros of the query: any finite chunk will do
            const int at = FULL || 32 * s + 8 * g < D ? 32 * s + 8 * g : 0;
            x.a[s] = *reinterpret_cast<const u32x4*>(kr + at);
            x.b[s] = *reinterpret_cast<const u32x4*>(kr + 4 * D + at);
        }
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
            const int d = 16 * dt + lr;
            x.v[dt] = *reinterpret_cast<const u32x4*>(vr + (int64_t(FULL ? d : min(d, D - 1)) << a.shift));
        }
    };
    auto compute = [&](int kt, Keys& x) __attribute__((always_inline)) {
        const int k0 = kt * 32, key = k0 + vcol;
        const bool edge = k0 < t.full_lo || k0 + 31 > t.full_hi || __any(x.bad);
        f32x4 sa = {0.f, 0.f, 0.f, 0.f}, sb = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            sa = E::mfma16(x.a[s], qf[s], sa);
            sb = E::mfma16(x.b[s], qf[s], sb);
        }
        if (edge) {
            // values that no row may see can be anything in memory: make them zero
            u32x4 keep;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool y = !x.bad & (key + 2 * j >= t.kmin) & (key + 2 * j <= t.kmax);
                const bool z = !x.bad & (key + 2 * j + 1 >= t.kmin) & (key + 2 * j + 1 <= t.kmax);
                keep[j] = (y ? 0xFFFFu : 0u) | (z ? 0xFFFF0000u : 0u);
                if (x.bad | (key + j > hi) | (key + j < lo)) sa[j] = kNegInf;
                if (x.bad | (key + 4 + j > hi) | (key + 4 + j < lo)) sb[j] = kNegInf;
            }
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) x.v[dt] &= keep;
        }
        float mx = fmaxf(fmaxf(fmaxf(sa[0], sa[1]), fmaxf(sa[2], sa[3])),
                         fmaxf(fmaxf(sb[0], sb[1]), fmaxf(sb[2], sb[3])));
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        if (__any(mx > m)) {
            const float mn = fmaxf(m, mx);
            const float alpha = __builtin_amdgcn_exp2f((m - (mn == kNegInf ? 0.f : mn)) * c);
            m = mn;
            l *= alpha;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) o[dt] *= alpha;
        }
        const float mc = (m == kNegInf ? 0.f : m * c) - kBias<E>;
        float p[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            p[j] = __builtin_amdgcn_exp2f(fmaf(sa[j], c, -mc));
            p[4 + j] = __builtin_amdgcn_exp2f(fmaf(sb[j], c, -mc));
        }
        l += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
        // the probabilities as matrix-core operands: one rounding to the type of the values
        const u32x4 pf = {pack16<E>(p[0], p[1]), pack16<E>(p[2], p[3]), pack16<E>(p[4], p[5]),
                          pack16<E>(p[6], p[7])};
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[dt] = E::mfma16(x.v[dt], pf, o[dt]);
    };
    int kt = begin + wave;
    if (kt < end) {
        // tiles behind the last one are the last again
        auto clip = [&](int k) { return min(k, end - 1); };
        pages(kt);
        for (; kt < end; kt += NW) {
            load(kt, cur);
            pages(clip(kt + NW));
            compute(kt, cur);
        }
    }

    // join the waves
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
        mlbuf[wave][lr][0] = m;
        mlbuf[wave][lr][1] = l;
    }
    constexpr int TPR = NW * 64 / MT;  // threads per row
    const int jr = threadIdx.x / TPR, jt = threadIdx.x % TPR;
#pragma unroll
    for (int d0 = 0; d0 < DP; d0 += DC) {
        __syncthreads();
#pragma unroll
        for (int dt = 0; dt < DC / 16; ++dt)
            *reinterpret_cast<f32x4*>(&obuf[wave][lr][16 * dt + 4 * g]) = o[d0 / 16 + dt];
        __syncthreads();
        const int i = (t.rho0 + jr) / a.g;
        if (i >= t.n) continue;
        float mm = kNegInf;
#pragma unroll
        for (int w = 0; w < NW; ++w) mm = fmaxf(mm, mlbuf[w][jr][0]);
        const float ms = mm == kNegInf ? 0.f : mm;
        float wt[NW], sum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            wt[w] = __builtin_amdgcn_exp2f((mlbuf[w][jr][0] - ms) * c);
            sum = fmaf(wt[w], mlbuf[w][jr][1], sum);
        }
        const int head = hk * a.g + t.rho0 + jr - i * a.g;
        const int64_t rowi = int64_t(t.c0 + i) * a.heads + head;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;  // NaN stays NaN
        for (int d = jt * 4; d < DC && d0 + d < D; d += TPR * 4) {
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(&obuf[w][jr][d]);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = fmaf(wt[w], x[j], v[j]);
            }
            if (ks.used == 1) {
                const u32x2 w2 = {pack16<E>(v[0] * inv, v[1] * inv), pack16<E>(v[2] * inv, v[3] * inv)};
                *reinterpret_cast<u32x2*>(a.y + (t.c0 + i) * a.ld_y + int64_t(head) * D + d0 + d) = w2;
            } else {
                *reinterpret_cast<f32x4*>(a.opart + (rowi * a.nsplit + split) * D + d0 + d) = v;
            }
        }
        if (d0 == 0 && jt == 0) {
            if (a.nsplit > 1) put_ml(a, rowi, split, ks, mm, sum);
            if (ks.used == 1 && a.lse) {
                a.lse[rowi] = sum == 0.f ? kNegInf
                                         : fmaf(mm, a.scale, logf(sum) - kBias<E> * 0.6931471805599453f);
            }
        }
    }
}

// Join the splits of a row: one wave a row where they are few, else four (64 splits of 192 rows of 256
// columns: 24 us with one, 5 with four).  Lane = split for the weights, then four columns.  Bound by the
// latency of the loads, so eight are on their way at once; four waves issue them before they know which
// splits have keys, and use what those wrote only.
template <class E, int WPR>
__global__ void __launch_bounds__(256) k_attn_join(AttnArgs a) {
    __shared__ float buf[WPR][256];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t row = WPR == 1 ? int64_t(blockIdx.x) * 4 + wave : blockIdx.x;
    if (row >= int64_t(a.T) * a.heads) return;
    const bool in = 4 * lane < a.D;
    const float* src = a.opart + row * a.nsplit * a.D + (in ? 4 * lane : 0);
    const int s0 = WPR == 1 ? 0 : wave;
    f32x4 x[8];
    auto load = [&](int s, int end) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (s + WPR * j < end)
                x[j] = *reinterpret_cast<const f32x4*>(src + int64_t(s + WPR * j) * a.D);
    };
    if (WPR > 1) load(s0, a.nsplit);
    float m = kNegInf, l = -1.f;
    if (lane < a.nsplit) {
        m = a.ml[(row * a.nsplit + lane) * 2];
        l = a.ml[(row * a.nsplit + lane) * 2 + 1];
    }
    if (__builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, l))) < 0.f)
        return;  // done in one split, which wrote no more than this
    const int used = __popcll(__ballot(!(l < 0.f)));  // the first ones
    if (lane >= used) m = kNegInf, l = 0.f;
    if (WPR == 1) load(s0, used);
    float mm = m;
#pragma unroll
    for (int o = 32; o; o >>= 1) mm = fmaxf(mm, __shfl_xor(mm, o));
    const float c = a.scale * 1.4426950408889634f;
    const float w = __builtin_amdgcn_exp2f((m - (mm == kNegInf ? 0.f : mm)) * c);
    const float sum = wave_sum(w * l);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // NaN stays NaN
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int s = s0; s < used; s += 8 * WPR) {
        if (s != s0) load(s, used);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int at = s + WPR * j;
            if (at >= used) break;
            const float ws = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), at));
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fmaf(ws, x[j][i], v[i]);
        }
    }
    const int64_t tok = row / a.heads;
    const int head = int(row % a.heads);
    uint16_t* dst = a.y + tok * a.ld_y + int64_t(head) * a.D;
    if constexpr (WPR == 1) {
        if (in)
            *reinterpret_cast<u32x2*>(dst + 4 * lane) =
                u32x2{pack16<E>(v[0] * inv, v[1] * inv), pack16<E>(v[2] * inv, v[3] * inv)};
    } else {
        *reinterpret_cast<f32x4*>(&buf[wave][4 * lane]) = v;
        __syncthreads();
        const int d = threadIdx.x;
        if (d < a.D) {
            float z = 0.f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) z += buf[i][d];
            dst[d] = uint16_t(bits16<E>(z * inv));
        }
    }
    if (lane == 0 && (WPR == 1 || wave == 0) && a.lse)
        a.lse[row] = sum == 0.f ? kNegInf : fmaf(mm, a.scale, logf(sum) - kBias<E> * 0.6931471805599453f);
}

// ---------------------------------------------------------------- host half

struct AttnGeom {
    bool lds;       // tiles of kAttnTileRows with the keys in LDS, otherwise register tiles of 16 rows
    bool few;       // few rows a request: the loads of a tile before its matrix-core steps
    int tiles, nsplit, split_tiles;
    size_t opart, ml, bytes;
};

// Up to 16 rows of D > 128 take register tiles: their 64 KB tiles leave the LDS kernel one workgroup a
// compute unit, which cannot hide the cache's latency (32 requests of up to 8,000 keys, 24/4 heads of
// 256: 121 against 153 us).  Everything else takes LDS tiles: 64 requests of one token, D = 64: 415
// against 837 us; 8 tokens over 65,472 keys, 40/8 heads of 128: 53 against 200 us, 24/4 heads of 256:
// 59 against 153 us.
AttnGeom attn_geom(const vqmlp_attn_desc& d, int cus) {
    AttnGeom G{};
    const int g = d.heads / d.kv_heads;
    const int64_t all = int64_t(d.T) * g;
    const int64_t rows = std::max<int64_t>(1, (all + d.R - 1) / std::max(1, d.R));
    const size_t rows_all = size_t(d.T) * d.heads;
    G.lds = d.D <= 128 || rows > 16;
    // with loads first 8 tokens over 65,472 keys take 54 us for 40/8 heads of 128 (58 with loads between
    // the steps), 64 ragged requests of one token 403 (420), but 24/4 heads of 256 take 63 (59)
    G.few = rows * d.D <= 64 * 128;
    const int mt = G.lds ? kAttnTileRows : 16, key_tile = G.lds ? 64 : 32;
    G.tiles = int(all / mt) + d.R + 1;
    const int64_t active = std::max<int64_t>(d.R, (all + mt - 1) / mt) * d.kv_heads;
    // A launch holds fewer than 2^32 threads: the places of all tiles' splits, the join's rows.
    const int64_t places = ((1 << 24) - 1) / (int64_t(G.tiles) * d.kv_heads);
    const int most = rows_all >= size_t(1) << 26
                         ? 1 : int(std::min<int64_t>(kMaxSplit, std::max<int64_t>(1, d.R > 1 ? (places - 1) | 1 : places)));
    auto splits = [&](int key_tiles) {
        if (G.lds) {
            // Times in us.  A workgroup passes over a tile in 1 us and 0.35 more for each wave with rows
            // (D = 128), if all of them together stay below 5 TB/s of keys and values (which the row tiles
            // of a request share); two tiles' worth to start and end each; the join writes and reads FP32
            // sums at about 4 TB/s.  512 rows of 40/8 heads of 128 over 33,001 keys: 425 us with the three
            // splits that this chooses, 618 / 507 / 454 / 430 / 432 with 1 / 2 / 4 / 6 / 8.  max_kv is the longest of
            // several requests: half of the estimate is for all being as long, half for that one alone.
            const int64_t slots = int64_t(cus) * (d.D <= 128 ? 2 : 1);
            const double alone = (1.0 + 0.35 * double(std::min<int64_t>(4, (rows + 31) / 32))) * d.D / 128;
            int nsplit = 1;
            double best = 1e300;
            for (int ns = 1; ns <= std::min(most, std::max(1, key_tiles / 4)); ++ns) {
                const int64_t blocks = active * ns;
                const int64_t busy = std::min((blocks + cus - 1) / cus * cus, slots);  // as full as the fullest
                const double tile = std::max(alone, double(busy) * key_tile * d.D * 4 / 5e6 * d.R * d.kv_heads / active);
                const double tiles = (key_tiles + ns - 1) / ns + 2;
                double cost = double((blocks + slots - 1) / slots) * tiles * tile;
                if (d.R > 1) cost = 0.5 * cost + 0.5 * tiles * alone;
                if (ns > 1) cost += 4 + ns * double(rows_all) * d.D * 8 / 4e6 * (d.R > 1 ? 0.5 : 1.0);
                if (cost < best) best = cost, nsplit = ns;
            }
            return nsplit;
        }
        // four workgroups a compute unit: 123 us at the sizes above, 127 / 130 / 147 with 3 / 6 / 12
        const int64_t want = (int64_t(cus) * 4 + active - 1) / active;
        return int(std::min<int64_t>(std::min<int64_t>(want, std::max(1, key_tiles / 8)), most));
    };
    // Through a window a row tile sees that many keys and one for each of its tokens: one request of a
    // token over 32,000 keys, 40/8 heads of 128, window 4,096: 15 us, 27 with splits for all 32,000; 64
    // ragged requests, window 1,024: 53 and 75.  No more splits than without it, so that a workspace made
    // without it holds.
    int key_tiles = (std::max(1, d.max_kv) - 1) / key_tile + 1;
    G.nsplit = splits(key_tiles);
    if (d.window) {
        const int64_t reach = int64_t(d.window) + std::min(d.T, (mt + g - 1) / g);  // from any key on
        key_tiles = int(std::min<int64_t>(key_tiles, (reach + key_tile - 2) / key_tile + 1));
        G.nsplit = std::min(G.nsplit, splits(key_tiles));
    }
    G.split_tiles = (key_tiles + G.nsplit - 1) / G.nsplit;
    G.opart = 0;
    G.ml = align256(G.nsplit > 1 ? rows_all * G.nsplit * d.D * 4 : 0);
    G.bytes = G.ml + align256(G.nsplit > 1 ? rows_all * G.nsplit * 8 : 0);
    return G;
}

bool attn_page_shift(int page_size, int* shift) {
    for (int s = 3; s <= 10; ++s)
        if (page_size == 1 << s) return *shift = s, true;
    return false;
}

vqmlp_status attn_check(const vqmlp_attn_desc* p, const char* who, int* shift) {
    OP_REQUIRE(p, "%s: null description", who);
    const vqmlp_attn_desc& d = *p;
    OP_REQUIRE(op_dtype16(d.dtype), "%s: dtype %d is not F16 or BF16", who, d.dtype);
    OP_REQUIRE(attn_page_shift(d.page_size, shift), "%s: page_size %d is not a power of two in 8..1024",
               who, d.page_size);
    OP_REQUIRE(d.T >= 0 && d.R >= 1 && d.heads >= 1 && d.kv_heads >= 1 && d.n_pages >= 1 &&
                   d.table_width >= 1 && d.window >= 0 && d.max_kv >= 0,
               "%s: a size is out of range", who);
    OP_REQUIRE(d.D >= 8 && d.D <= 256 && d.D % 8 == 0, "%s: D=%d is not a multiple of 8 up to 256", who, d.D);
    OP_REQUIRE(d.heads % d.kv_heads == 0, "%s: heads=%d is no multiple of kv_heads=%d", who, d.heads,
               d.kv_heads);
    if (d.heads / d.kv_heads > 64 || d.R > 65536 || d.kv_heads > 65535)
        OP_FAIL(VQMLP_ERR_UNSUPPORTED, "%s: heads / kv_heads above 64 or R above 65536", who);
    if (int64_t(d.T) * d.heads > 0x3FFFFFFF)
        OP_FAIL(VQMLP_ERR_UNSUPPORTED, "%s: T * heads above 2^30 - 1", who);
    // a launch holds fewer than 2^32 threads; attn_geom splits no further than that
    if ((int64_t(d.T) * (d.heads / d.kv_heads) / kAttnTileRows + d.R + 1) * d.kv_heads >= (1 << 24))
        OP_FAIL(VQMLP_ERR_UNSUPPORTED, "%s: (T * heads / kv_heads / 128 + R + 1) * kv_heads is not below 2^24", who);
    OP_REQUIRE((int64_t(d.n_pages) << *shift) <= 0x7FFFFFFF && (int64_t(d.table_width) << *shift) <= 0x3FFFFFFF,
               "%s: slots pass 2^31 - 1 or positions 2^30 - 1", who);
    OP_REQUIRE(d.scale > 0.f && d.scale < __builtin_inff(), "%s: scale is not positive and finite", who);
    return VQMLP_OK;
}

template <class E>
void launch_attn(const AttnArgs& a, const AttnGeom& G, int dtype, hipStream_t s) {
    if (G.lds) {
        launch_attn_tile(a, dtype, G.few, G.tiles, s);
    } else {
        const dim3 grid(G.tiles, a.kv_heads, a.nsplit);
        if (a.D == 256) k_attn_wave<E, true><<<grid, 256, 0, s>>>(a);
        else k_attn_wave<E, false><<<grid, 256, 0, s>>>(a);
    }
    if (a.nsplit > 1) {
        const int64_t rows = int64_t(a.T) * a.heads;
        if (a.nsplit <= 8 || rows >= (1 << 24)) k_attn_join<E, 1><<<dim3((rows + 3) / 4), 256, 0, s>>>(a);
        else k_attn_join<E, 4><<<dim3(rows), 256, 0, s>>>(a);
    }
}

}  // namespace

}  // namespace vqmlp

extern "C" vqmlp_status vqmlp_paged_attn_workspace(const vqmlp_attn_desc* p, size_t* bytes) {
    using namespace vqmlp;
    OP_REQUIRE(bytes, "vqmlp_paged_attn_workspace: null pointer");
    int shift = 0, cus = 0;
    if (const vqmlp_status st = attn_check(p, "vqmlp_paged_attn_workspace", &shift)) return st;
    if (const int st = device_cus(&cus)) return static_cast<vqmlp_status>(st);
    *bytes = attn_geom(*p, cus).bytes;
    return op_ok();
}

extern "C" vqmlp_status vqmlp_paged_attn(const vqmlp_attn_desc* p, void* workspace,
                                         size_t workspace_bytes, void* stream) {
    using namespace vqmlp;
    int shift = 0, cus = 0;
    if (const vqmlp_status st = attn_check(p, "vqmlp_paged_attn", &shift)) return st;
    const vqmlp_attn_desc& d = *p;
    if (d.T == 0) return op_ok();
    OP_REQUIRE(d.q && d.y && d.k_cache && d.v_cache && d.table && d.cu_q && d.kv_len,
               "vqmlp_paged_attn: null pointer");
    const int64_t row = int64_t(d.heads) * d.D;
    OP_REQUIRE((d.T == 1 || (d.ld_q >= row && d.ld_y >= row)) && d.ld_q >= 0 && d.ld_y >= 0 &&
                   d.ld_q <= (int64_t(1) << 40) && d.ld_y <= (int64_t(1) << 40) && d.ld_q % 8 == 0 &&
                   d.ld_y % 8 == 0,
               "vqmlp_paged_attn: token strides have to be multiples of 8, at least heads * D");
    OP_REQUIRE(d.ld_table >= d.table_width, "vqmlp_paged_attn: ld_table is below table_width");
    OP_REQUIRE(op_aligned(d.q, 16) && op_aligned(d.y, 16) && op_aligned(d.k_cache, 16) &&
                   op_aligned(d.v_cache, 16) && op_aligned(d.table, 4) && op_aligned(d.cu_q, 4) &&
                   op_aligned(d.kv_len, 4) && op_aligned(d.lse, 4),
               "vqmlp_paged_attn: q, y and the caches have to be 16-byte aligned, the rest 4-byte");
    if (const int st = device_cus(&cus)) return static_cast<vqmlp_status>(st);
    const AttnGeom G = attn_geom(d, cus);
    if (G.bytes) {
        OP_REQUIRE(workspace && op_aligned(workspace, 256),
                   "vqmlp_paged_attn: the workspace is null or not 256-byte aligned");
        if (workspace_bytes < G.bytes)
            OP_FAIL(VQMLP_ERR_WORKSPACE, "vqmlp_paged_attn: workspace holds %zu bytes, this call needs %zu",
                    workspace_bytes, G.bytes);
    }
    AttnArgs a;
    a.q = static_cast<const uint16_t*>(d.q);
    a.y = static_cast<uint16_t*>(d.y);
    a.lse = d.lse;
    a.kc = static_cast<const uint16_t*>(d.k_cache);
    a.vc = static_cast<const uint16_t*>(d.v_cache);
    a.table = d.table;
    a.cu = d.cu_q;
    a.kv_len = d.kv_len;
    a.opart = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + G.opart);
    a.ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + G.ml);
    a.ld_table = d.ld_table;
    a.ld_q = d.ld_q;
    a.ld_y = d.ld_y;
    a.T = d.T;
    a.R = d.R;
    a.heads = d.heads;
    a.kv_heads = d.kv_heads;
    a.g = d.heads / d.kv_heads;
    a.D = d.D;
    a.shift = shift;
    a.n_pages = d.n_pages;
    a.window = std::min(d.window, 0x3FFFFFFF);
    a.nsplit = G.nsplit;
    a.split_tiles = G.split_tiles;
    a.width = d.table_width;
    a.scale = d.scale;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (d.dtype == VQMLP_F16) launch_attn<F16>(a, G, d.dtype, s);
    else launch_attn<BF16>(a, G, d.dtype, s);
    if (trace_enabled())
        trace_line("paged_attn T=%d R=%d heads=%d/%d D=%d: %s tiles, %d rows, %d key splits%s", d.T, d.R,
                   d.heads, d.kv_heads, d.D, G.lds ? "LDS" : "register", G.lds ? kAttnTileRows : 16,
                   G.nsplit, G.nsplit > 1 ? " + join" : "");
    return op_launched("vqmlp_paged_attn");
}
