// attn_tile.hip -- paged attention for many rows: prompts and prompt chunks (gfx950).
//
// The mathematics, the packing of rows and the transposed products are those of attn.hip; here
// four waves share a tile of 64 keys in LDS and each has 32 RB rows of its own, 32x32x16
// matrix-core steps.  Bound by the matrix cores and, beside them, by the exponentials.
#include "attn.h"

namespace vqmlp {

namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void global_void;

constexpr int kKT = 64;  // keys of a tile

template <class E, int DP, int RB, bool FULL>
__global__ void __launch_bounds__(256, DP == 64 || RB == 1 ? 2 : 1) k_attn_tile(AttnArgs a) {
    constexpr int KS = DP / 16, DB = DP / 32, NI = DP / 32;
    constexpr int MT = 128 * RB;
    constexpr int RPI = 512 / DP;  // key rows per load instruction
    __shared__ __attribute__((aligned(1024))) uint8_t kbuf[2][kKT * DP * 2];
    __shared__ __attribute__((aligned(1024))) uint8_t vbuf[2][kKT * DP * 2];
    const int groups = a.kv_heads * a.nsplit;
    const int x = blockIdx.x / groups, gi = blockIdx.x % groups;
    const int hk = gi % a.kv_heads, split = gi / a.kv_heads;
    Tile t;
    if (!find_tile<MT>(a, x, t)) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 31, lh = lane >> 5;
    const int D = FULL ? DP : a.D;
    const int P1 = (1 << a.shift) - 1;

    int lo[RB], hi[RB];
    u32x4 qf[RB][KS];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        const int rho = t.rho0 + 32 * (RB * wave + b) + lr;
        const int i = rho / a.g, hh = rho - i * a.g;
        const bool real = i < t.n;
        const int p = t.kv - t.n + i;
        hi[b] = real && t.r < a.R ? min(p, (a.width << a.shift) - 1) : -1;
        lo[b] = a.window ? max(0, p - a.window + 1) : 0;
        const uint16_t* src = a.q + (t.c0 + i) * a.ld_q + int64_t(hk * a.g + hh) * a.D + 8 * lh;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            qf[b][s] = u32x4{0, 0, 0, 0};
            if (real && (FULL || 16 * s + 8 * lh < D))
                qf[b][s] = *reinterpret_cast<const u32x4*>(src + 16 * s);
        }
    }
    float m[RB], l[RB];
    f32x16 o[RB][DB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        m[b] = kNegInf;
        l[b] = 0.f;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[b][d][i] = 0.f;
    }
    const float c = a.scale * 1.4426950408889634f;

    const int kt0 = t.kmin / kKT;
    const int nt = t.kmax >= t.kmin ? t.kmax / kKT + 1 - kt0 : 0;
    const int begin = kt0 + min(nt, split * a.split_tiles);
    const int end = kt0 + (split == a.nsplit - 1 ? nt : min(nt, (split + 1) * a.split_tiles));
    const int32_t* row = a.table + (t.r < a.R ? t.r : 0) * a.ld_table;
    auto page_of = [&](int key) { return row[min(key >> a.shift, a.width - 1)]; };

    // Staging.  A load instruction writes 1 KB of LDS, 16 bytes a lane in order.  K lies there as
    // [key][D] and V as [d][64 keys], the 16-byte chunks of a row permuted by an exclusive or so
    // that eight neighbouring lanes of an operand read touch all banks.
    const int krow = lane / (DP / 8), kslot = lane % (DP / 8);
    const int vrow = lane >> 3, vchunk = (lane & 7) ^ vrow;
    auto kf = [](int key) { return (key & 3) | ((key >> 1) & 4); };
    int vp_n = 0, kp_n[2] = {0, 0};
    auto pages = [&](int kt) {
        vp_n = page_of(kt * kKT + 8 * vchunk);
        kp_n[0] = page_of(kt * kKT + 16 * wave);
        kp_n[1] = page_of(kt * kKT + 16 * wave + 8);
    };
    auto stage = [&](int kt, int buf) -> bool {  // true: a page of the tile is outside the cache
        const int k0 = kt * kKT;
        const bool bad = uint32_t(vp_n) >= uint32_t(a.n_pages);
        const int vp = bad ? 0 : vp_n;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int key = 16 * wave + j * RPI + krow;
            const int kp = uint32_t(kp_n[j * 2 / NI]) >= uint32_t(a.n_pages) ? 0 : kp_n[j * 2 / NI];
            int chunk = kslot ^ kf(key);
            if (!FULL && 8 * chunk >= D) chunk = 0;  // meets zeros of the query
            const uint16_t* src = a.kc + (((int64_t(kp) * a.kv_heads + hk) << a.shift) + ((k0 + key) & P1)) * D + 8 * chunk;
            __builtin_amdgcn_global_load_lds((global_void*)src, (lds_void*)&kbuf[buf][(wave * NI + j) * 1024], 16, 0, 0);
        }
        const uint16_t* vsrc = a.vc + ((int64_t(vp) * a.kv_heads + hk) * D << a.shift) + ((k0 + 8 * vchunk) & P1);
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            int d = (wave * NI + j) * 8 + vrow;
            if (!FULL) d = min(d, D - 1);
            __builtin_amdgcn_global_load_lds((global_void*)(vsrc + (int64_t(d) << a.shift)),
                                             (lds_void*)&vbuf[buf][(wave * NI + j) * 1024], 16, 0, 0);
        }
        return __any(bad);
    };

    // operand addresses: row m of the K operand takes key 16(a/2) + 8h + 4(a%2) + b, m = 8a + 4h + b,
    // so that a lane's sixteen scores are keys 8 lh .. 8 lh + 7 of both 16-key steps.
    const int key_m = 16 * (lr >> 4) + 8 * ((lr >> 2) & 1) + 4 * ((lr >> 3) & 1) + (lr & 3);
    int kaddr[4], vaddr[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        kaddr[s] = key_m * DP * 2 + (((2 * s + lh) ^ kf(key_m)) * 16);
        vaddr[s] = lr * 128 + (((2 * s + lh) ^ (lr & 7)) * 16);
    }

    // one tile: EDGE where some row does not see all its keys
    auto compute = [&](int kt, int buf, auto edge_c) {
        constexpr bool EDGE = decltype(edge_c)::value;
        const int k0 = kt * kKT;
        f32x16 s[RB][2];
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[b][sb][i] = 0.f;
#pragma unroll
            for (int st = 0; st < KS; ++st) {
                const u32x4 k = *reinterpret_cast<const u32x4*>(&kbuf[buf][kaddr[st & 3] + (st >> 2) * 128 + sb * 32 * DP * 2]);
#pragma unroll
                for (int b = 0; b < RB; ++b) s[b][sb] = E::mfma32(k, qf[b][st], s[b][sb]);
            }
        }
        u32x4 pf[RB][4];
        bool there[4];
        if constexpr (EDGE) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                there[q] = uint32_t(page_of(k0 + 16 * q + 8 * lh)) < uint32_t(a.n_pages);
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            if constexpr (EDGE) {
#pragma unroll
                for (int sb = 0; sb < 2; ++sb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int k = k0 + 32 * sb + 16 * (i >> 3) + 8 * lh + (i & 7);
                        if (!there[2 * sb + (i >> 3)] || k > hi[b] || k < lo[b]) s[b][sb][i] = kNegInf;
                    }
            }
            float mx = s[b][0][0];
#pragma unroll
            for (int sb = 0; sb < 2; ++sb)
#pragma unroll
                for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[b][sb][i]);
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            if (__any((mx - m[b]) * c > 3.f)) {
                const float mn = fmaxf(m[b], mx);
                const float alpha = __builtin_amdgcn_exp2f((m[b] - (mn == kNegInf ? 0.f : mn)) * c);
                m[b] = mn;
                l[b] *= alpha;
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[b][d][i] *= alpha;
            }
            const float mc = (m[b] == kNegInf ? 0.f : m[b] * c) - kBias<E>;
            float sum = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float p[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    p[j] = __builtin_amdgcn_exp2f(fmaf(s[b][q >> 1][8 * (q & 1) + j], c, -mc));
                    sum += p[j];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) pf[b][q][j] = pack16<E>(p[2 * j], p[2 * j + 1]);
            }
            l[b] += sum;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            u32x4 keep;
            if constexpr (EDGE) {
                const int k = k0 + 16 * q + 8 * lh;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool x0 = there[q] && k + 2 * j >= t.kmin && k + 2 * j <= t.kmax;
                    const bool x1 = there[q] && k + 2 * j + 1 >= t.kmin && k + 2 * j + 1 <= t.kmax;
                    keep[j] = (x0 ? 0xFFFFu : 0u) | (x1 ? 0xFFFF0000u : 0u);
                }
            }
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                u32x4 v = *reinterpret_cast<const u32x4*>(&vbuf[buf][vaddr[q] + d * 4096]);
                if constexpr (EDGE) v &= keep;
#pragma unroll
                for (int b = 0; b < RB; ++b) o[b][d] = E::mfma32(v, pf[b][q], o[b][d]);
            }
        }
    };

    bool bad = false, bad_n = false;
    if (begin < end) {
        pages(begin);
        bad_n = stage(begin, 0);
        if (begin + 1 < end) pages(begin + 1);
    }
    for (int kt = begin; kt < end; ++kt) {
        const int buf = (kt - begin) & 1;
        __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): this wave's part of the tile is in LDS
        __syncthreads();
        bad = bad_n;
        if (kt + 1 < end) {
            bad_n = stage(kt + 1, buf ^ 1);
            if (kt + 2 < end) pages(kt + 2);
        }
        const int k0 = kt * kKT;
        if (k0 < t.full_lo || k0 + kKT - 1 > t.full_hi || bad) compute(kt, buf, std::true_type{});
        else compute(kt, buf, std::false_type{});
    }

#pragma unroll
    for (int b = 0; b < RB; ++b) {
        l[b] += __shfl_xor(l[b], 32);
        const int rho = t.rho0 + 32 * (RB * wave + b) + lr;
        const int i = rho / a.g, hh = rho - i * a.g;
        if (i >= t.n) continue;
        const int head = hk * a.g + hh;
        const int64_t rowi = int64_t(t.c0 + i) * a.heads + head;
        if (a.nsplit > 1) {
            float* dst = a.opart + (rowi * a.nsplit + split) * D;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int at = 32 * d + 8 * j + 4 * lh;
                    if (FULL || at < D)
                        *reinterpret_cast<f32x4*>(dst + at) =
                            f32x4{o[b][d][4 * j], o[b][d][4 * j + 1], o[b][d][4 * j + 2], o[b][d][4 * j + 3]};
                }
            if (lh == 0) {
                a.ml[(rowi * a.nsplit + split) * 2] = m[b];
                a.ml[(rowi * a.nsplit + split) * 2 + 1] = l[b];
            }
        } else {
            const float inv = l[b] == 0.f ? 0.f : 1.f / l[b];  // NaN stays NaN
            uint16_t* dst = a.y + (t.c0 + i) * a.ld_y + int64_t(head) * D;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int at = 32 * d + 8 * j + 4 * lh;
                    if (FULL || at < D)
                        *reinterpret_cast<u32x2*>(dst + at) =
                            u32x2{pack16<E>(o[b][d][4 * j] * inv, o[b][d][4 * j + 1] * inv),
                                  pack16<E>(o[b][d][4 * j + 2] * inv, o[b][d][4 * j + 3] * inv)};
                }
            if (lh == 0 && a.lse)
                a.lse[rowi] = l[b] == 0.f ? kNegInf
                                          : fmaf(m[b], a.scale, logf(l[b]) - kBias<E> * 0.6931471805599453f);
        }
    }
}

template <class E, int DP>
void launch_dp(const AttnArgs& a, int rb, unsigned blocks, hipStream_t s) {
    if (a.D == DP) {
        if (rb == 1) k_attn_tile<E, DP, 1, true><<<blocks, 256, 0, s>>>(a);
        else k_attn_tile<E, DP, 2, true><<<blocks, 256, 0, s>>>(a);
    } else {
        if (rb == 1) k_attn_tile<E, DP, 1, false><<<blocks, 256, 0, s>>>(a);
        else k_attn_tile<E, DP, 2, false><<<blocks, 256, 0, s>>>(a);
    }
}

template <class E>
void launch_e(const AttnArgs& a, int rb, unsigned blocks, hipStream_t s) {
    if (a.D <= 64) launch_dp<E, 64>(a, rb, blocks, s);
    else if (a.D <= 128) launch_dp<E, 128>(a, rb, blocks, s);
    else launch_dp<E, 256>(a, rb, blocks, s);
}

}  // namespace

void launch_attn_tile(const AttnArgs& a, int dtype, int rb, int tiles, hipStream_t s) {
    const unsigned blocks = unsigned(tiles) * a.kv_heads * a.nsplit;
    if (dtype == VQMLP_F16) launch_e<F16>(a, rb, blocks, s);
    else launch_e<BF16>(a, rb, blocks, s);
}

}  // namespace vqmlp
