// attn.h -- shared by the attention kernels (attn.hip, attn_tile.hip): arguments, row tiles of the
// packed requests, element-type constants.
#pragma once
#include "op.h"

namespace vqmlp {

constexpr float kNegInf = -__builtin_inff();
constexpr int kMaxSplit = 64;

struct AttnArgs {
    const uint16_t* q;
    uint16_t* y;
    float* lse;
    const uint16_t *kc, *vc;
    const int32_t *table, *cu, *kv_len;
    float* opart;  // [row][split][D], row = token * heads + head (split launches only)
    float* ml;     // [row][split][2]: maximum of the scores, sum (-1: this split has no keys and wrote
                   // nothing; in split 0: the row is done)
    int64_t ld_table, ld_q, ld_y;
    int T, R, heads, kv_heads, g, D, shift, n_pages, window, nsplit, split_tiles;
    int width;     // pages per table row
    float scale;
};

// exp2 of a difference to the maximum: fp16 probabilities carry a factor 2^12, so that keys down to
// 2^-36 of the largest still count (binary16 ends at 2^-24; 2^12 times any sum of them stays far
// inside fp32).  bfloat16 has the range by itself.
template <class E>
constexpr float kBias = __is_same(E, F16) ? 12.f : 0.f;

struct Tile {       // what one workgroup works on
    int r, n;       // request (R: the rows behind the last request), its new tokens
    int c0;         // its first row
    int rho0;       // first packed row of the tile
    int kv;         // keys of the request
    int kmin, kmax; // keys seen by any row of the tile
    int full_lo, full_hi;  // keys seen by every row of the tile
};

// Row tiles of all requests in one launch without their lengths on the host: request r owns tile
// numbers floor(cu[r] g / MT) + r and on, which is always enough for ceil(n g / MT) tiles, and
// the numbers left over return.  Every wave looks the request up for itself, 64 at a time.
template <int MT>
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int x, Tile& t) {
    const int lane = threadIdx.x & 63;
    auto row = [&](int r) { return min(max(a.cu[r], 0), a.T); };
    auto start = [&](int c, int r) { return int(int64_t(c) * a.g / MT) + r; };
    int count = 0;
    for (int r0 = 0; r0 <= a.R; r0 += 64) {
        const int r = r0 + lane;
        const bool le = r <= a.R && start(row(r), r) <= x;
        count += __popcll(__ballot(le));
    }
    t.r = max(0, count - 1);
    t.c0 = row(t.r);
    const int c1 = t.r < a.R ? row(t.r + 1) : a.T;
    t.n = c1 - t.c0;
    t.rho0 = (x - start(t.c0, t.r)) * MT;
    if (t.rho0 < 0 || int64_t(t.rho0) >= int64_t(t.n) * a.g) return false;
    t.kv = t.r < a.R ? max(a.kv_len[t.r], 0) : 0;
    const int i0 = t.rho0 / a.g;
    const int i1 = int(min(int64_t(t.rho0) + MT - 1, int64_t(t.n) * a.g - 1) / a.g);
    const int p0 = t.kv - t.n + i0, p1 = t.kv - t.n + i1;
    const int cap = a.width << a.shift;
    t.kmax = t.r < a.R ? min(p1, cap - 1) : -1;
    t.kmin = a.window ? max(0, p0 - a.window + 1) : 0;
    t.full_hi = min(p0, cap - 1);
    t.full_lo = a.window ? max(0, p1 - a.window + 1) : 0;
    return true;
}

// The key tiles of a split: a request of up to split_tiles of them is done in one, whatever the others
// need.  `used` splits have keys; the last one takes what is left.
struct Split {
    int begin, end, used;
};
__device__ __forceinline__ Split key_split(const AttnArgs& a, const Tile& t, int split, int shift) {
    const int kt0 = t.kmin >> shift;
    const int nt = t.kmax >= t.kmin ? (t.kmax >> shift) + 1 - kt0 : 0;
    Split s;
    s.used = max(1, min(a.nsplit, (nt + a.split_tiles - 1) / a.split_tiles));
    s.begin = kt0 + min(nt, split * a.split_tiles);
    s.end = kt0 + (split == a.nsplit - 1 ? nt : min(nt, (split + 1) * a.split_tiles));
    return s;
}
// What the join reads of a row besides the sums themselves.
__device__ __forceinline__ void put_ml(const AttnArgs& a, int64_t row, int split, const Split& s, float m, float l) {
    float* ml = a.ml + row * a.nsplit * 2;
    ml[2 * split] = m;
    ml[2 * split + 1] = s.used == 1 ? -1.f : l;
    if (split == 0 && s.used > 1)
        for (int i = s.used; i < a.nsplit; ++i) ml[2 * i + 1] = -1.f;
}

// Many rows (attn_tile.hip).
constexpr int kAttnTileRows = 128;
void launch_attn_tile(const AttnArgs& a, int dtype, bool few, int tiles, hipStream_t s);

}  // namespace vqmlp
