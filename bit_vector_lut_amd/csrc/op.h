// op.h -- shared by the operators around the MLP (norm.hip, pages.hip, attn.hip, linear.hip):
// element types, 8-element chunks and the host half's argument checks.
#pragma once
#include "device.h"
#include "internal.h"
#include "vqmlp.h"

namespace vqmlp {

typedef __bf16 bhalf8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Conversions and matrix-core steps of the two 16-bit types.  Every float to 16-bit conversion
// rounds to nearest even; the hardware does both.
struct F16 {
    typedef _Float16 T;
    static __device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
        typedef _Float16 half2 __attribute__((ext_vector_type(2)));
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(half2, a), __builtin_bit_cast(half2, b), c, false);
    }
    static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                      __builtin_bit_cast(half8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a),
                                                      __builtin_bit_cast(half8, b), c, 0, 0, 0);
    }
};
struct BF16 {
    typedef __bf16 T;
    static __device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
        typedef __bf16 bhalf2 __attribute__((ext_vector_type(2)));
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bhalf2, a), __builtin_bit_cast(bhalf2, b), c, false);
    }
    static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bhalf8, a),
                                                       __builtin_bit_cast(bhalf8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bhalf8, a),
                                                       __builtin_bit_cast(bhalf8, b), c, 0, 0, 0);
    }
};

template <class E>
__device__ __forceinline__ float lo16(uint32_t w) {
    return (float)__builtin_bit_cast(typename E::T, (uint16_t)w);
}
template <class E>
__device__ __forceinline__ float hi16(uint32_t w) {
    return (float)__builtin_bit_cast(typename E::T, (uint16_t)(w >> 16));
}
template <class E>
__device__ __forceinline__ uint32_t bits16(float f) {
    return __builtin_bit_cast(uint16_t, (typename E::T)f);
}
template <class E>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
    typedef typename E::T t2 __attribute__((ext_vector_type(2)));
    t2 v = {(typename E::T)a, (typename E::T)b};
    return __builtin_bit_cast(uint32_t, v);
}

// Sum / maximum over the 64 lanes, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// A value that all lanes share, in a scalar register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
// 16 bytes per lane from base + off (or src) to LDS, lane after lane from byte `at` on, without
// passing registers.  As the compiler's builtin it would make every later LDS read wait for all
// loads in flight, since the two might meet; here the caller's own wait and barrier order them.  m0
// has no other use in kernels that neither index registers nor send messages.
__device__ __forceinline__ void load_lds16(const void* base, uint32_t off, uint32_t at) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %0"
                 :: "s"(base), "v"(off), "s"(uniform(at)) : "memory");
}
__device__ __forceinline__ void load_lds16(const void* src, uint32_t at) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :: "v"(src), "s"(uniform(at)) : "memory");
}
// All of this wave's loads are done.
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ uint32_t lds_byte(const void* p) {
    return __builtin_amdgcn_readfirstlane(
        uint32_t(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) uint8_t*)p)));
}
// f(0), f(1), .., f(N - 1) with the number known at compile time
template <class F, int... Z>
__device__ __forceinline__ void each(F&& f, std::integer_sequence<int, Z...>) {
    (f(std::integral_constant<int, Z>{}), ...);
}
// x as if it were new here: what is made of it in a loop is made there and holds no registers across it
__device__ __forceinline__ int fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// ---- decays and units

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMinG = -80.f;  // e^-80 = 2e-35: nothing of the state before survives it in FP32

// e^x to about two roundings: the hardware's 2^h with h = x log2 e, and what h lost as a factor 1 + r.
__device__ __forceinline__ float exp_f32(float x) {
    const float h = x * kLog2e;
    const float r = fmaf(x, kLog2e, -h) + x * float(1.4426950408889634 - double(kLog2e));
    return __builtin_amdgcn_exp2f(h) * fmaf(r, kLn2, 1.f);
}

// The log of a decay from kMinG on; NaN stays NaN.
__device__ __forceinline__ float bounded(float g) { return g < kMinG ? kMinG : g; }

// Sum over the 2^n lanes of a head, n up to 5, for several of them at once.
template <int N>
__device__ __forceinline__ void head_sums(float (&v)[N], int lanes) {
    auto step = [&](auto ctrl) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            v[j] += __builtin_bit_cast(
                float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v[j]), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    if (lanes > 1) step(std::integral_constant<int, 0xB1>{});   // the neighbour
    if (lanes > 2) step(std::integral_constant<int, 0x4E>{});   // the other two of four
    if (lanes > 4) step(std::integral_constant<int, 0x141>{});  // the other four of eight
    if (lanes > 8) step(std::integral_constant<int, 0x140>{});  // the other eight of a row
    if (lanes > 16)
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] += __shfl_xor(v[j], 16);
}

// Prefix over the 64 lanes with data-parallel moves: within rows of 16 lanes, then across them.
template <class T, class F>
__device__ __forceinline__ T lane_scan(T v, T none, F&& op) {
    auto step = [&](auto ctrl, auto rows) __attribute__((always_inline)) {
        struct Words { int w[sizeof(T) / 4]; };
        Words n = __builtin_bit_cast(Words, none);
        const Words x = __builtin_bit_cast(Words, v);
#pragma unroll
        for (size_t i = 0; i < sizeof(T) / 4; ++i)
            n.w[i] = __builtin_amdgcn_update_dpp(n.w[i], x.w[i], decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
        v = op(v, __builtin_bit_cast(T, n));
    };
    typedef std::integral_constant<int, 0xF> all;
    step(std::integral_constant<int, 0x111>{}, all{});  // from 1, 2, 4 and 8 lanes below in the row
    step(std::integral_constant<int, 0x112>{}, all{});
    step(std::integral_constant<int, 0x114>{}, all{});
    step(std::integral_constant<int, 0x118>{}, all{});
    step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});  // a row's last lane to the next row
    step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});  // lane 31 to the upper half
    return v;
}
// Maximum over the lanes with the same lane % 16, in all of them.  The operands of a swap are two values to
// the compiler, which takes both results for one otherwise.
__device__ __forceinline__ float column_max(float v) {
    uint32_t x = __builtin_bit_cast(uint32_t, v);  // not negative: the bits are in the values' order
    const auto a = __builtin_amdgcn_permlane32_swap(x, uint32_t(fresh(int(x))), false, false);
    x = max(uint32_t(a[0]), uint32_t(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(x, uint32_t(fresh(int(x))), false, false);
    return __builtin_bit_cast(float, max(uint32_t(b[0]), uint32_t(b[1])));
}

// 2^e, e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __builtin_bit_cast(float, uint32_t(e + 127) << 23); }
// Exponent of |x| (floor of log2), -127 for zero and subnormals.
__device__ __forceinline__ int expo(float x) {
    return int((__builtin_bit_cast(uint32_t, x) >> 23) & 0xFF) - 127;
}

// ---- packed requests: first rows, state slots

// What the operators with a state per request share.
struct Packed {
    const int32_t *cu, *ctx, *index;
    int T, R, n_states;
};
__device__ __forceinline__ int packed_row(const Packed& p, int r) { return min(max(p.cu[r], 0), p.T); }
// The state slot of a request, or -1, and whether it starts from what the slot holds.
__device__ __forceinline__ int packed_slot(const Packed& p, int r, bool* old) {
    int s = p.index ? p.index[r] : r;
    if (uint32_t(s) >= uint32_t(p.n_states)) s = -1;
    *old = s >= 0 && (!p.ctx || p.ctx[r] > 0);
    return s;
}

// Units of at most L tokens of all requests in one launch without their lengths on the host: request r
// owns unit numbers floor(cu[r] / L) + r and on (enough for ceil(n / L), and one where n is 0); number R
// owns the rows behind the last.  T / L + R + 1 numbers in all.
struct PackedUnit {
    int r, c0, n, seg, nseg, first;  // request, its first row and tokens; unit of it, units; its first's number
};
// For a whole wave.  The owner of number x is found 64 requests a step; numbers of nobody give false.
__device__ __forceinline__ bool packed_unit(const Packed& p, int L, int x, PackedUnit& u) {
    const int lane = threadIdx.x & 63;
    int r = 0;
    for (int step = p.R >= 4096 ? 4096 : p.R >= 64 ? 64 : 1; step; step /= 64) {
        const int i = r + lane * step;
        const int owned = __popcll(__ballot(i <= p.R && packed_row(p, min(i, p.R)) / L + i <= x));
        r += max(0, owned - 1) * step;
    }
    u.r = r;
    u.c0 = packed_row(p, r);
    const int c1 = r < p.R ? packed_row(p, r + 1) : p.T;
    u.n = max(0, c1 - u.c0);
    u.first = u.c0 / L + r;
    u.seg = x - u.first;
    u.nseg = max(1, (u.n + L - 1) / L);
    return u.seg >= 0 && u.seg < u.nseg;
}

// ---- host half

inline bool op_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool op_dtype16(int d) { return d == VQMLP_F16 || d == VQMLP_BF16; }

#define OP_FAIL(st, ...) \
    return static_cast<vqmlp_status>(vqmlp::set_last_error(st, __VA_ARGS__))
#define OP_REQUIRE(cond, ...) \
    do { if (!(cond)) OP_FAIL(VQMLP_ERR_INVALID_ARG, __VA_ARGS__); } while (0)

inline vqmlp_status op_ok() { return static_cast<vqmlp_status>(set_last_error(VQMLP_OK, "%s", "")); }

inline vqmlp_status op_launched(const char* what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) OP_FAIL(VQMLP_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
    return op_ok();
}

}  // namespace vqmlp
