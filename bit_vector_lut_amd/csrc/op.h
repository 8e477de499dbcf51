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
