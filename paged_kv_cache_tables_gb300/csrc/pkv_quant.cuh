// The cache held in 8 bits: e4m3 codes, converted two at a time, and the scale
// of a block.  Inline PTX, written for this library.
#pragma once

#include <stdint.h>

#include <cmath>

#include "pkv_device.cuh"

namespace pkv {

constexpr float kCodeMax = 448.f;   // the largest e4m3 value

// Two e4m3 codes (the low byte first) as an fp16 pair; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(r)
        : "r"(codes));
    return r;
}

// Four codes as two pairs.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t codes, uint32_t &first, uint32_t &second) {
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(first), "=r"(second)
        : "r"(codes));
}

// The codes next to four values (ties to even; beyond 448 the code of 448; NaN
// stays NaN), `a` in the lowest byte.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// The same in e5m2 (beyond 57,344 its code), and back.
__device__ __forceinline__ uint32_t to_e5m2x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e5m2x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e5m2x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

__device__ __forceinline__ void e5m2x4_to_f16x4(uint32_t codes, uint32_t &first, uint32_t &second) {
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e5m2x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e5m2x2 %1, hi;\n\t}"
        : "=r"(first), "=r"(second)
        : "r"(codes));
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t pair) { return __half22float2(*reinterpret_cast<__half2 *>(&pair)); }

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// log2 x (hardware approximation).
__device__ __forceinline__ float log2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A 16-bit pair as floats.
template <typename T>
__device__ __forceinline__ float2 pair_to_f32(uint32_t w) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else
        return f16x2_to_f32(w);
}

// The scale for values of magnitude at most a (finite): the least power of two
// s >= 2^-60 with a <= 448 s.  448 = 1.75 * 2^8.  A power of two, so that x / s
// and a later change of scale are exact (short of e4m3's subnormals): e4m3 is
// a floating-point format, and loses no precision to the up to one binade of
// range that a finer scale would use.
__device__ __forceinline__ float block_scale(float a, int least = -60) {
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)max(e, 127 + least) << 23);
}

// What both attention calls refuse.
inline int quant_attention_refusal(int num_seqs, int num_blocks, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                   int max_blocks_per_seq, int window, int num_sinks, float scale, int dtype, int out_dtype) {
    if (num_seqs < 0 || num_blocks <= 0 || num_kv_heads <= 0 || num_q_heads <= 0 || max_blocks_per_seq <= 0 || window <= 0 ||
        num_sinks < 0)
        return PKV_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    if (num_q_heads > 1 << 16) return PKV_ERR_UNSUPPORTED;   // (offsets in a unit's rows of queries are 32-bit)
    if (num_q_heads / num_kv_heads > 16 || block_size != 16 || (head_dim != 64 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
    if (dtype != PKV_DTYPE_F16 && dtype != PKV_DTYPE_BF16) return PKV_ERR_UNSUPPORTED;
    if (out_dtype != dtype && out_dtype != PKV_DTYPE_F32) return PKV_ERR_UNSUPPORTED;
    if (!(std::isfinite(scale) && scale > 0.f)) return PKV_ERR_INVALID_ARG;
    if ((int64_t)num_blocks * num_kv_heads * block_size >= (int64_t)1 << 31) return PKV_ERR_UNSUPPORTED;
    if ((int64_t)num_seqs * max_blocks_per_seq >= (int64_t)1 << 31 || max_blocks_per_seq > (1 << 26)) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

}  // namespace pkv
