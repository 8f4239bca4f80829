// append.cuh -- what one warp writes of one token into the paged latent cache: the slot check and
// the latent's 512 values as they are (bf16), as e4m3 codes with a scale per token, or as an NVFP4
// row.  Shared by mla_append_kv (append.cu) and mla_rope_append_kv (rope.cu), whose bf16 and
// e4m3 latents are therefore the same bit for bit.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/mla.h"

namespace mla::append {

constexpr int kWarps = 8;  // tokens per CTA

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// e4m3 codes of (lo, hi): round to nearest, ties to even, magnitudes past 448 give 448 with
// their sign (the hardware conversion).  lo lands in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// e2m1 codes of (lo, hi): round to nearest, ties to even, magnitudes past 6 give 6 with their sign
// (the hardware conversion); lo lands in the low nibble.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// Value of an e4m3 code (exact: through f16).
__device__ __forceinline__ float e4m3_value(uint32_t code)
{
    uint32_t h2;
    const uint16_t c = (uint16_t)(code & 0xFFu);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
    return __half2float(__ushort_as_half((unsigned short)(h2 & 0xFFFFu)));
}

// Slot of token i, or -1 when the token is skipped (negative slot, or out of the pool: then
// the error bit is set).
template <bool kLate = false>
__device__ __forceinline__ int64_t token_slot(const int32_t* slots, int64_t i, int64_t num_slots, uint32_t* dev_error,
                                              int lane)
{
    const int32_t slot = kLate ? __ldcg(slots + i) : __ldg(slots + i);
    if (slot < 0) return -1;
    if (slot >= num_slots) {
        if (lane == 0) atomicOr(dev_error, MLA_DEVERR_BAD_SLOT);
        return -1;
    }
    return slot;
}

// Input rows: through the read-only path, or (kLate) through L2, for kernels that may have been
// started while the kernel that writes the rows was still running.
template <bool kLate>
__device__ __forceinline__ uint4 load_row16(const uint4* p)
{
    return kLate ? __ldcg(p) : __ldg(p);
}

// bf16 cache: the latent is the first 64 x 16 bytes of the slot's 72 x 16.
template <bool kLate = false>
__device__ __forceinline__ void store_latent_bf16(const uint4* __restrict__ src, int lane, int64_t slot,
                                                  uint4* __restrict__ pool)
{
    uint4* dst = pool + slot * 72;
    const uint4 a = load_row16<kLate>(src + lane), b = load_row16<kLate>(src + 32 + lane);
    dst[lane] = a;
    dst[32 + lane] = b;
}

// The 16 latent values of lane l, [16 l, 16 l + 16), in fp32.
template <bool kLate>
__device__ __forceinline__ void load_latent16(const uint4* __restrict__ src, int lane, float (&v)[16])
{
    const uint4 a = load_row16<kLate>(src + 2 * lane), b = load_row16<kLate>(src + 2 * lane + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        v[2 * k] = bf16_lo(w[k]);
        v[2 * k + 1] = bf16_hi(w[k]);
    }
}

__device__ __forceinline__ float max_abs16(const float (&v)[16])
{
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) m = fmaxf(m, fabsf(v[k]));
    return m;
}

__device__ __forceinline__ float warp_max(float m)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    return m;
}

// FP8 cache: lane l quantises latent elements [16 l, 16 l + 16) and stores their 16 codes.
template <bool kLate = false>
__device__ __forceinline__ void store_latent_fp8(const uint4* __restrict__ src, int lane, int64_t slot,
                                                 uint4* __restrict__ c8, float* __restrict__ scale)
{
    float v[16];
    load_latent16<kLate>(src, lane, v);
    const float amax = warp_max(max_abs16(v));
    const float sigma = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
    uint32_t codes[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float q0 = __fdiv_rn(v[4 * k], sigma), q1 = __fdiv_rn(v[4 * k + 1], sigma);
        const float q2 = __fdiv_rn(v[4 * k + 2], sigma), q3 = __fdiv_rn(v[4 * k + 3], sigma);
        codes[k] = e4m3x2(q0, q1) | (e4m3x2(q2, q3) << 16);
    }
    c8[slot * 32 + lane] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
    if (lane == 0) scale[slot] = sigma;
}

// NVFP4 cache: 288-byte rows, the 512 latent codes (two per byte, value 2j in the low nibble of
// byte j) then 32 e4m3 block scales.  Lane l owns block l, latent values [16 l, 16 l + 16): its
// 8 code bytes and its scale byte.  All arithmetic in fp32 with IEEE division, in the order of the
// format's definition; a block whose scale rounds to zero stores zeros of its values' signs.
// kByProducts: the two constants are applied as products with their fp32 reciprocals, the way
// tensor expressions divide by a number (max|c| / 2688.0 of a GPU tensor): values then differ from
// the quotients' only where a quotient lies at the border between two codes.
template <bool kLate = false, bool kByProducts = false>
__device__ __forceinline__ void store_latent_nvfp4(const uint4* __restrict__ src, int lane, int64_t slot,
                                                   uint8_t* __restrict__ rows, float* __restrict__ scale)
{
    constexpr int kRowBytes = 512 / 2 + 512 / 16;
    float v[16];
    load_latent16<kLate>(src, lane, v);
    const float bmax = max_abs16(v), amax = warp_max(bmax);
    const float over = kByProducts ? __fmul_rn(amax, 1.f / 2688.f) : __fdiv_rn(amax, 2688.f);
    const float sigma = amax > 0.f ? over : 1.f;
    const float sixes = __fdiv_rn(bmax, sigma);
    const uint32_t s8 = e4m3x2(kByProducts ? __fmul_rn(sixes, 1.f / 6.f) : __fdiv_rn(sixes, 6.f), 0.f) & 0xFFu;
    const float den = __fmul_rn(sigma, e4m3_value(s8));
    uint32_t code[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        uint32_t byte;
        if (den == 0.f)
            byte = (signbit(v[2 * k]) ? 0x8u : 0u) | (signbit(v[2 * k + 1]) ? 0x80u : 0u);
        else
            byte = e2m1x2(__fdiv_rn(v[2 * k], den), __fdiv_rn(v[2 * k + 1], den));
        code[k >> 2] |= byte << (8 * (k & 3));
    }
    uint8_t* row = rows + slot * kRowBytes;
    *reinterpret_cast<uint2*>(row + 8 * lane) = make_uint2(code[0], code[1]);
    row[256 + lane] = (uint8_t)s8;
    if (lane == 0) scale[slot] = sigma;
}

}  // namespace mla::append
