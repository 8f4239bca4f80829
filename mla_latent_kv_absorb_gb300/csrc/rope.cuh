// rope.cuh -- rotary positions on part of a head: the angle in fixed point and the rows' rotation.
//
// Angle: turns per position are a 64-bit fraction, so position * step modulo 2^64 is the fraction
// of a turn exactly, at any position (a product in fp32 would lose it: one ulp of 10^6 radians is
// 0.06).  Its top 32 bits, as a signed number of half turns in [-1, 1), are within 2^-33 turn of
// it and go to sincospi in fp32 (another 2^-25 of a half turn).
//
// Rows: one unit of a head's row is 16 bytes (or one element or pair, where pointers, strides or
// sizes do not allow that).  Units of the rotated part come first: an interleaved unit holds whole
// pairs, a half-layout unit is the two 16-byte pieces i and i + dim / 2; the other units copy.
// A thread takes the same unit of R heads of one token, so that its sines and cosines serve R rows.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/mla.h"
#include "ptx.cuh"

namespace mla::rope {

constexpr int kThreads = 256;

// cos and sin (times m) of position * step turns.
__device__ __forceinline__ void turn(int32_t position, uint64_t step, float m, float& c, float& s)
{
    const uint64_t phase = (uint64_t)(int64_t)position * step + 0x80000000ull;  // rounded to 2^-32 turn
    const float half_turns = __int2float_rn((int32_t)(phase >> 32)) * 0x1p-31f;
    sincospif(half_turns, &s, &c);
    c *= m;
    s *= m;
}

__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_float(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }

// N elements as one load or store (16 bytes), or element by element.  Loads go through L2: the
// kernel may have been started while the kernel that writes x still ran.
template <typename T, int N>
struct Piece {
    static constexpr bool kVector = N * sizeof(T) == 16;
    alignas(kVector ? 16 : sizeof(T)) T v[N];
    __device__ __forceinline__ void load(const T* p)
    {
        if constexpr (kVector) {
            *reinterpret_cast<uint4*>(v) = __ldcg(reinterpret_cast<const uint4*>(p));
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = __ldcg(p + i);
        }
    }
    __device__ __forceinline__ void store(T* p) const
    {
        if constexpr (kVector) {
            *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) p[i] = v[i];
        }
    }
};

struct Rows {
    const void* x;
    int64_t x_token, x_head;  // strides in elements
    void* out;
    int64_t out_token, out_head;
    void* rest;  // NULL: the other elements go to out, at their place
    int64_t rest_token, rest_head;
    const int32_t* positions;
    int32_t heads, groups;  // groups = tokens * heads / R
    int32_t dim, offset;
    int32_t rot_units, units;  // units == rot_units: nothing to copy (in place)
    int32_t lanes;             // groups per block
};

// The pieces of one group (R heads of one token): units first, first + stride, ...
template <typename T, int V, bool kHalf, int R>
__device__ __forceinline__ void rotate_group(const Rows& a, const mla_rope_config& cfg, int group, int first,
                                             int stride)
{
    constexpr int kPairs = kHalf ? V : (V > 1 ? V / 2 : 1);  // pairs of a unit
    constexpr int kPiece = kHalf ? V : 2 * kPairs;           // consecutive elements
    const int per_token = a.heads / R;
    const int token = group / per_token, head = (group - token * per_token) * R;
    const T* x = static_cast<const T*>(a.x) + token * a.x_token + head * a.x_head;
    for (int u = first; u < a.units; u += stride) {
        if (u < a.rot_units) {
            Piece<T, kPiece> p[R], q[R];  // q: the second half's pieces (half layout)
            const T* src = x + a.offset + u * kPiece;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                p[r].load(src + r * a.x_head);
                if (kHalf) q[r].load(src + r * a.x_head + a.dim / 2);
            }
            const int32_t position = __ldcg(a.positions + token);
            float c[kPairs], s[kPairs];
#pragma unroll
            for (int i = 0; i < kPairs; ++i) turn(position, cfg.step[u * kPairs + i], cfg.magnitude, c[i], s[i]);
            T* dst = static_cast<T*>(a.out) + token * a.out_token + head * a.out_head + (a.rest ? 0 : a.offset) +
                     u * kPiece;
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    T& e0 = kHalf ? p[r].v[i] : p[r].v[2 * i];
                    T& e1 = kHalf ? q[r].v[i] : p[r].v[(2 * i + 1) % kPiece];
                    const float x0 = as_float(e0), x1 = as_float(e1);
                    e0 = from_float<T>(x0 * c[i] - x1 * s[i]);
                    e1 = from_float<T>(x0 * s[i] + x1 * c[i]);
                }
                p[r].store(dst + r * a.out_head);
                if (kHalf) q[r].store(dst + r * a.out_head + a.dim / 2);
            }
        } else {
            const int j = (u - a.rot_units) * V;              // place among the other elements
            const int at = j < a.offset ? j : j + a.dim;      // place in the head
            Piece<T, V> p[R];
#pragma unroll
            for (int r = 0; r < R; ++r) p[r].load(x + at + r * a.x_head);
            T* dst = a.rest ? static_cast<T*>(a.rest) + token * a.rest_token + head * a.rest_head + j
                            : static_cast<T*>(a.out) + token * a.out_token + head * a.out_head + at;
            const int64_t step = a.rest ? a.rest_head : a.out_head;
#pragma unroll
            for (int r = 0; r < R; ++r) p[r].store(dst + r * step);
        }
    }
}

// The groups of block `block`: its threads are a.lanes groups of min(units, kThreads) threads.
template <typename T, int V, bool kHalf, int R>
__device__ __forceinline__ void rotate_block(const Rows& a, const mla_rope_config& cfg, int block)
{
    const int width = a.units < kThreads ? a.units : kThreads;
    const int lane = threadIdx.x / width;
    const int64_t group = (int64_t)block * a.lanes + lane;
    if (lane < a.lanes && group < a.groups)
        rotate_group<T, V, kHalf, R>(a, cfg, (int)group, threadIdx.x - lane * width, width);
}

template <typename T, int V, bool kHalf, int R>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Rows a,
                                                        const __grid_constant__ mla_rope_config cfg)
{
    dev::griddep_wait();
    rotate_block<T, V, kHalf, R>(a, cfg, blockIdx.x);
}

}  // namespace mla::rope
