// rope.cuh -- rotary positions on part of a head: the angle in fixed point and the rows' rotation.
//
// Angle: turns per position are a 64-bit fraction, so position * step modulo 2^64 is the fraction
// of a turn exactly, at any position (a product in fp32 would lose it: one ulp of 10^6 radians is
// 0.06).  Its top 32 bits are within 2^-33 turn of it.  The nearest quarter turn is taken off in
// integers, and sine and cosine of what is left, |x| <= pi / 4, are their Taylor series to x^9 and
// x^10 (the next terms are below 2e-9), so that no range reduction in floats and no special case is
// left (128 heads of 192, 4,096 tokens: 71 us with sincospi of the half turns, 67 us so).
//
// Rows: one unit of a head's row is 16 bytes (or one element or pair, where pointers, strides or
// sizes do not allow that).  Units of the rotated part come first: an interleaved unit holds whole
// pairs, a half-layout unit is the two 16-byte pieces i and i + dim / 2; the other units copy.
// A thread takes the same unit of R heads of one token, so that its sines and cosines and its index
// arithmetic serve R rows (the same 4,096 tokens: 101 us with R = 1, 71 with 2, 60 with 4, 62 with 8
// and 16), and the copying threads are kept apart from the rotating ones (67 -> 59.7 us: 402 MB at
// 99.6 % of the measured copy rate).
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
    const uint32_t turns = (uint32_t)(((uint64_t)(int64_t)position * step + 0x80000000ull) >> 32);  // 2^-32 turn
    const uint32_t quarter = (turns + 0x20000000u) >> 30;
    const float x = __int2float_rn((int32_t)(turns - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi 2^-32
    const float x2 = x * x;
    float sn = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);  // 1 / 9!, -1 / 7!
    sn = fmaf(sn, x2, 8.3333333e-3f);
    sn = fmaf(sn, x2, -1.6666667e-1f);
    sn = fmaf(sn * x2, x, x);
    float cs = fmaf(x2, -2.7557319e-7f, 2.4801587e-5f);  // -1 / 10!, 1 / 8!
    cs = fmaf(cs, x2, -1.3888889e-3f);
    cs = fmaf(cs, x2, 4.1666667e-2f);
    cs = fmaf(cs, x2, -0.5f);
    cs = fmaf(cs, x2, 1.0f);
    const float a = quarter & 1 ? sn : cs, b = quarter & 1 ? cs : sn;
    c = (quarter + 1) & 2 ? -a * m : a * m;
    s = quarter & 2 ? -b * m : b * m;
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

// The groups of block `block`.  The threads of the rotated units come first and the copying ones
// behind them, so that few warps have both kinds.
template <typename T, int V, bool kHalf, int R>
__device__ __forceinline__ void rotate_block(const Rows& a, const mla_rope_config& cfg, int block)
{
    const int tid = threadIdx.x;
    int lane = 0, unit = tid, stride = kThreads;
    if (a.units <= kThreads) {
        const int copying = a.units - a.rot_units, rotating = a.rot_units * a.lanes, i = tid - rotating;
        stride = a.units;
        if (i < 0)
            lane = tid / a.rot_units, unit = tid - lane * a.rot_units;
        else if (copying > 0)
            lane = i / copying, unit = a.rot_units + i - lane * copying;
        else
            lane = a.lanes;  // no part
    }
    const int64_t group = (int64_t)block * a.lanes + lane;
    if (lane < a.lanes && group < a.groups) rotate_group<T, V, kHalf, R>(a, cfg, (int)group, unit, stride);
}

template <typename T, int V, bool kHalf, int R>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Rows a,
                                                        const __grid_constant__ mla_rope_config cfg)
{
    dev::griddep_wait();
    rotate_block<T, V, kHalf, R>(a, cfg, blockIdx.x);
}

}  // namespace mla::rope
