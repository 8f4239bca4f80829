// w4.cu -- mla_linear_w4: out[r,h,n] = t * sum_k x[r,h,k] W[h,n,k] with W in 4 bits and a scale per
// group of k (declared in include/mla.h).
//
// One warp per output column n of one head and per kRows rows of x: each lane takes 32 consecutive
// k (16 bytes of codes) at a time, and the lanes' sums are joined at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/mla.h"
#include "launch.cuh"
#include "nvtx_range.h"
#include "ptx.cuh"

namespace mla::w4 {

constexpr int kWarps = 8;
constexpr int kRows = 4;

struct Args {
    const __nv_bfloat16* x;
    int64_t x_row, x_head;
    const uint8_t* codes;
    const void* scale;
    const uint8_t* zero;
    __nv_bfloat16* out;
    int64_t out_row, out_head;
    float tensor_scale;
    int rows, n, k, group;
    bool early;  // kernels behind this one may start before it ends (they wait for `out` themselves)
};

__device__ __forceinline__ float e2m1_value(uint32_t code)
{
    const uint32_t m = code & 7u;
    const float a = m < 2u ? 0.5f * (float)m : (float)(2u + (m & 1u)) * (float)(1u << (m >> 1)) * 0.25f;
    return code & 8u ? -a : a;
}

__device__ __forceinline__ float e4m3_value(uint32_t code)
{
    uint32_t h2;
    const uint16_t c = (uint16_t)(code & 0xFFu);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
    return __half2float(__ushort_as_half((unsigned short)(h2 & 0xFFFFu)));
}

template <bool kInt4>
__global__ void __launch_bounds__(kWarps * 32) linear_w4_kernel(const __grid_constant__ Args a)
{
    dev::griddep_wait();
    if (a.early) dev::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, h = blockIdx.y, r0 = blockIdx.z * kRows;
    const int n = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (n >= a.n) return;
    const int64_t row = (int64_t)h * a.n + n;
    const int groups = a.k / a.group;
    float acc[kRows] = {};
    for (int k = 32 * lane; k < a.k; k += 1024) {
        const uint4 c4 = __ldcg(reinterpret_cast<const uint4*>(a.codes + row * (a.k / 2) + k / 2));
        const uint32_t word[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t g = row * groups + (k + 8 * j) / a.group;
            float s, z = 0.f;
            if (kInt4) {
                s = __bfloat162float(__ldcg(static_cast<const __nv_bfloat16*>(a.scale) + g));
                z = a.zero ? (float)__ldcg(a.zero + g) : 8.f;
            } else {
                s = e4m3_value(__ldcg(static_cast<const uint8_t*>(a.scale) + g));
            }
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t code = (word[j] >> (4 * i)) & 15u;
                w[i] = (kInt4 ? (float)code - z : e2m1_value(code)) * s;
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (r0 + r >= a.rows) break;
                const uint4 v = __ldcg(reinterpret_cast<const uint4*>(a.x + (r0 + r) * a.x_row + h * a.x_head + k + 8 * j));
                const uint32_t xv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[r] += dev::bf16_lo(xv[i]) * w[2 * i];
                    acc[r] += dev::bf16_hi(xv[i]) * w[2 * i + 1];
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], off);
        if (lane == 0 && r0 + r < a.rows)
            a.out[(r0 + r) * a.out_row + h * a.out_head + n] = __float2bfloat16_rn(acc[r] * a.tensor_scale);
    }
}

}  // namespace mla::w4

namespace {

mla_status linear_w4(int32_t rows, const void* x, int64_t x_row_stride, int64_t x_head_stride, const mla_w4_weight* w,
                     void* out, int64_t out_row_stride, int64_t out_head_stride, bool early, void* stream)
{
    using namespace mla::w4;
    using mla::is_aligned;
    constexpr int64_t kMaxStride = (int64_t)1 << 40;
    const auto stride_ok = [](int64_t s) { return s >= 0 && s <= kMaxStride; };
    if (rows < 0 || !w || (w->format != MLA_W4_INT4 && w->format != MLA_W4_NVFP4)) return MLA_ERR_INVALID_ARG;
    const bool int4 = w->format == MLA_W4_INT4;
    if (w->heads < 1 || w->n < 1 || w->k < 1 || !std::isfinite(w->tensor_scale)) return MLA_ERR_INVALID_ARG;
    if (int4 ? (w->group != 32 && w->group != 64 && w->group != 128) : w->group != 16) return MLA_ERR_INVALID_ARG;
    if (w->k % w->group || w->k % 32 || (!int4 && w->zero)) return MLA_ERR_INVALID_ARG;
    if (!stride_ok(x_row_stride) || !stride_ok(x_head_stride) || !stride_ok(out_row_stride) || !stride_ok(out_head_stride))
        return MLA_ERR_INVALID_ARG;
    if (rows == 0) return MLA_OK;
    if (!x || !out || !w->codes || !w->scale || x == out) return MLA_ERR_INVALID_ARG;
    if (!mla::distinct_elements(rows, out_row_stride, w->heads, out_head_stride, w->n)) return MLA_ERR_INVALID_ARG;
    if (!is_aligned(x, 16) || !is_aligned(w->codes, 16) || !is_aligned(out, 2) || (int4 && !is_aligned(w->scale, 2)) ||
        (rows > 1 && x_row_stride % 8) || (w->heads > 1 && x_head_stride % 8))
        return MLA_ERR_ALIGNMENT;
    if (w->heads > 65535 || (int64_t)w->heads * w->n >= ((int64_t)1 << 31) || rows > 65535 * kRows)
        return MLA_ERR_UNSUPPORTED;
    Args a = {};
    a.x = static_cast<const __nv_bfloat16*>(x);
    a.x_row = x_row_stride;
    a.x_head = x_head_stride;
    a.codes = static_cast<const uint8_t*>(w->codes);
    a.scale = w->scale;
    a.zero = static_cast<const uint8_t*>(w->zero);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.out_row = out_row_stride;
    a.out_head = out_head_stride;
    a.tensor_scale = w->tensor_scale;
    a.rows = rows;
    a.n = w->n;
    a.k = w->k;
    a.group = w->group;
    a.early = early;
    const dim3 grid((unsigned)((w->n + kWarps - 1) / kWarps), (unsigned)w->heads, (unsigned)((rows + kRows - 1) / kRows));
    return mla::launch_dependent("4-bit product kernel launch", int4 ? linear_w4_kernel<true> : linear_w4_kernel<false>,
                                 grid, dim3(kWarps * 32), 0, stream, a);
}

// The step's per-head products: 128 heads, contiguous rows.
mla_status head_product(int32_t batch, const void* x, const mla_w4_weight* w, int32_t n, int32_t k, void* out,
                        void* stream)
{
    if (batch <= 0 || !w || w->heads != MLA_NUM_HEADS || w->n != n || w->k != k) return MLA_ERR_INVALID_ARG;
    return linear_w4(batch, x, (int64_t)MLA_NUM_HEADS * k, k, w, out, (int64_t)MLA_NUM_HEADS * n, n, true, stream);
}

}  // namespace

extern "C" MLA_API mla_status mla_linear_w4(int32_t rows, const void* x, int64_t x_row_stride, int64_t x_head_stride,
                                            const mla_w4_weight* w, void* out, int64_t out_row_stride,
                                            int64_t out_head_stride, void* stream)
{
    const mla::NvtxRange nvtx_range("mla_linear_w4");
    return linear_w4(rows, x, x_row_stride, x_head_stride, w, out, out_row_stride, out_head_stride, false, stream);
}

extern "C" MLA_API mla_status mla_absorb_q_w4(const void* q_c, const mla_w4_weight* w_uk, void* q_abs, int32_t batch,
                                              void* stream)
{
    const mla::NvtxRange nvtx_range("mla_absorb_q_w4");
    return head_product(batch, q_c, w_uk, MLA_LATENT_DIM, MLA_HEAD_DIM, q_abs, stream);
}

extern "C" MLA_API mla_status mla_out_proj_w4(const void* o_lat, const mla_w4_weight* w_uv, void* out, int32_t batch,
                                              void* stream)
{
    const mla::NvtxRange nvtx_range("mla_out_proj_w4");
    return head_product(batch, o_lat, w_uv, MLA_HEAD_DIM, MLA_LATENT_DIM, out, stream);
}
