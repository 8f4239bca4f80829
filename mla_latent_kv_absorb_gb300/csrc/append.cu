// append.cu -- mla_append_kv: write new tokens' rows into the paged latent cache (declared in
// include/mla.h).
//
// Each token stores its 512-d latent c_KV and its 64-d rotated RoPE key k_R once ("撕開
// DeepSeek MLA 源碼", section 1); pages hold 64 tokens (section 3).  For the FP8 cache the
// latent is quantised on the way in: one fp32 scale per token, sigma = max|c| / 448, and the
// e4m3 code nearest c / sigma.  For the NVFP4 cache (the page's "NVFP4 quantized gather" names
// the format; the two-level scaling below is this library's reading): sigma = max|c| / 2688 per
// token, one e4m3 scale per 16 latent values, S_b = nearest e4m3 to ((max|c| over the block) /
// sigma) / 6, and the e2m1 code nearest c / (sigma S_b).
//
// One warp per token.  A token is 1152 bytes of bf16 input and at most 1152 bytes of output,
// so the kernel is a few coalesced 16-byte loads and stores per lane; at decode batch sizes it
// is launch-bound and no staging in shared memory or TMA would pay.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdio>

#include "../../include/mla.h"
#include "append.cuh"
#include "nvtx_range.h"

namespace mla {
void set_last_error_text(const char* text);
}

namespace mla::append {

// bf16 cache: row = c_KV (64 x 16 B) then k_R (8 x 16 B), 72 x 16 B per slot.
__global__ void __launch_bounds__(kWarps * 32) append_bf16_kernel(const uint4* __restrict__ c_kv,
                                                                   const uint4* __restrict__ k_r,
                                                                   const int32_t* __restrict__ slots, int n,
                                                                   int64_t num_slots, uint4* __restrict__ pool,
                                                                   uint32_t* dev_error)
{
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (i >= n) return;
    const int64_t slot = token_slot(slots, i, num_slots, dev_error, lane);
    if (slot < 0) return;
    store_latent_bf16(c_kv + i * 64, lane, slot, pool);
    if (lane < 8) pool[slot * 72 + 64 + lane] = __ldg(k_r + i * 8 + lane);
}

__global__ void __launch_bounds__(kWarps * 32) append_fp8_kernel(const uint4* __restrict__ c_kv,
                                                                  const uint4* __restrict__ k_r,
                                                                  const int32_t* __restrict__ slots, int n,
                                                                  int64_t num_slots, uint4* __restrict__ c8,
                                                                  float* __restrict__ scale, uint4* __restrict__ kr,
                                                                  uint32_t* dev_error)
{
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (i >= n) return;
    const int64_t slot = token_slot(slots, i, num_slots, dev_error, lane);
    if (slot < 0) return;
    store_latent_fp8(c_kv + i * 64, lane, slot, c8, scale);
    if (lane < 8) kr[slot * 8 + lane] = __ldg(k_r + i * 8 + lane);
}

__global__ void __launch_bounds__(kWarps * 32) append_nvfp4_kernel(const uint4* __restrict__ c_kv,
                                                                    const uint4* __restrict__ k_r,
                                                                    const int32_t* __restrict__ slots, int n,
                                                                    int64_t num_slots, uint8_t* __restrict__ rows,
                                                                    float* __restrict__ scale, uint4* __restrict__ kr,
                                                                    uint32_t* dev_error)
{
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (i >= n) return;
    const int64_t slot = token_slot(slots, i, num_slots, dev_error, lane);
    if (slot < 0) return;
    store_latent_nvfp4(c_kv + i * 64, lane, slot, rows, scale);
    if (lane < 8) kr[slot * 8 + lane] = __ldg(k_r + i * 8 + lane);
}

}  // namespace mla::append

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

extern "C" MLA_API mla_status mla_append_kv(int32_t num_tokens, const void* c_kv, const void* k_r,
                                            const int32_t* slots, mla_kv_dtype kv_dtype, int32_t num_pool_pages,
                                            void* kv_pool, float* kv_scale, void* kr_pool, uint32_t* dev_error,
                                            void* stream)
{
    const mla::NvtxRange nvtx_range("mla_append_kv");
    using namespace mla::append;
    if (num_tokens < 0 || num_pool_pages <= 0) return MLA_ERR_INVALID_ARG;
    if (kv_dtype != MLA_KV_BF16 && kv_dtype != MLA_KV_FP8_E4M3 && kv_dtype != MLA_KV_NVFP4)
        return MLA_ERR_INVALID_ARG;
    if (num_tokens == 0) return MLA_OK;
    if (!c_kv || !k_r || !slots || !kv_pool || !dev_error) return MLA_ERR_INVALID_ARG;
    const bool fp8 = kv_dtype != MLA_KV_BF16;  // both quantised caches keep a scale and k_R apart
    if (fp8 && (!kv_scale || !kr_pool)) return MLA_ERR_INVALID_ARG;
    if (!aligned(c_kv, 16) || !aligned(k_r, 16) || !aligned(kv_pool, 16) || !aligned(slots, 4) ||
        !aligned(dev_error, 4) || (fp8 && (!aligned(kr_pool, 16) || !aligned(kv_scale, 4))))
        return MLA_ERR_ALIGNMENT;
    const int64_t num_slots = (int64_t)num_pool_pages * MLA_PAGE_SIZE;
    const dim3 grid((unsigned)(((int64_t)num_tokens + kWarps - 1) / kWarps)), block(kWarps * 32);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uint4* src_c = static_cast<const uint4*>(c_kv);
    const uint4* src_r = static_cast<const uint4*>(k_r);
    if (kv_dtype == MLA_KV_NVFP4)
        append_nvfp4_kernel<<<grid, block, 0, s>>>(src_c, src_r, slots, num_tokens, num_slots,
                                                   static_cast<uint8_t*>(kv_pool), kv_scale,
                                                   static_cast<uint4*>(kr_pool), dev_error);
    else if (fp8)
        append_fp8_kernel<<<grid, block, 0, s>>>(src_c, src_r, slots, num_tokens, num_slots,
                                                 static_cast<uint4*>(kv_pool), kv_scale, static_cast<uint4*>(kr_pool),
                                                 dev_error);
    else
        append_bf16_kernel<<<grid, block, 0, s>>>(src_c, src_r, slots, num_tokens, num_slots,
                                                  static_cast<uint4*>(kv_pool), dev_error);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        char msg[200];
        snprintf(msg, sizeof msg, "append kernel launch: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
        mla::set_last_error_text(msg);
        return MLA_ERR_CUDA;
    }
    return MLA_OK;
}
