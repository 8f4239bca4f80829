// rope.cu -- rotary positions (mla_rope_init, mla_rope) and the cache append that applies them on
// the way (mla_rope_append_kv); declared in include/mla.h.
//
// Both kernels move data once and are bound by HBM when there is much of it and by the launch when
// there is little.  The append is one warp per token, as in append.cu, with one pair of the key per
// lane; the blocks behind the last token split and rotate the queries, so that a decode step needs
// one launch between its projections and its absorb.
//
// Both start early (programmatic dependent launch) and wait for the kernel ahead before they touch
// memory, but let nothing start before they have ended: the decode kernel reads q_R and the cache's
// pages without a wait of its own.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/mla.h"
#include "append.cuh"
#include "launch.cuh"
#include "nvtx_range.h"
#include "rope.cuh"

namespace mla::rope {

struct Append {
    const __nv_bfloat16* c_kv;
    int64_t c_stride;
    const __nv_bfloat16* k_r;
    int64_t k_stride;
    const int32_t* positions;
    const int32_t* slots;
    int32_t n;
    int32_t blocks;  // blocks of the append; the rest rotate queries
    int64_t num_slots;
    void* pool;
    float* scale;
    __nv_bfloat16* kr;
    uint32_t* dev_error;
    bool four;  // the queries in groups of four heads
};

template <int kCache, bool kHalf>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const __grid_constant__ Append a,
                                                               const __grid_constant__ Rows q,
                                                               const __grid_constant__ mla_rope_config cfg)
{
    dev::griddep_wait();
    if ((int)blockIdx.x >= a.blocks) {
        const int block = (int)blockIdx.x - a.blocks;
        if (a.four)
            rotate_block<__nv_bfloat16, 8, kHalf, 4>(q, cfg, block);
        else
            rotate_block<__nv_bfloat16, 8, kHalf, 1>(q, cfg, block);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * append::kWarps + (threadIdx.x >> 5);
    if (i >= a.n) return;
    const int64_t slot = append::token_slot<true>(a.slots, i, a.num_slots, a.dev_error, lane);
    if (slot < 0) return;
    const uint4* c = reinterpret_cast<const uint4*>(a.c_kv + i * a.c_stride);
    __nv_bfloat16* key;  // where the slot's rotated key goes
    if constexpr (kCache == MLA_KV_BF16) {
        append::store_latent_bf16<true>(c, lane, slot, static_cast<uint4*>(a.pool));
        key = static_cast<__nv_bfloat16*>(a.pool) + slot * 576 + 512;
    } else {
        if constexpr (kCache == MLA_KV_FP8_E4M3)
            append::store_latent_fp8<true>(c, lane, slot, static_cast<uint4*>(a.pool), a.scale);
        else
            append::store_latent_nvfp4<true, true>(c, lane, slot, static_cast<uint8_t*>(a.pool), a.scale);
        key = a.kr + slot * 64;
    }
    // lane l: pair l
    const __nv_bfloat16* k = a.k_r + i * a.k_stride;
    float cs, sn;
    turn(__ldcg(a.positions + i), cfg.step[lane], cfg.magnitude, cs, sn);
    if constexpr (kHalf) {
        const float x0 = as_float(__ldcg(k + lane)), x1 = as_float(__ldcg(k + 32 + lane));
        key[lane] = __float2bfloat16_rn(x0 * cs - x1 * sn);
        key[32 + lane] = __float2bfloat16_rn(x0 * sn + x1 * cs);
    } else {
        const uint32_t w = __ldcg(reinterpret_cast<const uint32_t*>(k) + lane);
        const float x0 = dev::bf16_lo(w), x1 = dev::bf16_hi(w);
        reinterpret_cast<uint32_t*>(key)[lane] = dev::pack_bf16x2(x0 * cs - x1 * sn, x0 * sn + x1 * cs);
    }
}

}  // namespace mla::rope

namespace {

using mla::is_aligned;

constexpr int64_t kMaxStride = (int64_t)1 << 40;

bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

bool config_ok(const mla_rope_config* r)
{
    return r && r->dim >= 2 && r->dim <= MLA_ROPE_MAX_DIM && r->dim % 2 == 0 &&
           (r->layout == MLA_ROPE_INTERLEAVED || r->layout == MLA_ROPE_HALF) && std::isfinite(r->magnitude) &&
           r->magnitude > 0.f;
}

// Four heads a thread share one set of sines when that leaves four blocks for every SM; with fewer
// rows than that the launch bounds the call and one head a thread spreads them widest.
bool four_heads(int64_t tokens, int32_t heads, int32_t units)
{
    return heads % 4 == 0 && tokens * heads / 4 * units >= (int64_t)152 * 4 * mla::rope::kThreads;
}

// Units, lanes and blocks for `tokens` rows of heads; a.units and a.heads are set.
int64_t lay_out(mla::rope::Rows* a, int64_t tokens, bool four)
{
    const int64_t groups = tokens * a->heads / (four ? 4 : 1);
    a->groups = (int32_t)groups;
    a->lanes = a->units < mla::rope::kThreads ? mla::rope::kThreads / a->units : 1;
    return (groups + a->lanes - 1) / a->lanes;
}

template <typename T, int V, bool kHalf>
mla_status launch_rope_r(const mla::rope::Rows& a, const mla_rope_config& cfg, int64_t blocks, bool four, void* stream)
{
    using namespace mla::rope;
    return mla::launch_dependent("rope kernel launch", four ? rope_kernel<T, V, kHalf, 4> : rope_kernel<T, V, kHalf, 1>,
                                 dim3((unsigned)blocks), dim3(kThreads), 0, stream, a, cfg);
}

template <typename T>
mla_status launch_rope(const mla::rope::Rows& a, const mla_rope_config& cfg, int64_t blocks, bool four, bool vec,
                       void* stream)
{
    constexpr int V = 16 / sizeof(T);
    if (cfg.layout == MLA_ROPE_HALF)
        return vec ? launch_rope_r<T, V, true>(a, cfg, blocks, four, stream)
                   : launch_rope_r<T, 1, true>(a, cfg, blocks, four, stream);
    return vec ? launch_rope_r<T, V, false>(a, cfg, blocks, four, stream)
               : launch_rope_r<T, 1, false>(a, cfg, blocks, four, stream);
}

}  // namespace

extern "C" MLA_API mla_status mla_rope_init(const mla_rope_options* opts, mla_rope_config* rope)
{
    if (!opts || !rope) return MLA_ERR_INVALID_ARG;
    const int32_t dim = opts->dim;
    const double base = opts->base == 0.0 ? 10000.0 : opts->base;
    const double fast = opts->beta_fast == 0.0 ? 32.0 : opts->beta_fast;
    const double slow = opts->beta_slow == 0.0 ? 1.0 : opts->beta_slow;
    const double factor = opts->factor;
    if (dim < 2 || dim > MLA_ROPE_MAX_DIM || dim % 2) return MLA_ERR_INVALID_ARG;
    if (opts->layout != MLA_ROPE_INTERLEAVED && opts->layout != MLA_ROPE_HALF) return MLA_ERR_INVALID_ARG;
    if (opts->scaling < MLA_ROPE_NONE || opts->scaling > MLA_ROPE_YARN) return MLA_ERR_INVALID_ARG;
    if (!(base > 1.0) || !std::isfinite(base)) return MLA_ERR_INVALID_ARG;
    if (!(opts->magnitude >= 0.0) || !std::isfinite(opts->magnitude) || opts->magnitude > 1e30)
        return MLA_ERR_INVALID_ARG;
    if (opts->inv_freq && opts->scaling != MLA_ROPE_NONE) return MLA_ERR_INVALID_ARG;
    if (opts->scaling == MLA_ROPE_LINEAR && (!(factor > 0.0) || !std::isfinite(factor))) return MLA_ERR_INVALID_ARG;
    if (opts->scaling == MLA_ROPE_YARN && (!(factor >= 1.0) || !std::isfinite(factor) || opts->original_len <= 0 ||
                                           !(slow > 0.0) || !(fast > slow) || !std::isfinite(fast)))
        return MLA_ERR_INVALID_ARG;

    const double kPi = 3.14159265358979323846;
    double low = 0.0, high = 0.0;
    if (opts->scaling == MLA_ROPE_YARN) {
        // the pair index whose frequency turns `turns` times over the trained length
        const auto pair = [&](double turns) {
            return dim * std::log(opts->original_len / (turns * 2.0 * kPi)) / (2.0 * std::log(base));
        };
        low = std::fmax(std::floor(pair(fast)), 0.0);
        high = std::fmin(std::ceil(pair(slow)), dim - 1.0);
    }
    double m = opts->magnitude;
    if (m == 0.0) m = opts->scaling == MLA_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
    mla_rope_config r = {};
    r.dim = dim;
    r.layout = opts->layout;
    r.magnitude = (float)m;
    if (!(r.magnitude > 0.f)) return MLA_ERR_INVALID_ARG;  // underflowed
    for (int i = 0; i < dim / 2; ++i) {
        double f = opts->inv_freq ? opts->inv_freq[i] : std::pow(base, -2.0 * i / dim);
        if (opts->inv_freq && (!(f >= 0.0) || !std::isfinite(f))) return MLA_ERR_INVALID_ARG;
        if (opts->scaling == MLA_ROPE_LINEAR) f /= factor;
        if (opts->scaling == MLA_ROPE_YARN) {
            const double ramp = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
            f = f * (1.0 - ramp) + f / factor * ramp;
        }
        const double turns = f / (2.0 * kPi);
        const double part = turns - std::floor(turns);
        r.step[i] = (uint64_t)std::ldexp(part, 64);  // part < 1 with 53 bits: at most 2^64 - 2^11
    }
    *rope = r;
    return MLA_OK;
}

extern "C" MLA_API mla_status mla_rope(const mla_rope_config* rope, mla_dtype dtype, int32_t num_tokens,
                                       int32_t num_heads, int32_t head_dim, int32_t rot_offset, const void* x,
                                       int64_t x_token_stride, int64_t x_head_stride, void* out,
                                       int64_t out_token_stride, int64_t out_head_stride, void* rest,
                                       int64_t rest_token_stride, int64_t rest_head_stride, const int32_t* positions,
                                       void* stream)
{
    const mla::NvtxRange nvtx_range("mla_rope");
    if (!config_ok(rope) || (dtype != MLA_BF16 && dtype != MLA_FP16 && dtype != MLA_FP32)) return MLA_ERR_INVALID_ARG;
    if (num_tokens < 0 || num_heads < 1 || rot_offset < 0 || head_dim < rope->dim || rot_offset > head_dim - rope->dim)
        return MLA_ERR_INVALID_ARG;
    if (!stride_ok(x_token_stride) || !stride_ok(x_head_stride) || !stride_ok(out_token_stride) ||
        !stride_ok(out_head_stride) || (rest && (!stride_ok(rest_token_stride) || !stride_ok(rest_head_stride))))
        return MLA_ERR_INVALID_ARG;
    if (num_tokens == 0) return MLA_OK;
    if (!x || !out || !positions) return MLA_ERR_INVALID_ARG;
    if ((int64_t)num_tokens * num_heads >= ((int64_t)1 << 31) || head_dim > 65536) return MLA_ERR_UNSUPPORTED;
    const int32_t others = head_dim - rope->dim;
    const bool in_place = out == x;
    if (in_place && (rest || (num_tokens > 1 && x_token_stride != out_token_stride) ||
                     (num_heads > 1 && x_head_stride != out_head_stride)))
        return MLA_ERR_INVALID_ARG;
    if (rest && (others == 0 || rest == x || rest == out)) return MLA_ERR_INVALID_ARG;
    if (!mla::distinct_elements(num_tokens, out_token_stride, num_heads, out_head_stride, rest ? rope->dim : head_dim) ||
        (rest && !mla::distinct_elements(num_tokens, rest_token_stride, num_heads, rest_head_stride, others)))
        return MLA_ERR_INVALID_ARG;
    const int es = dtype == MLA_FP32 ? 4 : 2, V = 16 / es;
    if (!is_aligned(x, es) || !is_aligned(out, es) || !is_aligned(rest, es) || !is_aligned(positions, 4))
        return MLA_ERR_ALIGNMENT;

    const bool half = rope->layout == MLA_ROPE_HALF, copy = !in_place && others > 0;
    const auto pieces = [&](const void* p, int64_t ts, int64_t hs) {
        return is_aligned(p, 16) && (num_tokens == 1 || ts % V == 0) && (num_heads == 1 || hs % V == 0);
    };
    const bool vec = pieces(x, x_token_stride, x_head_stride) && pieces(out, out_token_stride, out_head_stride) &&
                     (!rest || pieces(rest, rest_token_stride, rest_head_stride)) && rot_offset % V == 0 &&
                     rope->dim % (half ? 2 * V : V) == 0 && (!copy || others % V == 0);
    mla::rope::Rows a = {};
    a.x = x;
    a.x_token = x_token_stride;
    a.x_head = x_head_stride;
    a.out = out;
    a.out_token = out_token_stride;
    a.out_head = out_head_stride;
    a.rest = rest;
    a.rest_token = rest_token_stride;
    a.rest_head = rest_head_stride;
    a.positions = positions;
    a.heads = num_heads;
    a.dim = rope->dim;
    a.offset = rot_offset;
    a.rot_units = rope->dim / (vec ? (half ? 2 * V : V) : 2);
    a.units = a.rot_units + (copy ? others / (vec ? V : 1) : 0);
    const bool four = four_heads(num_tokens, num_heads, a.units);
    const int64_t blocks = lay_out(&a, num_tokens, four);
    if (dtype == MLA_BF16) return launch_rope<__nv_bfloat16>(a, *rope, blocks, four, vec, stream);
    if (dtype == MLA_FP16) return launch_rope<__half>(a, *rope, blocks, four, vec, stream);
    return launch_rope<float>(a, *rope, blocks, four, vec, stream);
}

extern "C" MLA_API mla_status mla_rope_append_kv(const mla_rope_config* rope, int32_t num_tokens, const void* c_kv,
                                                 int64_t c_kv_stride, const void* k_r, int64_t k_r_stride,
                                                 const int32_t* positions, const int32_t* slots,
                                                 mla_kv_dtype kv_dtype, int32_t num_pool_pages, void* kv_pool,
                                                 float* kv_scale, void* kr_pool, const void* q,
                                                 int64_t q_token_stride, int64_t q_head_stride, void* q_c, void* q_r,
                                                 uint32_t* dev_error, void* stream)
{
    const mla::NvtxRange nvtx_range("mla_rope_append_kv");
    using namespace mla::rope;
    if (!config_ok(rope) || rope->dim != MLA_ROPE_DIM || num_tokens < 0 || num_pool_pages <= 0)
        return MLA_ERR_INVALID_ARG;
    if (kv_dtype != MLA_KV_BF16 && kv_dtype != MLA_KV_FP8_E4M3 && kv_dtype != MLA_KV_NVFP4)
        return MLA_ERR_INVALID_ARG;
    if (!stride_ok(c_kv_stride) || !stride_ok(k_r_stride) || (q && (!stride_ok(q_token_stride) || !stride_ok(q_head_stride))))
        return MLA_ERR_INVALID_ARG;
    if (num_tokens == 0) return MLA_OK;
    if (!c_kv || !k_r || !positions || !slots || !kv_pool || !dev_error) return MLA_ERR_INVALID_ARG;
    const bool quant = kv_dtype != MLA_KV_BF16;
    if (quant && (!kv_scale || !kr_pool)) return MLA_ERR_INVALID_ARG;
    if (q && (!q_c || !q_r || q_c == q || q_r == q || q_c == q_r)) return MLA_ERR_INVALID_ARG;
    if (!is_aligned(c_kv, 16) || !is_aligned(k_r, 16) || !is_aligned(kv_pool, 16) || !is_aligned(slots, 4) ||
        !is_aligned(positions, 4) || !is_aligned(dev_error, 4) ||
        (num_tokens > 1 && (c_kv_stride % 8 || k_r_stride % 8 || (q && q_token_stride % 8))) ||
        (quant && (!is_aligned(kr_pool, 16) || !is_aligned(kv_scale, 4))) ||
        (q && (!is_aligned(q, 16) || !is_aligned(q_c, 16) || !is_aligned(q_r, 16) || q_head_stride % 8)))
        return MLA_ERR_ALIGNMENT;
    if (num_tokens > (1 << 23)) return MLA_ERR_UNSUPPORTED;

    const bool half = rope->layout == MLA_ROPE_HALF;
    Append a = {};
    a.c_kv = static_cast<const __nv_bfloat16*>(c_kv);
    a.c_stride = c_kv_stride;
    a.k_r = static_cast<const __nv_bfloat16*>(k_r);
    a.k_stride = k_r_stride;
    a.positions = positions;
    a.slots = slots;
    a.n = num_tokens;
    a.blocks = (num_tokens + mla::append::kWarps - 1) / mla::append::kWarps;
    a.num_slots = (int64_t)num_pool_pages * MLA_PAGE_SIZE;
    a.pool = kv_pool;
    a.scale = kv_scale;
    a.kr = static_cast<__nv_bfloat16*>(kr_pool);
    a.dev_error = dev_error;
    Rows r = {};
    int64_t blocks = a.blocks;
    if (q) {
        r.x = q;
        r.x_token = q_token_stride;
        r.x_head = q_head_stride;
        r.out = q_r;
        r.out_token = MLA_NUM_HEADS * MLA_ROPE_DIM;
        r.out_head = MLA_ROPE_DIM;
        r.rest = q_c;
        r.rest_token = MLA_NUM_HEADS * MLA_HEAD_DIM;
        r.rest_head = MLA_HEAD_DIM;
        r.positions = positions;
        r.heads = MLA_NUM_HEADS;
        r.dim = MLA_ROPE_DIM;
        r.offset = MLA_HEAD_DIM;
        r.rot_units = MLA_ROPE_DIM / (half ? 16 : 8);
        r.units = r.rot_units + MLA_HEAD_DIM / 8;
        a.four = four_heads(num_tokens, r.heads, r.units);
        blocks += lay_out(&r, num_tokens, a.four);
    }
    const auto go = [&](auto kernel) {
        return mla::launch_dependent("rope append kernel launch", kernel, dim3((unsigned)blocks), dim3(kThreads), 0,
                                     stream, a, r, *rope);
    };
    switch (kv_dtype) {
        case MLA_KV_BF16: return half ? go(rope_append_kernel<MLA_KV_BF16, true>) : go(rope_append_kernel<MLA_KV_BF16, false>);
        case MLA_KV_FP8_E4M3:
            return half ? go(rope_append_kernel<MLA_KV_FP8_E4M3, true>) : go(rope_append_kernel<MLA_KV_FP8_E4M3, false>);
        default: return half ? go(rope_append_kernel<MLA_KV_NVFP4, true>) : go(rope_append_kernel<MLA_KV_NVFP4, false>);
    }
}
