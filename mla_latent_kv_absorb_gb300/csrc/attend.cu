// attend.cu -- shared prefixes (mla_prefix_open, mla_prefix_attend) and windowed prefill chunks
// (mla_prefill_window); declared in include/mla.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/mla.h"
#include "attend.cuh"
#include "expand.cuh"
#include "launch.cuh"
#include "nvtx_range.h"

namespace mla {
// gather.cu: `len` rows of one sequence into contiguous bf16 rows [len][576]; row t is token t below
// skip_from and token t + skip behind it
mla_status gather_one_sequence(mla_kv_dtype kv_dtype, const void* kv_pool, const float* kv_scale, const void* kr_pool,
                               int32_t num_pool_pages, const int32_t* block_table_row, int32_t max_pages, int32_t len,
                               void* out, uint32_t* dev_error, void* stream, int32_t skip_from = 0, int32_t skip = 0);
}  // namespace mla

namespace {

using mla::attend::Layout;
using mla::is_aligned;

constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int64_t kMaxKeys = (int64_t)65535 * 128;  // as mla_prefill_decompressed
constexpr int32_t kMaxRows = 65536;

size_t up_1k(size_t x) { return (x + 1023) & ~(size_t)1023; }

bool cache_ok(mla_kv_dtype kv_dtype, const void* kv_pool, const float* kv_scale, const void* kr_pool)
{
    if (kv_dtype != MLA_KV_BF16 && kv_dtype != MLA_KV_FP8_E4M3 && kv_dtype != MLA_KV_NVFP4) return false;
    return kv_pool && (kv_dtype == MLA_KV_BF16 || (kv_scale && kr_pool));
}

bool cache_aligned(mla_kv_dtype kv_dtype, const void* kv_pool, const float* kv_scale, const void* kr_pool)
{
    return is_aligned(kv_pool, 16) && (kv_dtype == MLA_KV_BF16 || (is_aligned(kr_pool, 16) && is_aligned(kv_scale, 4)));
}

// The maps of q_c [rows][128][128], q_r [rows][128][64], k and v [128][keys][128] and k_r [keys] rows of
// `kr_stride` elements: boxes of 64 columns by 128 rows, by 128 keys (64 in a pair), by 64 keys for the values.
struct Maps {
    CUtensorMap qc, qr, k, kr, v, out;  // out: a chunk's alone, boxes of 16 rows of one head by 64 columns
};

bool make_maps(Maps* m, const void* q_c, const void* q_r, const void* k, const void* v, const void* k_r,
               int64_t kr_stride, int64_t rows, int64_t keys, bool pair, const void* out)
{
    using mla::make_bf16_map;
    const cuuint64_t qc_dims[3] = {128, 128, (cuuint64_t)rows}, qc_str[2] = {128 * 2, 128 * 128 * 2};
    const cuuint64_t qr_dims[3] = {64, 128, (cuuint64_t)rows}, qr_str[2] = {64 * 2, 128 * 64 * 2};
    const cuuint32_t q_box[3] = {64, 1, 128}, o_box[3] = {64, 1, 16};
    const cuuint64_t k_dims[3] = {128, (cuuint64_t)keys, 128}, k_str[2] = {128 * 2, (cuuint64_t)keys * 128 * 2};
    const cuuint32_t k_box[3] = {64, pair ? 64u : 128u, 1}, v_box[3] = {64, 64, 1};
    const cuuint64_t r_dims[2] = {64, (cuuint64_t)keys}, r_str[1] = {(cuuint64_t)kr_stride * 2};
    const cuuint32_t r_box[2] = {64, pair ? 64u : 128u};
    return make_bf16_map(&m->qc, q_c, 3, qc_dims, qc_str, q_box) && make_bf16_map(&m->qr, q_r, 3, qr_dims, qr_str, q_box) &&
           make_bf16_map(&m->k, k, 3, k_dims, k_str, k_box) && make_bf16_map(&m->v, v, 3, k_dims, k_str, v_box) &&
           make_bf16_map(&m->kr, k_r, 2, r_dims, r_str, r_box) &&
           (!out || make_bf16_map(&m->out, out, 3, qc_dims, qc_str, o_box));
}

template <bool kChunk, bool kPair>
mla_status launch_attend(const Maps& m, const mla::attend::Params& p, int workers, void* stream)
{
    using namespace mla::attend;
    const auto kernel = attend_kernel<kChunk, kPair>;
    const mla_status st = mla::cuda_status(
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<kPair>::kSmemBytes),
        "cudaFuncSetAttribute(max dynamic shared memory)");
    if (st != MLA_OK) return st;
    const auto launch = [&](const OutMap<kChunk>& out) {
        return mla::launch_dependent("attend kernel launch", kernel, dim3((unsigned)(kPair ? 2 * workers : workers)),
                                     dim3(kThreads), Layout<kPair>::kSmemBytes, stream, m.qc, m.qr, m.k, m.kr, m.v, out, p);
    };
    if constexpr (kChunk)
        return launch(m.out);
    else
        return launch(NoMap{});
}

mla_status sm_count(int* sms)
{
    int dev = 0;
    const mla_status st = mla::cuda_status(cudaGetDevice(&dev), "cudaGetDevice");
    if (st != MLA_OK) return st;
    return mla::cuda_status(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev), "cudaDeviceGetAttribute");
}

// The keys and values of `num` gathered rows of 576 for all heads: k and v [128][num][128].  Called directly
// behind gather_one_sequence: the kernel reads the weights before it waits for the kernel ahead of it, and
// what was launched before that one has ended by then only because the gather waits before it lets the next
// kernel start.
mla_status expand_rows(const void* rows, const void* w_uk, const void* w_uv, void* k, void* v, int32_t num,
                       uint32_t* dev_error, int sms, void* stream)
{
    using namespace mla::expand;
    CUtensorMap tm_rows, tm_uk, tm_uv;
    const cuuint64_t r_dims[2] = {512, (cuuint64_t)num}, r_str[1] = {576 * 2};
    const cuuint64_t w_dims[2] = {512, 128 * 128}, w_str[1] = {512 * 2};
    const cuuint32_t box[2] = {64, 128};
    if (!mla::make_bf16_map(&tm_rows, rows, 2, r_dims, r_str, box) || !mla::make_bf16_map(&tm_uk, w_uk, 2, w_dims, w_str, box) ||
        !mla::make_bf16_map(&tm_uv, w_uv, 2, w_dims, w_str, box))
        return MLA_ERR_CUDA;
    const mla_status st = mla::cuda_status(
        cudaFuncSetAttribute(expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes),
        "cudaFuncSetAttribute(max dynamic shared memory)");
    if (st != MLA_OK) return st;
    Params p = {};
    p.rows = num;
    p.products = (int64_t)((num + kRowsTile - 1) / kRowsTile) * kProducts;
    p.k = static_cast<__nv_bfloat16*>(k);
    p.v = static_cast<__nv_bfloat16*>(v);
    p.dev_error = dev_error;
    p.timeout_ns = kTimeoutNs;
    const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(sms / 2, p.products));
    return mla::launch_dependent("expand kernel launch", expand_kernel, dim3((unsigned)(2 * pairs)),
                                 dim3(kThreads), kSmemBytes, stream, tm_rows, tm_uk, tm_uv, p);
}

// How the prefix form cuts its work: by CTAs of 128 rows, with more rows by pairs of them.
struct Cut {
    bool pair;
    int groups, group_rows, rows_cap, tiles, workers;
    int64_t slots;
    size_t lse_off, total;  // workspace: partials [slots][rows_cap][128] fp32, then [slots][rows_cap] fp32
};

Cut cut_prefix(int32_t rows, int32_t prefix_len, int32_t num_sms)
{
    Cut c;
    c.pair = rows > 128;
    c.group_rows = c.pair ? 256 : 128;
    c.groups = (rows + c.group_rows - 1) / c.group_rows;
    c.rows_cap = std::min(rows, c.group_rows);
    c.tiles = (prefix_len + 127) / 128;
    c.workers = (int)std::min<int64_t>(c.pair ? std::max(1, num_sms / 2) : num_sms, (int64_t)c.groups * 128 * c.tiles);
    c.slots = (int64_t)c.workers + (int64_t)c.groups * 128 - 1;
    c.lse_off = (size_t)c.slots * c.rows_cap * 128 * 4;
    c.total = c.lse_off + (size_t)c.slots * c.rows_cap * 4;
    return c;
}

bool prefix_sizes_ok(int32_t rows, int32_t prefix_len, int32_t num_sms)
{
    return rows >= 1 && prefix_len >= 1 && num_sms >= 1;
}

bool prefix_sizes_fit(int32_t rows, int32_t prefix_len, int32_t num_sms)
{
    return rows <= kMaxRows && prefix_len <= kMaxKeys && num_sms <= 4096;
}

// A chunk's keys: the sinks and everything from the first query's window on, without the tokens between.
struct Span {
    int32_t skip_from, skip, keys;
    size_t k, v, total;  // workspace: rows [keys][576], k and v [128][keys][128], bf16, 1 KB aligned
};

Span chunk_span(int32_t seq_len, int32_t chunk_len, int32_t window, int32_t sinks)
{
    Span s;
    const int64_t first = std::max<int64_t>(0, (int64_t)seq_len - chunk_len - window + 1);
    s.skip_from = sinks;
    s.skip = (int32_t)std::max<int64_t>(0, first - sinks);
    s.keys = seq_len - s.skip;
    s.k = up_1k((size_t)s.keys * 576 * 2);
    s.v = s.k + up_1k((size_t)s.keys * 128 * 128 * 2);
    s.total = s.v + up_1k((size_t)s.keys * 128 * 128 * 2);
    return s;
}

// Whether a chunk's rows go to CTAs of 128 or to pairs of 256.  Each worker takes whole (head, group) segments in
// rounds; a segment costs its key tiles and some 3,000 cycles.  A pair's tile takes 1,650 cycles and serves 256
// rows; a CTA alone brings in the whole tile for 128, 1,850, but has fewer keys that only other rows of the
// group see, and smaller pieces to share out.  Whole calls, pairs against CTAs alone: 257 queries under 511
// 59.0 and 49.3 us, 1,024 under 512 99.3 and 97.4, 2,000 under 300 153 and 145, 4,096 under 1,024 415 and 423; where
// the two estimates lie close it can miss: 4,096 under 128 take CTAs alone, 242 us, where pairs take 236.
constexpr int64_t kPairTile = 1650, kAloneTile = 1850, kSegment = 3000;

struct ChunkCut {
    bool pair;
    int groups, workers;
    int64_t cycles;
};

ChunkCut cut_chunk(bool pair, int32_t chunk_len, int32_t window, int32_t sinks, int32_t keys, int sms)
{
    ChunkCut c;
    const int rows = pair ? 256 : 128;
    c.pair = pair;
    c.groups = (chunk_len + rows - 1) / rows;
    c.workers = (int)std::min<int64_t>(pair ? std::max(1, sms / 2) : sms, (int64_t)c.groups * 128);
    const int64_t rounds = ((int64_t)c.groups * 128 + c.workers - 1) / c.workers;
    const int64_t seen = std::min<int64_t>(keys, (int64_t)window + rows - 1);
    const int64_t tiles = (seen + 127) / 128 + (std::min<int64_t>(sinks, keys - seen) + 127) / 128;
    c.cycles = rounds * (tiles * (pair ? kPairTile : kAloneTile) + kSegment);
    return c;
}

bool chunk_sizes_ok(int32_t seq_len, int32_t chunk_len, int32_t window, int32_t sinks)
{
    return seq_len >= 1 && chunk_len >= 1 && chunk_len <= seq_len && window >= 1 && sinks >= 0;
}

}  // namespace

extern "C" MLA_API mla_status mla_prefix_open(mla_kv_dtype kv_dtype, const void* kv_pool, const float* kv_scale,
                                              const void* kr_pool, int32_t num_pool_pages,
                                              const int32_t* block_table_row, int32_t max_pages, int32_t prefix_len,
                                              const void* w_uk, const void* w_uv, void* rows, void* k, void* v,
                                              uint32_t* dev_error, void* stream)
{
    const mla::NvtxRange nvtx_range("mla_prefix_open");
    if (!cache_ok(kv_dtype, kv_pool, kv_scale, kr_pool) || !block_table_row || !w_uk || !w_uv || !rows || !k || !v ||
        !dev_error || rows == k || rows == v || k == v)
        return MLA_ERR_INVALID_ARG;
    if (prefix_len < 1 || num_pool_pages < 1 || max_pages < 1 || ((int64_t)prefix_len + 63) / 64 > max_pages)
        return MLA_ERR_INVALID_ARG;
    if (!cache_aligned(kv_dtype, kv_pool, kv_scale, kr_pool) || !is_aligned(block_table_row, 4) || !is_aligned(w_uk, 16) ||
        !is_aligned(w_uv, 16) || !is_aligned(rows, 16) || !is_aligned(k, 16) || !is_aligned(v, 16) || !is_aligned(dev_error, 4))
        return MLA_ERR_ALIGNMENT;
    if (prefix_len > kMaxKeys) return MLA_ERR_UNSUPPORTED;
    int sms = 0;
    mla_status st = sm_count(&sms);
    if (st != MLA_OK) return st;
    st = mla::gather_one_sequence(kv_dtype, kv_pool, kv_scale, kr_pool, num_pool_pages, block_table_row,
                                             max_pages, prefix_len, rows, dev_error, stream);
    if (st != MLA_OK) return st;
    return expand_rows(rows, w_uk, w_uv, k, v, prefix_len, dev_error, sms, stream);
}

extern "C" MLA_API size_t mla_prefix_attend_workspace_bytes(int32_t num_rows, int32_t prefix_len, int32_t num_sms)
{
    if (!prefix_sizes_ok(num_rows, prefix_len, num_sms) || !prefix_sizes_fit(num_rows, prefix_len, num_sms)) return 0;
    return cut_prefix(num_rows, prefix_len, num_sms).total;
}

extern "C" MLA_API mla_status mla_prefix_attend(int32_t num_rows, int32_t prefix_len, int32_t num_sms, const void* q_c,
                                                const void* q_r, const void* k, const void* v, const void* k_r,
                                                int64_t k_r_stride, float softmax_scale, const void* own_out,
                                                const float* own_lse, void* workspace, size_t workspace_bytes,
                                                void* out, float* lse, uint32_t* dev_error, void* stream)
{
    const mla::NvtxRange nvtx_range("mla_prefix_attend");
    if (num_rows < 0 || prefix_len < 1 || num_sms < 1 || !(softmax_scale > 0.f) || !std::isfinite(softmax_scale) ||
        k_r_stride < 64 || k_r_stride > ((int64_t)1 << 32))
        return MLA_ERR_INVALID_ARG;
    if (num_rows == 0) return MLA_OK;
    if (!q_c || !q_r || !k || !v || !k_r || !workspace || !out || !dev_error || (own_out == nullptr) != (own_lse == nullptr))
        return MLA_ERR_INVALID_ARG;
    if (!is_aligned(q_c, 16) || !is_aligned(q_r, 16) || !is_aligned(k, 16) || !is_aligned(v, 16) || !is_aligned(k_r, 16) ||
        k_r_stride % 8 || !is_aligned(workspace, 16) || !is_aligned(own_out, 16) || !is_aligned(out, 16) ||
        !is_aligned(own_lse, 4) || !is_aligned(lse, 4) || !is_aligned(dev_error, 4))
        return MLA_ERR_ALIGNMENT;
    if (!prefix_sizes_fit(num_rows, prefix_len, num_sms)) return MLA_ERR_UNSUPPORTED;
    const Cut c = cut_prefix(num_rows, prefix_len, num_sms);
    if (workspace_bytes < c.total) return MLA_ERR_WORKSPACE;
    Maps m = {};
    if (!make_maps(&m, q_c, q_r, k, v, k_r, k_r_stride, num_rows, prefix_len, c.pair, nullptr)) return MLA_ERR_CUDA;
    mla::attend::Params p = {};
    p.rows = num_rows;
    p.keys = prefix_len;
    p.scale_log2 = softmax_scale * kLog2e;
    p.groups = c.groups;
    p.dev_error = dev_error;
    p.timeout_ns = kTimeoutNs;
    p.tiles = c.tiles;
    p.rows_cap = c.rows_cap;
    p.ws_o = static_cast<float*>(workspace);
    p.ws_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + c.lse_off);
    const mla_status st = c.pair ? launch_attend<false, true>(m, p, c.workers, stream)
                                 : launch_attend<false, false>(m, p, c.workers, stream);
    if (st != MLA_OK) return st;
    mla::attend::Merge a = {};
    a.ws_o = p.ws_o;
    a.ws_lse = p.ws_lse;
    a.rows = num_rows;
    a.rows_cap = c.rows_cap;
    a.groups = c.groups;
    a.group_rows = c.group_rows;
    a.tiles = c.tiles;
    a.workers = c.workers;
    a.own_out = static_cast<const __nv_bfloat16*>(own_out);
    a.own_lse = own_lse;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    using mla::attend::kMergeWarps;
    const int64_t halves = (int64_t)num_rows * 128;  // of warps
    return mla::launch_dependent("prefix merge kernel launch", mla::attend::prefix_merge_kernel,
                                 dim3((unsigned)((halves + 2 * kMergeWarps - 1) / (2 * kMergeWarps))), dim3(32 * kMergeWarps), 0, stream, a);
}

extern "C" MLA_API size_t mla_prefill_window_workspace_bytes(int32_t seq_len, int32_t chunk_len, int32_t window,
                                                             int32_t sinks)
{
    if (!chunk_sizes_ok(seq_len, chunk_len, window, sinks)) return 0;
    return chunk_span(seq_len, chunk_len, window, sinks).total;
}

extern "C" MLA_API mla_status mla_prefill_window(mla_kv_dtype kv_dtype, const void* kv_pool, const float* kv_scale,
                                                 const void* kr_pool, int32_t num_pool_pages,
                                                 const int32_t* block_table_row, int32_t max_pages, int32_t seq_len,
                                                 int32_t chunk_len, int32_t window, int32_t sinks, const void* q_c,
                                                 const void* q_r, const void* w_uk, const void* w_uv,
                                                 float softmax_scale, void* workspace, size_t workspace_bytes,
                                                 void* out, uint32_t* dev_error, void* stream)
{
    const mla::NvtxRange nvtx_range("mla_prefill_window");
    if (!cache_ok(kv_dtype, kv_pool, kv_scale, kr_pool) || !block_table_row || !q_c || !q_r || !w_uk || !w_uv ||
        !workspace || !out || !dev_error)
        return MLA_ERR_INVALID_ARG;
    if (!chunk_sizes_ok(seq_len, chunk_len, window, sinks) || num_pool_pages < 1 || max_pages < 1 ||
        ((int64_t)seq_len + 63) / 64 > max_pages || !(softmax_scale > 0.f) || !std::isfinite(softmax_scale))
        return MLA_ERR_INVALID_ARG;
    if (!cache_aligned(kv_dtype, kv_pool, kv_scale, kr_pool) || !is_aligned(block_table_row, 4) || !is_aligned(q_c, 16) ||
        !is_aligned(q_r, 16) || !is_aligned(w_uk, 16) || !is_aligned(w_uv, 16) || !is_aligned(workspace, 16) ||
        !is_aligned(out, 16) || !is_aligned(dev_error, 4))
        return MLA_ERR_ALIGNMENT;
    const Span s = chunk_span(seq_len, chunk_len, window, sinks);
    if (s.keys > kMaxKeys) return MLA_ERR_UNSUPPORTED;
    if (workspace_bytes < s.total) return MLA_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    void *k = ws + s.k, *v = ws + s.v;
    int sms = 0;
    mla_status st = sm_count(&sms);
    if (st != MLA_OK) return st;
    ChunkCut c = cut_chunk(true, chunk_len, window, sinks, s.keys, sms);
    const ChunkCut alone = cut_chunk(false, chunk_len, window, sinks, s.keys, sms);
    if (alone.cycles < c.cycles) c = alone;
    Maps m;
    if (!make_maps(&m, q_c, q_r, k, v, ws + 512 * 2, 576, chunk_len, s.keys, c.pair, out)) return MLA_ERR_CUDA;
    st = mla::gather_one_sequence(kv_dtype, kv_pool, kv_scale, kr_pool, num_pool_pages, block_table_row, max_pages, s.keys, ws,
                                  dev_error, stream, s.skip_from, s.skip);
    if (st == MLA_OK) st = expand_rows(ws, w_uk, w_uv, k, v, s.keys, dev_error, sms, stream);
    if (st != MLA_OK) return st;
    mla::attend::Params p = {};
    p.rows = chunk_len;
    p.keys = s.keys;
    p.scale_log2 = softmax_scale * kLog2e;
    p.groups = c.groups;
    p.dev_error = dev_error;
    p.timeout_ns = kTimeoutNs;
    p.hi0 = seq_len - chunk_len - s.skip;
    p.window = std::min(window, seq_len);
    p.sinks = std::min(sinks, seq_len);
    return c.pair ? launch_attend<true, true>(m, p, c.workers, stream) : launch_attend<true, false>(m, p, c.workers, stream);
}
