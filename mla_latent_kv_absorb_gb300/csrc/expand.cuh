// expand.cuh -- the decompression of gathered cache rows: for every head the keys and values
//
//   k[h,i,:] = W_UK[h] c_i,   v[h,i,:] = W_UV[h] c_i     (page 1 section 4, path A)
//
// for the rows c_i (512 values) of a prefix or of a chunk's span.  256 products (two weights, 128 heads) of
// [128 rows x 512] by [512 x 128] for every tile of 128 rows, 33.5 MFLOP a row: bound by the tensor cores.
//
// Persistent: the products lie in one line, row tile by row tile, which the CTAs cut evenly.  A CTA keeps the
// tile's rows in shared memory (128 KB) and streams the weights through a ring of 16 KB chunks ([128 outputs]
// [64 k]: four MMAs each) from L2, where all 32 MB of them lie.  Four accumulators in tensor memory, so that
// the outputs of a product leave (eight warps, two products at a time) while the next ones are computed.  What
// bounds it then is a chunk's way into the SM: 16 KB for 256 cycles of MMAs, where tiled copies come at some 42
// bytes a cycle.  (The GEMM of the step with one CTA a product reads the rows again for every product, 32 KB
// for the same MMAs, and starts each product cold: 334 us for 4,100 rows.)
#pragma once
#include "attend.cuh"

namespace mla {
namespace expand {

using attend::wait_all;

constexpr int kThreads = 32 * 11;
constexpr int kChunk = 16384;              // [128][64] bf16
constexpr int kChunks = 8;                 // of a product's 512 k
constexpr int kSlots = 6;
constexpr int kOffRing = kChunks * kChunk;
constexpr int kOffBar = kOffRing + kSlots * kChunk;
constexpr int kBarWFull = 0, kBarWEmpty = kSlots, kBarAFull = 2 * kSlots, kBarAEmpty = kBarAFull + kChunks,
              kBarDFull = kBarAEmpty + kChunks, kBarDFree = kBarDFull + 4, kBarEnd = kBarDFree + 4, kBars = kBarEnd + 1;
constexpr int kSmemBytes = kOffBar + 8 * kBars + 16;
constexpr int kProducts = 256;             // of a row tile: W_UK of 128 heads, then W_UV
static_assert(kSmemBytes <= 232448, "a CTA's shared memory");

struct Params {
    int rows;
    int64_t products;  // kProducts x row tiles
    __nv_bfloat16 *k, *v;  // [128][rows][128]
    uint32_t* dev_error;
    uint64_t timeout_ns;
};
// Phases: W full/empty by slot, A full/empty by chunk and row tile, D full/free by accumulator; each is waited
// for in order by one role, and the next phase needs that role's progress.

__global__ void __launch_bounds__(kThreads, 1)
expand_kernel(const __grid_constant__ CUtensorMap tm_rows, const __grid_constant__ CUtensorMap tm_uk,
              const __grid_constant__ CUtensorMap tm_uv, const __grid_constant__ Params p)
{
    using namespace dev;
    using namespace attend;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bars = sbase + kOffBar;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + kOffBar + 8 * kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    const auto bar = [&](int id) { return bars + 8 * id; };

    if (sbase & 1023u) {
        if (threadIdx.x == 0) raise_error(p.dev_error, MLA_DEVERR_SMEM_ALIGN);
        return;
    }
    if (threadIdx.x == 0) {
        for (int b = 0; b < kBarDFree; ++b) mbar_init(bar(b), 1);
        for (int b = 0; b < 4; ++b) mbar_init(bar(kBarDFree + b), 4);  // one arrive per warp of the accumulator's set
        mbar_init(bar(kBarEnd), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_holder), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
    const WaitCtx w{p.timeout_ns, abort_flag, p.dev_error};
    const int64_t first = first_unit(blockIdx.x, p.products, gridDim.x), end = first_unit(blockIdx.x + 1, p.products, gridDim.x);

    if (warp == 0) {
        // the weights do not depend on the kernel before: they are under way while it ends
        const bool leader = elect_lane();
        const uint64_t pol = l2_policy_evict_last();
        int r = 0, s = 0, phase = 0;
        bool ok = true;
        for (int64_t at = first; ok && at < end; ++at) {
            const int which = (int)(at % kProducts), row = (which & 127) * 128;
            const CUtensorMap* map = which < 128 ? &tm_uk : &tm_uv;
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
                if (!(ok = r < kSlots || wait_all(bar(kBarWEmpty + s), phase - 1, w))) break;
                if (leader) {
                    mbar_arrive_expect_tx(bar(kBarWFull + s), kChunk);
                    tma_load_2d(sbase + kOffRing + s * kChunk, map, bar(kBarWFull + s), 64 * c, row, pol);
                }
                ++r;
                if (++s == kSlots) {
                    s = 0;
                    ++phase;
                }
            }
        }
        for (int k = r > kSlots ? r - kSlots : 0; k < r; ++k)
            drain_phase(bar(kBarWFull + k % kSlots), k / kSlots, w.timeout_ns);
    } else if (warp == 2) {
        griddep_wait();  // the rows come from the kernel before
        const bool leader = elect_lane();
        const uint64_t pol = l2_policy_evict_last();
        int n = 0;  // row tiles
        int part = 0;  // chunks of the last one that were requested
        bool ok = true;
        for (int64_t at = first; ok && at < end; at = (at / kProducts + 1) * kProducts, ++n) {
            const int row = (int)(at / kProducts) * 128;
            part = 0;
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
                if (n > 0 && !(ok = wait_all(bar(kBarAEmpty + c), n - 1, w))) break;
                if (leader) {
                    mbar_arrive_expect_tx(bar(kBarAFull + c), kChunk);
                    tma_load_2d(sbase + c * kChunk, &tm_rows, bar(kBarAFull + c), 64 * c, row, pol);
                }
                part = c + 1;
            }
        }
        // every chunk's last load has landed before the CTA ends
        for (int c = 0; c < kChunks; ++c) {
            const int last = c < part ? n - 1 : n - 2;
            if (last >= 0) drain_phase(bar(kBarAFull + c), last, w.timeout_ns);
        }
    } else if (warp == 1) {
        constexpr uint32_t idesc = idesc_bf16(128, 128, false, false);
        const uint64_t a_desc = smem_desc(sbase, 16, 1024), w_desc = smem_desc(sbase + kOffRing, 16, 1024);
        constexpr uint64_t kChunk16 = kChunk >> 4;
        int s = 0, phase = 0, n = 0, j = 0;  // ring, row tiles, products
        bool ok = true;
        for (int64_t at = first; ok && at < end; ++at, ++j) {
            const bool fresh = at == first || at % kProducts == 0;
            const bool last = at + 1 == end || (at + 1) % kProducts == 0;
            const uint32_t d = tmem + 128 * (j & 3);
            if (j >= 4 && !(ok = wait_all(bar(kBarDFree + (j & 3)), (j >> 2) - 1, w))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
                if (fresh && !(ok = wait_all(bar(kBarAFull + c), n, w))) break;
                if (!(ok = wait_all(bar(kBarWFull + s), phase, w))) break;
                tc_fence_after();
                const uint64_t a = a_desc + c * kChunk16, b = w_desc + s * kChunk16;
                mma_ss_one(d, a, b, idesc, c != 0 ? 1u : 0u);
                mma_ss_one(d, a + 2, b + 2, idesc, 1u);
                mma_ss_one(d, a + 4, b + 4, idesc, 1u);
                mma_ss_one(d, a + 6, b + 6, idesc, 1u);
                mma_commit_one(bar(kBarWEmpty + s));
                if (last) mma_commit_one(bar(kBarAEmpty + c));
                if (++s == kSlots) {
                    s = 0;
                    ++phase;
                }
            }
            if (!ok) break;
            mma_commit_one(bar(kBarDFull + (j & 3)));
            n += last ? 1 : 0;
        }
        mma_commit_one(bar(kBarEnd));
    } else {
        // products j with j & 1 == set; a thread has one row
        const int set = (warp - 3) >> 2, q4 = warp & 3, row = 32 * q4 + lane;
        const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
        int j = set;
        for (int64_t at = first + set; at < end; at += 2, j += 2) {
            if (!wait_all(bar(kBarDFull + (j & 3)), j >> 2, w)) break;
            tc_fence_after();
            const int which = (int)(at % kProducts);
            const int64_t i = at / kProducts * 128 + row;
            __nv_bfloat16* dst = (which < 128 ? p.k : p.v) + ((int64_t)(which & 127) * p.rows + i) * 128;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t o[2][32];
                tmem_ld32(tmem + lane_base + 128 * (j & 3) + 64 * c, o[0]);
                tmem_ld32(tmem + lane_base + 128 * (j & 3) + 64 * c + 32, o[1]);
                tmem_wait_ld();
                if (c == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBarDFree + (j & 3)));
                }
                if (i < p.rows) {
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        const uint32_t* x = &o[v >> 2][8 * (v & 3)];
                        reinterpret_cast<uint4*>(dst + 64 * c)[v] =
                            make_uint4(pack_bf16x2(__uint_as_float(x[0]), __uint_as_float(x[1])),
                                       pack_bf16x2(__uint_as_float(x[2]), __uint_as_float(x[3])),
                                       pack_bf16x2(__uint_as_float(x[4]), __uint_as_float(x[5])),
                                       pack_bf16x2(__uint_as_float(x[6]), __uint_as_float(x[7])));
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        if (lane == 0) drain_phase(bar(kBarEnd), 0, w.timeout_ns);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace expand
}  // namespace mla
