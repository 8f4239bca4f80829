// expand.cuh -- the decompression of gathered cache rows: for every head the keys and values
//
//   k[h,i,:] = W_UK[h] c_i,   v[h,i,:] = W_UV[h] c_i     (page 1 section 4, path A)
//
// for the rows c_i (512 values) of a prefix or of a chunk's span.  128 products (one head's keys and values) of
// [256 rows x 512] by [512 x 256] for every tile of 256 rows, 33.5 MFLOP a row: bound by the tensor cores.
// Measured: 8,192 rows 152 us (under ncu; 1.81 PFLOP/s, tensor pipe 83 % busy), 4,100 rows 79.5, 2,051 rows 48.
// The rows are bf16, as mla_gather_kv gives them: of an FP8 or NVFP4 cache the product of code and token scale has been
// rounded once more (opened keys and values 0.0023 off 64 bits for 0.0017, relative L2).
//
// A pair of CTAs (two SMs) takes a product: M = 256, each CTA with 128 of the rows and of the sums, and half of
// N, the even one W_UK[h], the odd one W_UV[h].  Persistent: the products lie in one line, row tile by row tile,
// which the pairs cut evenly.  A CTA keeps its rows of the tile in shared memory (128 KB) and streams its
// weights through a ring of 16 KB chunks ([128 outputs][64 k]: four MMAs each) from L2, where all 32 MB of
// them lie.  Two accumulators in tensor memory, so that the outputs of a product leave while the next one is
// computed.  A pair, because the way into an SM bounds a CTA that takes its products alone: 16 KB for 256 cycles
// of MMAs, where tiled copies come at some 30 to 40 bytes a cycle; a pair's CTA needs them for 512.
#pragma once
#include "attend.cuh"

namespace mla {
namespace expand {

constexpr int kThreads = 32 * 11;
constexpr int kChunk = 16384;              // [128][64] bf16
constexpr int kChunks = 8;                 // of a product's 512 k
constexpr int kSlots = 6;                  // a chunk's way round takes some 2,700 cycles, its MMAs 512
constexpr int kRowsTile = 256;
constexpr int kOffRing = kChunks * kChunk;
constexpr int kOffBar = kOffRing + kSlots * kChunk;
constexpr int kBarWFull = 0, kBarWEmpty = kSlots, kBarAFull = 2 * kSlots, kBarAEmpty = kBarAFull + kChunks,
              kBarDFull = kBarAEmpty + kChunks, kBarEnd = kBarDFull + 2, kBarDFree = kBarEnd + 1, kBars = kBarDFree + 2;
constexpr int kSmemBytes = kOffBar + 8 * kBars + 16;
constexpr int kProducts = 128;             // of a row tile: one for each head
static_assert(kSmemBytes <= 232448, "a CTA's shared memory");

struct Params {
    int rows;
    int64_t products;  // kProducts x row tiles
    __nv_bfloat16 *k, *v;  // [128][rows][128]
    uint32_t* dev_error;
    uint64_t timeout_ns;
};
// Barriers: W and A full in the even CTA, by both CTAs' copies (a warp of the odd one that passed each arrival on
// took 1,800 cycles a chunk, the cost of a release to the cluster beside the output's stores); W and A empty and D
// full in both, by the pair's commits; D free in the even CTA, by both CTAs' sixteen output warps.
// Phases: W full/empty by slot, A full/empty by chunk and row tile, D full/free by accumulator; each is
// waited for in order by one role, and the next phase needs that role's progress.

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
expand_kernel(const __grid_constant__ CUtensorMap tm_rows, const __grid_constant__ CUtensorMap tm_uk,
              const __grid_constant__ CUtensorMap tm_uv, const __grid_constant__ Params p)
{
    using namespace dev;
    using namespace attend;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bars = sbase + kOffBar;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + kOffBar + 8 * kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    const auto bar = [&](int id) { return bars + 8 * id; };

    if (threadIdx.x == 0) {
        for (int b = 0; b < kBarDFree; ++b) mbar_init(bar(b), 1);
        for (int b = 0; b < 2; ++b) mbar_init(bar(kBarDFree + b), 16);  // one arrive per output warp of both CTAs
        const bool misaligned = (sbase & 1023u) != 0;
        if (misaligned) raise_error(p.dev_error, MLA_DEVERR_SMEM_ALIGN);
        *abort_flag = misaligned;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_holder), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers exist before anyone arrives remotely
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
    const WaitCtx w{p.timeout_ns, abort_flag, p.dev_error};
    const int64_t first = first_unit(blockIdx.x >> 1, p.products, gridDim.x >> 1),
                  end = first_unit((blockIdx.x >> 1) + 1, p.products, gridDim.x >> 1);

    if (*abort_flag) {
    } else if (warp == 0) {
        // The weights are under way while the gather ahead ends, which does not write them; whatever did has
        // ended, because the gather lets this kernel start only behind its own wait (see expand_rows).
        const bool leader = elect_lane();
        const uint64_t pol = l2_policy_evict_last();
        const CUtensorMap* map = rank == 0 ? &tm_uk : &tm_uv;
        const uint32_t full = map_to_cta(bar(kBarWFull), 0);
        int r = 0, s = 0, phase = 0;
        bool ok = true;
        for (int64_t at = first; ok && at < end; ++at) {
            const int row = (int)(at % kProducts) * 128;
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
                if (!(ok = r < kSlots || wait_all(bar(kBarWEmpty + s), phase - 1, w))) break;
                if (leader) {
                    if (rank == 0) mbar_arrive_expect_tx(bar(kBarWFull + s), 2 * kChunk);
                    tma_load_2d_pair(sbase + kOffRing + s * kChunk, map, full + 8 * s, 64 * c, row, pol);
                }
                ++r;
                if (++s == kSlots) {
                    s = 0;
                    ++phase;
                }
            }
        }
        if (rank == 0)  // the pair's loads have landed before either CTA ends
            for (int k = r > kSlots ? r - kSlots : 0; k < r; ++k)
                drain_phase(bar(kBarWFull + k % kSlots), k / kSlots, w.timeout_ns);
    } else if (warp == 2) {
        griddep_wait();  // the rows come from the kernel before
        griddep_launch_dependents();  // behind the wait: what starts now finds everything before this kernel written
        const bool leader = elect_lane();
        const uint64_t pol = l2_policy_evict_last();
        const uint32_t full = map_to_cta(bar(kBarAFull), 0);
        int n = 0;     // row tiles
        int part = 0;  // chunks of the last one that were requested
        bool ok = true;
        for (int64_t at = first; ok && at < end; at = (at / kProducts + 1) * kProducts, ++n) {
            const int row = (int)(at / kProducts) * kRowsTile + 128 * rank;  // may lie past the rows: read as zeros
            part = 0;
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
                if (n > 0 && !(ok = wait_all(bar(kBarAEmpty + c), n - 1, w))) break;
                if (leader) {
                    if (rank == 0) mbar_arrive_expect_tx(bar(kBarAFull + c), 2 * kChunk);
                    tma_load_2d_pair(sbase + c * kChunk, &tm_rows, full + 8 * c, 64 * c, row, pol);
                }
                part = c + 1;
            }
        }
        for (int c = 0; rank == 0 && c < kChunks; ++c) {
            const int last = c < part ? n - 1 : n - 2;
            if (last >= 0) drain_phase(bar(kBarAFull + c), last, w.timeout_ns);
        }
    } else if (warp == 1 && rank == 0) {
        constexpr uint32_t idesc = idesc_bf16(256, 256, false, false);
        const uint64_t a_desc = smem_desc(sbase, 16, 1024), w_desc = smem_desc(sbase + kOffRing, 16, 1024);
        constexpr uint64_t kChunk16 = kChunk >> 4;
        int s = 0, phase = 0, n = 0, j = 0;  // ring, row tiles, products
        bool ok = true;
        for (int64_t at = first; ok && at < end; ++at, ++j) {
            const bool fresh = at == first || at % kProducts == 0;
            const bool last = at + 1 == end || (at + 1) % kProducts == 0;
            const uint32_t d = tmem + 256 * (j & 1);
            if (j >= 2 && !(ok = wait_all(bar(kBarDFree + (j & 1)), (j >> 1) - 1, w))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
                if (fresh && !(ok = wait_all(bar(kBarAFull + c), n, w))) break;
                if (!(ok = wait_all(bar(kBarWFull + s), phase, w))) break;
                tc_fence_after();
                const uint64_t a = a_desc + c * kChunk16, b = w_desc + s * kChunk16;
                mma_ss_pair(d, a, b, idesc, c != 0 ? 1u : 0u);
                mma_ss_pair(d, a + 2, b + 2, idesc, 1u);
                mma_ss_pair(d, a + 4, b + 4, idesc, 1u);
                mma_ss_pair(d, a + 6, b + 6, idesc, 1u);
                mma_commit_pair(bar(kBarWEmpty + s));
                if (last) mma_commit_pair(bar(kBarAEmpty + c));
                if (++s == kSlots) {
                    s = 0;
                    ++phase;
                }
            }
            if (!ok) break;
            mma_commit_pair(bar(kBarDFull + (j & 1)));
            n += last ? 1 : 0;
        }
        mma_commit_pair(bar(kBarEnd));
    } else if (warp == 1) {
        // the odd CTA's MMAs are issued by the even one
    } else {
        // Four warps have the keys, four the values of 32 rows each, 16 rows at a time.  Two lanes exchange a pair
        // of columns, so that a quad writes 32 bytes of a row side by side: whole sectors.  (A row a lane, 16
        // bytes at a time, took four times a product's MMAs; through shared memory and TMA the smaller ring, or
        // the wait for the tile, cost more.)
        const int set = (warp - 3) >> 2, q4 = warp & 3, row = 128 * rank + 32 * q4 + (lane >> 2);
        const uint32_t from = tmem + ((uint32_t)(32 * q4) << 16) + 128 * set;
        const uint32_t r_free = map_to_cta(bar(kBarDFree), 0);
        const bool odd = lane & 1;
        const int col = odd ? 8 + 2 * (lane & 2) : 2 * (lane & 2);  // of the 16 columns of two steps
        __nv_bfloat16* const out = set == 0 ? p.k : p.v;
        int j = 0;
        for (int64_t at = first; at < end; ++at, ++j) {
            if (!wait_all(bar(kBarDFull + (j & 1)), j >> 1, w)) break;
            tc_fence_after();
            __nv_bfloat16* const head = out + (at % kProducts) * p.rows * 128;
            const int64_t i0 = at / kProducts * kRowsTile + row;
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {
                uint32_t o[64];
                tmem_ld_16x128(from + ((uint32_t)(16 * part) << 16) + 256 * (j & 1), o);
                tmem_wait_ld();
                if (part == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote_relaxed(r_free + 8 * (j & 1));
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int64_t i = i0 + 16 * part + 8 * x;
                    uint2* dst = reinterpret_cast<uint2*>(head + i * 128 + col);
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        const uint32_t a = pack_bf16x2(__uint_as_float(o[4 * k + 2 * x]), __uint_as_float(o[4 * k + 2 * x + 1]));
                        const uint32_t b = pack_bf16x2(__uint_as_float(o[4 * k + 4 + 2 * x]), __uint_as_float(o[4 * k + 5 + 2 * x]));
                        const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
                        if (i < p.rows) dst[2 * k] = odd ? make_uint2(other, b) : make_uint2(a, other);
                    }
                }
            }
        }
    }
    // After a wait that ran out the odd CTA's loads may be in flight without a barrier of its own: they land in
    // microseconds, and it waits a millisecond.
    if (threadIdx.x == 0 && *abort_flag)
        for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 1000000;) {
        }
    // the pair's last MMAs have finished before either CTA gives its memory back
    if (warp == 1 && lane == 0 && rank == 0 && !(sbase & 1023u)) drain_phase(bar(kBarEnd), 0, w.timeout_ns);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
    cluster_sync();  // no remote arrival at a CTA that has finished
}

}  // namespace expand
}  // namespace mla
