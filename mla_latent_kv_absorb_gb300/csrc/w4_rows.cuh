// w4_rows.cuh -- the 4-bit product for more rows, on tcgen05 (included by w4.cu).
//
// The weights are the M side here too: 128 outputs are the 128 lanes of tensor memory, up to 64 rows of
// x are the columns of the accumulator.  A thread unpacks the codes of one output, as w4.cu does,
// straight into its lane of tensor memory, where the MMA takes its A operand from, so that unpacked
// weights never pass through shared memory, and a group's scale is one number a thread: a group's MMAs
// start from zero, and its sums are added times the scale to the thread's own (a scale times a weight
// would round in bf16).  A thread block has two such halves, 256 outputs, over one ring of x:
//   1 thread      brings the packed codes, steps of 128 k (bulk copies)
//   1 thread      brings x (TMA, 128-byte swizzle)
//   4 warps       of each half unpack, into one of two buffers of 64 columns
//   1 thread      of each half issues the MMAs (16 k: 45 cycles for up to 64 rows; one thread for both
//                 halves waits for either in turn: 40.9 us where two take 31.3)
//   4 warps       of each half add up the groups in registers, and at the end of a tile write the
//                 outputs through shared memory, 16 bytes a thread
// A step of the two halves takes 0.7 us at groups of 128 (33 rows of 16384 -> 8192: 31.3 us, 2.2 TB/s;
// the weights' bytes alone 10.4 us, the MMAs 12): nothing in it is busy throughout, the chain of codes,
// unpacking, MMAs and sums through two buffers each is what it waits for (two microseconds less with
// the unpacking taken out, none with the sums).  What it took to get there, same case: one tile of 128
// outputs a thread block and x for each, 48 us; the rings counted without divisions, 37; two halves over
// one x, 36; codes two steps a copy and x one, 33.5 (an SM takes about 0.1 us for a copy of any size);
// the sums' registers kept from the other warps, which spilled, and one barrier less, 31.8.  Codes
// fetched a step ahead into registers: no gain.
#pragma once

namespace mla::w4::rows {

constexpr int kRows = 64, kTileN = 128, kHalves = 2;
constexpr int kBufs = 2, kACols = kBlockK / 2;  // of a half: as many of A as of D
constexpr int kScalers = 4 * kHalves, kUnpackers = 4 * kHalves;  // warps
constexpr int kCodesWarp = kScalers + kUnpackers, kXWarp = kCodesWarp + 1, kMmaWarp = kXWarp + 1;
constexpr int kThreads = 32 * (kMmaWarp + kHalves);
constexpr int kCodeSlots = 6, kXSlots = 8;   // the most; of two steps' codes half as many, of x as many as fit
constexpr int kXRing = 64 * 1024;
constexpr int kPitch = kTileN + 8;               // of the outputs on their way, bf16
constexpr int kSumPitch = kHalves * kTileN + 4;  // of a cluster's sums, fp32

template <int kGroup>
struct Cfg {
    static constexpr int kBlock = kCodeBytes + scale_bytes(kGroup) + zero_bytes(kGroup), kTile = 4 * kBlock;  // codes of a step
    static constexpr int kSlot = kHalves * kTile;
    static constexpr int kX = 0, kOut = kXRing, kCodes = kOut + kHalves * kRows * kPitch * 2,
                         kBars = kCodes + kCodeSlots * kSlot;
    static constexpr int kNumBars = 2 * (kCodeSlots + kXSlots + kHalves * 2 * kBufs) + 1;
    static constexpr int kBytes = kBars + 8 * kNumBars + 16;
    static_assert(kRows * kSumPitch * 4 <= kCodes, "a cluster's sums take the place of x");
    static_assert(kBytes <= 227 * 1024 && kBytes > 114 * 1024, "one thread block an SM, which takes all its tensor memory");
    static_assert(kHalves * kBufs * (kACols + kRows) <= 512, "tensor memory");
};

struct Args {
    const uint8_t* packed;
    int block_bytes;
    uint32_t zero_mask;
    __nv_bfloat16* out;
    int64_t out_row, out_head;
    float tensor_scale;
    int rows, cols;  // cols: the rows of a thread block, a multiple of 16
    int x_slots;
    int n, k_shift;            // k_shift: log2 of the packed layout's warps over k
    int panels, packed_steps;  // of one head, as packed
    int pairs, pairs_each;     // of tiles of 128 outputs, of one head
    int steps;                 // of 128 k; the codes come two at a time
    int splits;
    bool one_x;       // one x row for all heads
    bool out_octets;  // eight outputs are one aligned 16-byte store
    bool early;
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, uint32_t bar, int x, int y, int z, int w,
                                            uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void barrier_sync(uint32_t id, uint32_t threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

template <int kGroup>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ Args a)
{
    using C = Cfg<kGroup>;
    using namespace dev;
    constexpr bool kInt4 = kGroup >= 32;
    constexpr int kPerStep = kInt4 ? kBlockK / kGroup : 1;  // groups of a step
    constexpr int kGroupMmas = kBlockK / 16 / kPerStep;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)blockIdx.x % a.splits, pair0 = (int)blockIdx.x / a.splits * a.pairs_each;
    const int pairs = a.pairs - pair0 < a.pairs_each ? a.pairs - pair0 : a.pairs_each;
    const int h = blockIdx.y, r0 = (int)blockIdx.z * kRows;
    const int twos = (a.steps + 1) / 2;
    const int begin = 2 * (int)((int64_t)twos * rank / a.splits), to_two = 2 * (int)((int64_t)twos * (rank + 1) / a.splits);
    const int end = to_two < a.steps ? to_two : a.steps, ksteps = end - begin, all = pairs * ksteps;
    const uint32_t sbase = smem_u32(smem), bars = sbase + C::kBars;
    const uint32_t codes_full = bars, codes_empty = codes_full + 8 * kCodeSlots, x_full = codes_empty + 8 * kCodeSlots,
                   x_empty = x_full + 8 * kXSlots, a_full = x_empty + 8 * kXSlots, a_empty = a_full + 8 * kHalves * kBufs,
                   d_full = a_empty + 8 * kHalves * kBufs, d_empty = d_full + 8 * kHalves * kBufs,
                   mma_done = d_empty + 8 * kHalves * kBufs;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kBars + 8 * C::kNumBars);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_holder + 1);

    // Block nb (32 outputs) of the head's tile and k block kb, or NULL past the last panel.
    const auto block_at = [&](int tile, int nb, int kb) -> const uint8_t* {
        const int b = 4 * tile + nb, panel = b >> (2 - a.k_shift);
        if (panel >= a.panels) return nullptr;
        const int w = ((b << a.k_shift) & (kWarps - 1)) + (kb & ((1 << a.k_shift) - 1));
        return a.packed + ((((int64_t)h * a.panels + panel) * a.packed_steps + (kb >> a.k_shift)) * kWarps + w) * a.block_bytes;
    };
    const uint32_t tile_bytes = 4 * a.block_bytes;
    const bool ones = a.steps == 1;  // a slot has the codes of one step, not of two
    const int tile_off = ones ? C::kTile : 2 * C::kTile, slot_bytes = kHalves * tile_off, code_slots = ones ? kCodeSlots : kCodeSlots / 2;
    // of a tile in a slot: from one row of blocks to the next, and from one block over k to the next
    const int row_bytes = a.k_shift == 0 ? a.block_bytes : 2 * a.block_bytes, k_bytes = a.k_shift == 0 ? 4 * a.block_bytes : a.block_bytes;

    if (tid == 0) {
        const auto init = [](uint32_t bar, int count, int arrivals) {
            for (int i = 0; i < count; ++i) mbar_init(bar + 8 * i, arrivals);
        };
        init(codes_full, kCodeSlots, 1);
        init(codes_empty, kCodeSlots, kUnpackers + (kInt4 ? kScalers : 0));
        init(x_full, kXSlots, 1);
        init(x_empty, kXSlots, kHalves);
        init(a_full, kHalves * kBufs, 4);
        init(a_empty, kHalves * kBufs, 1);
        init(d_full, kHalves * kBufs, 1);
        init(d_empty, kHalves * kBufs, 4);
        init(mma_done, 1, kHalves);
        *abort = 0;
        fence_barrier_init();
    }
    if (warp == kCodesWarp && lane == 0) {
        tma_prefetch_desc(&tm_x);
        // to L2: no read of the weights, so it may come before the kernel ahead has ended
        if (a.k_shift == 0)
            for (int u = 0; u < kHalves && 2 * pair0 + u < a.panels; ++u)
                prefetch_l2(block_at(2 * pair0 + u, 0, begin), (ksteps < kCodeSlots ? ksteps : kCodeSlots) * tile_bytes);
    }
    griddep_wait();
    // Tensor memory is taken behind the kernel ahead and before the one behind may start, so that
    // nobody waits for tensor memory of a kernel that waits for him.
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_holder), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (a.early) griddep_launch_dependents();
    const uint32_t tmem_d = *tmem_holder, tmem_a = tmem_d + kHalves * kBufs * kRows;
    const WaitCtx wait{kTimeoutNs, abort, nullptr};
    float* sums = reinterpret_cast<float*>(smem);  // [row][kSumPitch], at the end
    // The swizzled tiles need a base of whole 1,024 bytes (uniform over the thread block).  Without it
    // nothing is brought and the outputs say so, as where a wait runs out.
    const bool aligned = (sbase & 1023u) == 0;
    bool ok = aligned;
    int issued = 0;  // copies, by the two threads that bring codes and x
    const int quarter = warp & 3, half = warp >> 2 & 1;

    // (rings are counted through: divisions by what is known at run time only take longer than a copy)
    if (warp == kCodesWarp) {
        if (lane == 0) {
            const int count = aligned ? pairs * ((ksteps + 1) / 2) : 0;
            int s = 0, slot = 0, turn = 0, pair = pair0, kb = begin;
            for (; s < count; ++s) {
                if (turn > 0 && !wait_phase(codes_empty + 8 * slot, turn - 1, wait)) break;
                const uint32_t to = sbase + C::kCodes + slot * slot_bytes, bar = codes_full + 8 * slot;
                const uint8_t* from = block_at(2 * pair, 0, kb);
                if (a.k_shift == 0) {  // four blocks of a step and four of the next lie side by side
                    const bool two = 2 * pair + 1 < a.panels;
                    const uint32_t bytes = end - kb > 1 ? 2 * tile_bytes : tile_bytes;
                    mbar_arrive_expect_tx(bar, two ? 2 * bytes : bytes);
                    bulk_load(to, from, bytes, bar);
                    if (two) bulk_load(to + tile_off, from + (int64_t)a.packed_steps * tile_bytes, bytes, bar);
                } else {  // two blocks over k of one row of blocks do, or all of two rows
                    const int rows_each = 4 >> a.k_shift, parts = min(2 * 4 >> (2 - a.k_shift), a.panels - (8 * pair >> (2 - a.k_shift)));
                    const uint32_t bytes = rows_each * 2 * a.block_bytes;
                    mbar_arrive_expect_tx(bar, parts * bytes);
                    for (int i = 0, per_tile = 4 / rows_each; i < parts; ++i)
                        bulk_load(to + (i >= per_tile ? tile_off + (i - per_tile) * bytes : i * bytes),
                                  block_at(2 * pair, i * rows_each, kb), bytes, bar);
                }
                if ((kb += 2) >= end) kb = begin, ++pair;
                if (++slot == code_slots) slot = 0, ++turn;
            }
            issued = s;
        }
    } else if (warp == kXWarp) {
        if (lane == 0) {
            const uint64_t keep = l2_policy_evict_last();  // x is read by every tile
            const int bytes = a.cols * 128;
            int s = 0, slot = 0, turn = 0, kb = begin;
            for (; aligned && s < all; ++s) {
                if (turn > 0 && !wait_phase(x_empty + 8 * slot, turn - 1, wait)) break;
                const uint32_t to = sbase + C::kX + slot * 2 * bytes, bar = x_full + 8 * slot;
                mbar_arrive_expect_tx(bar, 2 * bytes);
                tma_load_4d(to, &tm_x, bar, 0, a.one_x ? 0 : h, r0, 2 * kb, keep);
                if (++kb == end) kb = begin;
                if (++slot == a.x_slots) slot = 0, ++turn;
            }
            issued = s;
        }
    } else if (warp >= kMmaWarp) {
        if (lane == 0) {
            const int u = warp - kMmaWarp;
            const uint32_t idesc = idesc_bf16(128, a.cols, false, false), bytes = a.cols * 128;
            int slot = 0, turn = 0;
            for (int s = 0; s < all && ok; ++s) {
                const int ab = u * kBufs + s % kBufs;
                ok = wait_phase(x_full + 8 * slot, turn, wait) && wait_phase(a_full + 8 * ab, s / kBufs, wait);
                if (!ok) break;
                const uint64_t xd = smem_desc(sbase + C::kX + slot * 2 * bytes, 16, 1024);
                const uint64_t xd1 = smem_desc(sbase + C::kX + slot * 2 * bytes + bytes, 16, 1024);
#pragma unroll
                for (int i = 0; i < kPerStep; ++i) {
                    const int group = s * kPerStep + i, buf = u * kBufs + group % kBufs;
                    ok = ok && (group < kBufs || wait_phase(d_empty + 8 * buf, group / kBufs - 1, wait));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int m = 0; m < kGroupMmas; ++m) {
                        const int k = i * kGroupMmas + m;
                        mma_ts(tmem_d + buf * kRows, tmem_a + ab * kACols + 8 * k, (k < 4 ? xd : xd1) + (k % 4 * 32 >> 4), idesc,
                               m == 0 ? 0u : 1u);
                    }
                    mma_commit(d_full + 8 * buf);
                }
                if constexpr (kPerStep > 1) mma_commit(a_empty + 8 * ab);
                mma_commit(x_empty + 8 * slot);
                if (++slot == a.x_slots) slot = 0, ++turn;
            }
            mma_commit(mma_done);
        }
    } else if (warp >= kScalers) {
        const uint32_t to = tmem_a + ((uint32_t)(32 * quarter) << 16) + half * kBufs * kACols;
        // that the MMAs of a step are done; one group a step: its sums say so
        const uint32_t a_left = kPerStep > 1 ? a_empty : d_full;
        const uint8_t* block = smem + C::kCodes + half * tile_off + quarter * row_bytes;
        int slot = 0, turn = 0, kb = begin;
        for (int s = 0; s < all && ok; ) {
            ok = wait_warp(codes_full + 8 * slot, turn, wait);
            for (int two = 0; two < 2 && kb < end && ok; ++two, ++kb, ++s) {
                const int ab = s % kBufs;
                RowOfBlock<kGroup> w;
                w.load(block + slot * slot_bytes + two * k_bytes, lane);
                if (two == 1 || kb + 1 == end) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(codes_empty + 8 * slot);
                }
                ok = s < kBufs || wait_warp(a_left + 8 * (half * kBufs + ab), s / kBufs - 1, wait);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t v[16];
                    w.unpack(a.zero_mask, q, v);
                    tmem_st16(to + ab * kACols + 16 * q, v);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(a_full + 8 * (half * kBufs + ab));
            }
            if (kb >= end) kb = begin;
            if (++slot == code_slots) slot = 0, ++turn;
        }
    } else {
        const int chunks = a.cols / 16;
        const uint32_t from = tmem_d + ((uint32_t)(32 * quarter) << 16) + half * kBufs * kRows;
        const float unit = kInt4 ? 64.f : 256.f;
        const int rows = a.rows - r0 < kRows ? a.rows - r0 : kRows;
        __nv_bfloat16* stage = reinterpret_cast<__nv_bfloat16*>(smem + C::kOut) + half * kRows * kPitch;
        const uint8_t* block = smem + C::kCodes + half * tile_off + quarter * row_bytes;
        float acc[kRows];  // the rows of output 32 quarter + lane
#pragma unroll
        for (int i = 0; i < kRows; ++i) acc[i] = 0.f;
        int s = 0, slot = 0, turn = 0;
        for (int pair = pair0; pair < pair0 + pairs; ++pair) {
            for (int ks = 0; ks < ksteps && ok; ++ks, ++s) {
                float scale[kPerStep] = {};
                if constexpr (kInt4) {
                    const int two = ks & 1;
                    ok = two == 1 || wait_warp(codes_full + 8 * slot, turn, wait);
                    if (!ok) break;
                    RowOfBlock<kGroup>::scales(scale, block + slot * slot_bytes + two * k_bytes, lane);
                    if (two == 1 || ks + 1 == ksteps) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(codes_empty + 8 * slot);
                        if (++slot == code_slots) slot = 0, ++turn;
                    }
                }
#pragma unroll
                for (int i = 0; i < kPerStep; ++i) {
                    const int group = s * kPerStep + i, buf = group % kBufs;
                    ok = ok && wait_warp(d_full + 8 * (half * kBufs + buf), group / kBufs, wait);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < kRows / 16; ++c) {
                        if (c >= chunks) break;
                        uint32_t r[16];
                        tmem_ld16(from + buf * kRows + 16 * c, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            acc[16 * c + e] += kInt4 ? scale[i] * __uint_as_float(r[e]) : __uint_as_float(r[e]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(d_empty + 8 * (half * kBufs + buf));
                }
            }
            if (!ok) {  // given up: the outputs say so
#pragma unroll
                for (int i = 0; i < kRows; ++i) acc[i] = __uint_as_float(0x7FFFFFFFu);
            }
            if (a.splits > 1) {  // one pair: its sums are joined below
                barrier_sync(1, 32 * kScalers);  // the MMAs of both halves have left x, whose place they take
#pragma unroll
                for (int i = 0; i < kRows; ++i) sums[i * kSumPitch + half * kTileN + 32 * quarter + lane] = acc[i];
                break;
            }
            barrier_sync(1 + half, 128);  // the tile before has left
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                if (i / 16 < chunks) stage[i * kPitch + 32 * quarter + lane] = __float2bfloat16_rn(acc[i] * unit * a.tensor_scale);
                acc[i] = 0.f;
            }
            barrier_sync(1 + half, 128);
            const int n0 = (2 * pair + half) * kTileN;
            for (int e = tid & 127; e < rows * (kTileN / 8); e += 128) {
                const int r = e / (kTileN / 8), n = n0 + e % (kTileN / 8) * 8;
                const uint4 v = *reinterpret_cast<const uint4*>(stage + r * kPitch + n - n0);
                __nv_bfloat16* out = a.out + (int64_t)(r0 + r) * a.out_row + (int64_t)h * a.out_head + n;
                if (a.out_octets && n + 8 <= a.n) {
                    *reinterpret_cast<uint4*>(out) = v;
                } else {
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (n + i < a.n) out[i] = __ushort_as_bfloat16((unsigned short)(w[i / 2] >> (16 * (i & 1))));
                }
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    // Given up, which no thread finds out later than here: copies that nobody has waited for land before
    // their memory takes sums or goes to another thread block.
    if (*abort) {
        const bool codes = warp == kCodesWarp;
        const int slots = codes ? code_slots : a.x_slots;
        for (int i = issued < slots ? 0 : issued - slots; i < issued; ++i)
            drain_phase((codes ? codes_full : x_full) + 8 * (i % slots), i / slots, wait.timeout_ns);
        __syncthreads();
    }
    if (a.splits > 1) {
        // the sums of the cluster's blocks, added in the order of k, four outputs a thread
        if (*abort)  // x that came late may have overwritten them
            for (int i = tid; i < kRows * kSumPitch; i += kThreads) sums[i] = __uint_as_float(0x7FFFFFFFu);
        __syncwarp();
        cluster_sync();
        constexpr int kQuads = kHalves * kTileN / 4;
        const int rows = a.rows - r0 < kRows ? a.rows - r0 : kRows, n0 = pair0 * kHalves * kTileN;
        const float unit = kInt4 ? 64.f : 256.f;
        for (int e = rank * kThreads + tid; e < rows * kQuads; e += a.splits * kThreads) {
            const int r = e / kQuads, c = e % kQuads * 4, n = n0 + c;
            if (n >= a.n) continue;
            const uint32_t at = sbase + (r * kSumPitch + c) * 4;
            float4 v[8], sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int p = 0; p < 8; ++p)
                if (p < a.splits) v[p] = ld_cluster_f32x4(map_to_cta(at, p));
#pragma unroll
            for (int p = 0; p < 8; ++p)
                if (p < a.splits) sum.x += v[p].x, sum.y += v[p].y, sum.z += v[p].z, sum.w += v[p].w;
            const auto to_bf16 = [&](float f) { return __float2bfloat16_rn(f * unit * a.tensor_scale); };
            alignas(8) const __nv_bfloat16 o[4] = {to_bf16(sum.x), to_bf16(sum.y), to_bf16(sum.z), to_bf16(sum.w)};
            __nv_bfloat16* out = a.out + (int64_t)(r0 + r) * a.out_row + (int64_t)h * a.out_head + n;
            if (a.out_octets && n + 4 <= a.n) {
                *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(o);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < a.n) out[i] = o[i];
            }
        }
        __syncwarp();
        cluster_sync();  // no block leaves while another reads its sums
    }
    if (warp == kMmaWarp) {
        if (lane == 0) drain_phase(mma_done, 0, wait.timeout_ns);  // no MMA is under way when its memory goes
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_d, 512);
    }
}

// How a product is spread: one thread block per SM, several pairs of tiles each where there are more,
// clusters over k where there are fewer (of four at most: with eight, which find room on some GPCs
// only, 64 rows of 4096 -> 4096 took 23 us and not 15).
struct Spread {
    int pairs, steps, pairs_each, splits;
    int64_t blocks;
};
inline Spread spread_of(int rows, const mla_w4_weight& w)
{
    Spread p;
    p.pairs = (w.n + kHalves * kTileN - 1) / (kHalves * kTileN);
    p.steps = (w.k + kBlockK - 1) / kBlockK;
    p.pairs_each = p.splits = 1;
    const int64_t others = (int64_t)w.heads * ((rows + kRows - 1) / kRows), tasks = p.pairs * others;
    if (tasks > 152) {
        const int64_t each = (tasks + 151) / 152;
        p.pairs_each = (int)(each < p.pairs ? each : p.pairs);
    } else {
        for (const int s : {4, 2}) {
            if (p.steps < 4 * s || tasks * s > 144) continue;
            p.splits = s;
            break;
        }
    }
    p.blocks = (p.pairs + p.pairs_each - 1) / p.pairs_each * p.splits * others;
    return p;
}

// Whether this kernel is the faster one.  Either takes a fixed time and a time for its work: w4.cu's for
// every 32 outputs x 128 k x 8 rows of an SM (0.033 us, more where a thread block has few steps), this
// one for every step of 256 outputs x 128 k of a thread block, whatever number of rows up to 64 (0.8 us,
// with more groups of a step to add up 0.9 and 1.35 us, NVFP4 0.85 us).  In units of 0.033 us, fitted to
// measurements of 13 shapes with 17 to 128 rows; us of w4.cu's and of this kernel, groups of 128:
//   16384 -> 8192   25 rows 34.3 / 30.7   33: 40.5 / 31.3   64: 56.2 / 33.0   128: 106 / 56.2
//   4096 -> 4096    25 rows  8.2 / 12.1   33: 10.9 / 12.4   64: 13.6 / 13.3   128: 20.4 / 13.8
//   128 heads, 128 -> 512  17 rows 7.7 / 6.6   33: 10.5 / 7.2   64: 15.7 / 8.1   128: 30.9 / 15.4
// Not for 128 outputs or fewer, which leave a half idle (128 heads, 512 -> 128, 33 rows: 6.2 / 7.8 us,
// 64: 8.4 / 8.4, 128: 15.4 / 16.0),
// nor where x does not suit the tensor map: rows and heads apart from each other, k in whole 64.
template <int kGroup>
bool faster(const w4::Args& a, const mla_w4_weight& w, const Layout& l)
{
    const auto apart = [&](int64_t s) { return s >= w.k && s < ((int64_t)1 << 38); };
    if (a.rows <= 2 * kRowTile || w.n <= kTileN || w.k % 64 != 0 || (a.rows > 1 && !apart(a.x_row)) ||
        (w.heads > 1 && a.x_head != 0 && !apart(a.x_head)))
        return false;
    const double tiles = (double)l.panels * l.steps * kWarps * w.heads * ((a.rows + kRowTile - 1) / kRowTile) / 152;
    const Spread p = spread_of(a.rows, w);
    const double steps = (double)p.pairs_each * ((p.steps + p.splits - 1) / p.splits) * ((p.blocks + 151) / 152);
    constexpr double kStep = kGroup == 128 ? 24 : kGroup == 64 ? 28 : kGroup == 16 ? 26 : 41;
    return tiles * (1 + 1.5 / l.steps) > 45 + kStep * steps;
}

template <int kGroup>
mla_status launch(const w4::Args& from, const mla_w4_weight& w, const Layout& l, void* stream)
{
    using C = Cfg<kGroup>;
    Args a = {};
    a.cols = from.rows < kRows ? (from.rows + 15) / 16 * 16 : kRows;
    CUtensorMap tm_x;
    a.one_x = w.heads == 1 || from.x_head == 0;
    // 64 k, head, row, which 64 k: two pieces of 64 k of all rows are one copy
    const cuuint64_t dims[4] = {64, (cuuint64_t)(a.one_x ? 1 : w.heads), (cuuint64_t)from.rows, (cuuint64_t)w.k / 64};
    const cuuint64_t strides[3] = {(cuuint64_t)(a.one_x ? w.k : from.x_head) * 2, (cuuint64_t)(from.rows == 1 ? w.k : from.x_row) * 2, 128};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)a.cols, 2};
    if (!make_bf16_map(&tm_x, from.x, 4, dims, strides, box)) {
        set_last_error_text("4-bit product: no tensor map of x");
        return MLA_ERR_CUDA;
    }
    const int64_t row_blocks = ((int64_t)from.rows + kRows - 1) / kRows;
    a.packed = from.packed;
    a.block_bytes = from.block_bytes;
    a.zero_mask = from.zero_mask;
    a.out = from.out;
    a.out_row = from.out_row;
    a.out_head = from.out_head;
    a.tensor_scale = from.tensor_scale;
    a.rows = from.rows;
    a.n = from.n;
    a.k_shift = l.k_warps == 4 ? 2 : l.k_warps - 1;
    a.panels = (int)l.panels;
    a.packed_steps = (int)l.steps;
    const Spread p = spread_of(from.rows, w);
    a.pairs = p.pairs;
    a.pairs_each = p.pairs_each;
    a.steps = p.steps;
    a.splits = p.splits;
    a.x_slots = kXRing / (a.cols * 256) < kXSlots ? kXRing / (a.cols * 256) : kXSlots;
    a.out_octets = is_aligned(from.out, 16) && (from.rows == 1 || from.out_row % 8 == 0) && (w.heads == 1 || from.out_head % 8 == 0);
    a.early = from.early;
    const auto kernel = rows_kernel<kGroup>;
    const mla_status st = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes),
                                      "cudaFuncSetAttribute(max dynamic shared memory)");
    if (st != MLA_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.pairs + a.pairs_each - 1) / a.pairs_each * a.splits), (unsigned)w.heads, (unsigned)row_blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kBytes;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, tm_x, a), "4-bit product kernel launch");
}

}  // namespace mla::w4::rows
