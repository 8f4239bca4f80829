// attend.cuh -- attention of many query rows over decompressed keys and values, in two forms:
//
//   prefix  the rows of a whole decode batch attend to the one prefix that their sequences share
//           (every row sees every key); the result is a set of normalised partial outputs with
//           their log-sum-exps, which prefix_merge_kernel joins with each row's attention over its
//           sequence's own tokens;
//   chunk   the new tokens of one sequence under a sliding window: the query at position p sees the
//           keys j <= p with j > p - window or j < sinks.
//
// Keys and values are per head (page 1 section 4, path A): k, v [128 heads][keys][128] and k_R
// [keys][64], so a (row, key) pair costs 2 * (192 + 128) * 128 FLOP where the absorbed form costs
// 2 * (576 + 512) * 128, and 64 KB of keys and values are read for each prefix token however many
// rows there are: with up to some 220 rows that is what bounds the prefix form (HBM), beyond it
// the tensor cores.  Measured with the merge: 64 rows x 8,192 keys 85 us, 95 % of the copy rate; 256 rows x 16,384
// 254 us in a long run, 1.35 PFLOP/s (a plain library product 1.70 there), 220 alone (1.56; 1.91); a chunk of 4,096
// queries under a window of 1,024 303 us.
//
// A CTA holds a 128-row query tile of a head and streams 128-key tiles; with more than 128 rows a pair of CTAs
// (two SMs, MMAs of M = 256) holds 256 rows, and each brings in half of every key tile (64 keys) and of every
// value tile (64 dims).  Alone a CTA with 256 rows waited for its keys: 80 KB a tile and a ring of 128 KB.
// Step g is a key tile; the MMA order is PV(g), QK(g + 3), from one segment into the next (a segment's own
// beginning and end took 3,500 of 24,000 cycles a segment of a chunk).  Three score buffers and one output fill the
// tensor memory, so that two steps' scores lie ready when the softmax has finished with one.  (Two streams of every
// other tile, each with a score buffer, an output and a running softmax of its own: chunk 4,096 under 1,024 456 us
// for 444, prefix 64 x 8,192 85.3 for 84.8, 256 x 16,384 249 for 252.)
//   QK:  S[rows x 128] = Q [rows x 192] (q_c | q_R: three 64-column chunks in shared memory)
//                       x K tile [128 x 192] (k | k_R: three K-major chunks)
//   PV:  O[rows x 128] += P [rows x 128] (bf16 in TMEM over the first half of S) x V tile (MN-major)
// Everything that is streamed goes through one ring of slots, in the order in which the MMAs need it: a key chunk
// [128 keys][64] or 64 keys' values [64][128], in a pair half of it.  A slot is four MMAs, so the ring is as fine
// as the tensor core's work and a slot is free as soon as its four are done.
//
// Warp 0 streams the ring, warp 2 the query tiles, warp 1 issues the MMAs, warps 3-10 are the softmax
// of every step: a warp has 16 rows, a quad of lanes two of them (tcgen05.ld's 16x256b shape: lane l holds
// columns 8 k + 2 (l & 3), + 1 of rows l / 4 and l / 4 + 8), so that a row's maximum is two shuffles away.
// All eight warps work on one step: with four warps to every other step and a row a thread a step's softmax
// took 1,530 cycles, with halves of a row that agree through shared memory 1,450; this way 1,050.  What bounds it with
// many rows is no one thing: of some 1,700 cycles a step of 256 rows the MMAs execute 1,280; without any copies it
// takes 1,500, without the exponentials or with a third of the score products hardly less.
// The running maximum is that of the segment's first tile and moves only
// when a score exceeds it by more than 32 (log2 units), which loses nothing: fp32 and bf16 round relative to the
// value.  So a step takes its exponentials with the maximum that it has, looks at its scores beside that (no
// exchange between lanes), and does them again in the rare other case.  P is rounded to bf16 for the PV product
// (its sum l takes the unrounded values); scores, maxima, sums and O are fp32.
//
// The prefix form is persistent: the (head, row group, key tile) units lie in one line that the CTAs
// cut evenly, so that every SM streams the same number of bytes; a CTA's piece of one (head, group)
// run is a segment, written as one partial.  Every wait is bounded.
#pragma once
#include <type_traits>

#include "ptx.cuh"

namespace mla {
namespace attend {

using dev::WaitCtx;

// ---- The MMA warp runs as a whole, on values that are the same in all its lanes, and one elected lane
// issues: descriptors then live in uniform registers and an MMA is an instruction or two.  A single lane that
// computes them takes some ten instructions for each MMA, and waits for every one of them behind the two
// softmax warps of its SM sub-partition (measured beside eight warps that issue FMAs all the time: 134 cycles
// for an MMA of 64, against 71 this way).

__device__ __forceinline__ void mma_commit_one(uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// The same for a pair of CTAs (M = 256), issued in the even one.
__device__ __forceinline__ void mma_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
        : "memory");
}

// Arrives on the barrier at this offset in both CTAs when all earlier MMAs of the pair have finished.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// A ring slot's four MMAs and the commit that frees it, in one election: K steps of 16 columns of A (32 bytes in
// shared memory, 8 columns in tensor memory), of K-major keys (32 bytes) or of 16 MN-major rows of values (2,048 bytes).
template <bool kPair>
__device__ __forceinline__ void slot_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc, uint32_t bar)
{
#define MLA_SLOT_SS(GROUP, COMMIT)                                                          \
    asm volatile(                                                                           \
        "{\n\t.reg .pred p, t, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"                 \
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"              \
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"              \
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, %4, %4;\n\t"                             \
        "elect.sync _|e, 0xffffffff;\n\t"                                                  \
        "@e tcgen05.mma." GROUP ".kind::f16 [%0], %1, %2, %3, p;\n\t"                      \
        "@e tcgen05.mma." GROUP ".kind::f16 [%0], a1, b1, %3, t;\n\t"                      \
        "@e tcgen05.mma." GROUP ".kind::f16 [%0], a2, b2, %3, t;\n\t"                      \
        "@e tcgen05.mma." GROUP ".kind::f16 [%0], a3, b3, %3, t;\n\t"                      \
        "@e tcgen05.commit." GROUP ".mbarrier::arrive::one.shared::cluster" COMMIT ";\n\t}" \
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc), "r"(bar), "h"((uint16_t)3) : "memory")
    if (kPair)
        MLA_SLOT_SS("cta_group::2", ".multicast::cluster.b64 [%5], %6");
    else
        MLA_SLOT_SS("cta_group::1", ".b64 [%5]");
#undef MLA_SLOT_SS
}

// As slot_ss, with the first `pairs` (0, 1 or 2) pairs of the MMAs.
template <bool kPair>
__device__ __forceinline__ void slot_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t acc, int pairs,
                                        uint32_t bar)
{
#define MLA_SLOT_TS(GROUP, COMMIT)                                                          \
    asm volatile(                                                                           \
        "{\n\t.reg .pred p, t, e, e1, e2;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t" \
        "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\t"            \
        "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\t"        \
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, %4, %4;\n\t"                             \
        "elect.sync _|e, 0xffffffff;\n\t"                                                  \
        "setp.gt.and.s32 e1, %5, 0, e;\n\tsetp.gt.and.s32 e2, %5, 1, e;\n\t"              \
        "@e1 tcgen05.mma." GROUP ".kind::f16 [%0], [%1], %2, %3, p;\n\t"                   \
        "@e1 tcgen05.mma." GROUP ".kind::f16 [%0], [a1], b1, %3, t;\n\t"                   \
        "@e2 tcgen05.mma." GROUP ".kind::f16 [%0], [a2], b2, %3, t;\n\t"                   \
        "@e2 tcgen05.mma." GROUP ".kind::f16 [%0], [a3], b3, %3, t;\n\t"                   \
        "@e tcgen05.commit." GROUP ".mbarrier::arrive::one.shared::cluster" COMMIT ";\n\t}" \
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(acc), "r"(pairs), "r"(bar), "h"((uint16_t)3) : "memory")
    if (kPair)
        MLA_SLOT_TS("cta_group::2", ".multicast::cluster.b64 [%6], %7");
    else
        MLA_SLOT_TS("cta_group::1", ".b64 [%6]");
#undef MLA_SLOT_TS
}

// A bounded wait (as dev::wait_phase) that looks at the timer, which is slow to read, once in many polls.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t timeout_ns,
                                       uint32_t* dev_error)
{
    const uint64_t t0 = dev::globaltimer_ns();
    while (true) {
#pragma unroll 1
        for (int k = 0; k < 64; ++k)
            if (dev::mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if (dev::globaltimer_ns() - t0 > timeout_ns) {
            *abort = 1;
            dev::raise_error(dev_error, MLA_DEVERR_TIMEOUT);
            return false;
        }
    }
}

// The whole warp waits; the answer is a vote, the same in all lanes.  What the other CTA of a pair arrives for is
// in tensor memory (tcgen05 fences order it) or came by its copies, so the wait acquires for the CTA alone.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t phase, const WaitCtx& w)
{
    if (__all_sync(0xffffffffu, dev::mbar_try_wait(bar, phase & 1u))) return true;
    return __all_sync(0xffffffffu, wait_slow(bar, phase & 1u, w.abort, w.timeout_ns, w.dev_error));
}

__device__ __forceinline__ bool elect_lane()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(one));
    return one != 0;
}

// ---- Two floats at a time (one instruction each on sm_103a), and the largest of three.

__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 16 lanes (rows) x 8 K columns of 32 bits: r[4 k], r[4 k + 1] are columns 8 k + 2 (lane & 3) and the next
// of row lane / 4, r[4 k + 2], r[4 k + 3] those of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x128(uint32_t taddr, uint32_t (&r)[64])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}

// 16 rows x 32 columns in the 16x128b shape: r[2 k] is column 4 k + (lane & 3) of row lane / 4, r[2 k + 1] of
// row lane / 4 + 8: where the bf16 pairs of tmem_ld_16x128's columns go.
__device__ __forceinline__ void tmem_st_pairs(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}

constexpr int kTile = 128;                 // query rows of a tile, keys of a tile
constexpr int kThreads = 32 * 11;
constexpr int kSoftmaxWarp0 = 3;
constexpr uint32_t kTmemCols = 512;        // score buffer b at 128 b, O at 384
constexpr float kRescaleLog2 = 32.f;       // P up to 2^32, l and O below 2^32 x keys x |v|: far from fp32's 2^127

template <bool kPair>
struct Layout {
    static constexpr int kScores = 3;                        // score buffers, 128 columns each of tensor memory
    static constexpr int kOCol = kScores * 128;              // the output's 128 columns
    static constexpr int kSlot = kPair ? 8192 : 16384;
    static constexpr int kSlots = 131072 / kSlot;
    static constexpr int kQ = 3 * 16384;                     // a query tile; the next segment's is loaded beside it
    static constexpr int kOffRing = 2 * kQ;
    static constexpr int kOffBar = kOffRing + kSlots * kSlot;
    static constexpr int kBarFull = 0, kBarEmpty = kSlots;   // [slot]
    static constexpr int kBarQFull = 2 * kSlots, kBarQEmpty = kBarQFull + 2;  // [buffer]
    static constexpr int kBarSFull = kBarQEmpty + 2;         // [score buffer]
    static constexpr int kBarPReady = kBarSFull + kScores;   // [score buffer], every softmax warp's arrival
    static constexpr int kBarPV = kBarPReady + kScores;      // [score buffer], the PV of its P has finished
    static constexpr int kBarOFree = kBarPV + kScores;       // every softmax warp's arrival: the segment's O has been read
    static constexpr int kBarStage = kBarOFree + 1;          // [buffer], eight warps: the outputs staged there have left (chunk)
    static constexpr int kBarEnd = kBarStage + 2;            // every MMA has finished
    static constexpr int kBars = kBarEnd + 1;
    static constexpr int kSmemBytes = kOffBar + 8 * kBars + 16;
    static_assert(kSmemBytes <= 232448, "a CTA's shared memory");
};
// In a pair the barriers on which the MMAs wait (full, Q full, P ready, O free) are the even CTA's, by both CTAs'
// copies and warps; those that MMAs complete (empty, Q empty, S full, PV, end) are in both.
// Phase bookkeeping.  A barrier waited by parity must never run two phases ahead of its waiter:
//   S full [b]   completes once per step of buffer b; QK(g + 3) is issued only after the MMA warp
//                has seen P(g) ready, i.e. after the softmax has finished step g.
//   P ready [b]  arrives once per step; P(g + 3) needs S(g + 3), issued after that wait.
//   PV [b]       waited for at a segment's end and before O is scaled, for the step before the next: the PV three
//                steps ahead of it has finished (its S came after), PV(g + 3) needs P(g + 3).
//   Q full       a query load into a buffer is issued after its Q empty (the last QK of the segment before).
//   O free       once per segment; the next one's needs that segment's outputs, read after its last PV.
//   stage        a chunk's outputs leave through the query tile's buffer of their segment; the next query load into
//                it waits for that too.  They have left by the first step of the segment behind it; the scores ahead
//                of that step are of that segment, so nothing the step needs waits for that load.
//   ring         a slot is refilled only after its empty barrier, waited in order.

struct Params {
    int rows;            // query rows
    int keys;            // key rows
    float scale_log2;    // softmax_scale * log2(e)
    int groups;          // row groups of 128, in a pair 256
    uint32_t* dev_error;
    uint64_t timeout_ns;
    // prefix
    int tiles;           // key tiles of a run
    int rows_cap;        // rows of a partial
    float* ws_o;         // [slots][rows_cap][128]
    float* ws_lse;       // [slots][rows_cap]
    // chunk: query i sees the (compacted) keys c <= hi0 + i with c > hi0 + i - window or c < sinks
    int hi0, window, sinks;
};

// A worker's piece of one run.
struct Segment {
    int head, row0, cnt;  // cnt key tiles
    int lead, base;       // key tile n begins at key 128 n below lead, at base + 128 (n - lead) behind it
    int lead_end, end;    // no row of the group sees a key at or past these in the tiles below and from lead on
    int slot;             // the prefix's partial
};

// The first unit of worker (CTA or pair) c, of `units` in all shared by g <= units workers (each has one at least).
__host__ __device__ __forceinline__ int64_t first_unit(int64_t c, int64_t units, int64_t g) { return c * units / g; }

// Walks this worker's segments; every role walks the same ones.
template <bool kChunk, bool kPair>
struct Walk {
    static constexpr int kRows = kPair ? 2 * kTile : kTile;
    int64_t at, end;
    __device__ __forceinline__ int worker() const { return kPair ? blockIdx.x >> 1 : blockIdx.x; }
    __device__ __forceinline__ int workers() const { return kPair ? gridDim.x >> 1 : gridDim.x; }
    __device__ __forceinline__ explicit Walk(const Params& p)
    {
        if (kChunk) {
            at = worker();
            end = (int64_t)p.groups * 128;
        } else {
            const int64_t units = (int64_t)p.groups * 128 * p.tiles;
            at = first_unit(worker(), units, workers());
            end = first_unit(worker() + 1, units, workers());
        }
    }
    __device__ __forceinline__ bool next(const Params& p, Segment& s)
    {
        if (at >= end) return false;
        if (kChunk) {
            // a head's groups lie side by side: their windows overlap and are read from L2
            s.head = (int)at / p.groups;  // at most 128 x 65,535: a chunk has at most 65,535 groups of 128 (kMaxKeys)
            s.row0 = ((int)at - s.head * p.groups) * kRows;
            const int last = min(s.row0 + kRows, p.rows) - 1;
            const int lo = max(0, p.hi0 + s.row0 - p.window + 1);  // the first key in the first row's window
            s.lead = (min(p.sinks, lo) + kTile - 1) / kTile;
            s.base = max(s.lead * kTile, lo);
            s.cnt = s.lead + (p.hi0 + last - s.base + kTile) / kTile;  // the last key is hi0 + last
            s.end = p.hi0 + last + 1;
            s.lead_end = min(s.end, s.base > s.lead * kTile ? p.sinks : s.lead * kTile);
            s.slot = 0;
            at += workers();
        } else {
            const int run = (int)(at / p.tiles), n0 = (int)(at - (int64_t)run * p.tiles);
            s.head = run / p.groups;
            s.row0 = (run % p.groups) * kRows;
            s.cnt = (int)min((int64_t)(p.tiles - n0), end - at);
            s.lead = 0;
            s.base = n0 * kTile;
            s.lead_end = s.end = p.keys;
            s.slot = worker() + run;
            at += s.cnt;
        }
        return true;
    }
};

__device__ __forceinline__ int first_key(const Segment& s, int n)
{
    return n < s.lead ? n * kTile : s.base + (n - s.lead) * kTile;
}

// The keys of tile n that the products take: those that some row sees, up to a multiple of 32 (half of them are
// a pair's CTA's).  The others' scores stay what they were, and the softmax masks them.
__device__ __forceinline__ int tile_keys(const Segment& s, int n)
{
    return min(kTile, (((n < s.lead ? s.lead_end : s.end) - first_key(s, n)) + 31) & ~31);
}

// The map of the outputs, which a chunk alone writes by TMA.
struct NoMap {};
template <bool kChunk>
using OutMap = std::conditional_t<kChunk, CUtensorMap, NoMap>;

template <bool kChunk, bool kPair>
// 11 warps: three SM sub-partitions hold three of them, 16K registers each: at most 3 x 32 x 168
__global__ void __cluster_dims__(kPair ? 2 : 1, 1, 1) __maxnreg__(168)
attend_kernel(const __grid_constant__ CUtensorMap tm_qc, const __grid_constant__ CUtensorMap tm_qr,
              const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_kr,
              const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ OutMap<kChunk> tm_out,
              const __grid_constant__ Params p)
{
    using namespace dev;
    using L = Layout<kPair>;
    extern __shared__ __align__(1024) uint8_t smem[];
    // (through a shuffle, so that the compiler sees a value that is the warp's)
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = kPair ? (int)cluster_ctarank() : 0;
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bars = sbase + L::kOffBar;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::kOffBar + 8 * L::kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    const auto bar = [&](int id) { return bars + 8 * id; };
    // the barrier on which the MMA warp waits: the even CTA's
    const auto mma_bar = [&](int id) { return kPair ? map_to_cta(bars + 8 * id, 0) : bars + 8 * id; };

    if (threadIdx.x == 0) {
        constexpr int kWarps = kPair ? 16 : 8;  // softmax warps
        for (int s = 0; s < 2 * L::kSlots; ++s) mbar_init(bar(s), 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(L::kBarQFull + b), 1);
            mbar_init(bar(L::kBarQEmpty + b), 1);
            if (kChunk) mbar_init(bar(L::kBarStage + b), 8);
        }
        for (int b = 0; b < L::kScores; ++b) {
            mbar_init(bar(L::kBarSFull + b), 1);
            mbar_init(bar(L::kBarPReady + b), kWarps);
            mbar_init(bar(L::kBarPV + b), 1);
        }
        mbar_init(bar(L::kBarOFree), kWarps);
        mbar_init(bar(L::kBarEnd), 1);
        const bool misaligned = (sbase & 1023u) != 0;
        if (misaligned) raise_error(p.dev_error, MLA_DEVERR_SMEM_ALIGN);
        *abort_flag = misaligned;
        fence_barrier_init();
    }
    if (warp == 1) {
        if (kPair) {
            tmem_alloc_pair(smem_u32(tmem_holder), kTmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(tmem_holder), kTmemCols);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if (kPair)
        cluster_sync();  // both CTAs' barriers exist before anyone arrives remotely
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
    const WaitCtx w{p.timeout_ns, abort_flag, p.dev_error};
    Walk<kChunk, kPair> walk(p);
    Segment seg;

    if (*abort_flag) {
    } else if (warp == 0) {
        griddep_wait();  // keys, values and queries may come from the kernel before; nothing is written ahead of them
        const bool leader = elect_lane();
        // the prefix's keys and values are read once by one group of rows, k_R by every head
        const uint64_t pol_kv = kChunk || p.groups > 1 ? l2_policy_evict_last() : l2_policy_evict_first();
        const uint64_t pol_kr = l2_policy_evict_last();
        // Two walks: the keys are three steps ahead of the values, as the MMA warp takes them.  (The ring is all that is under way: bringing tiles
        // into L2 ahead of it costs more than it gives once the pieces follow one another without a gap: for 64 rows
        // and 8,192 tokens 90 us with the values two steps ahead, 95 with whole tiles and 124 with fourteen of them,
        // where 87 was without.  Of 10 to 16 slots a pair takes the same time.)
        Walk<kChunk, kPair> walk_k(p);
        Segment seg_k;
        bool more_k = walk_k.next(p, seg_k);
        int n_k = 0, g_k = 0, seg_no_k = 0;  // step of the segment, step, segment
        int r = 0, s = 0, phase = 0;
        bool ok = true;
        const uint32_t full0 = mma_bar(L::kBarFull);
        const auto take = [&]() {  // the next slot, free; its barrier expects the slot's bytes
            ok = r < L::kSlots || wait_all(bar(L::kBarEmpty + s), phase - 1, w);
            if (ok && leader && rank == 0) mbar_arrive_expect_tx(bar(L::kBarFull + s), (kPair ? 2 : 1) * L::kSlot);
            return ok;
        };
        const auto put = [&]() {
            ++r;
            if (++s == L::kSlots) {
                s = 0;
                ++phase;
            }
        };
        const auto load_k = [&]() {  // the next key tile
            // (in a pair the odd CTA's keys follow the even one's)
            const int j0 = first_key(seg_k, n_k) + (kPair ? rank * (tile_keys(seg_k, n_k) >> 1) : 0);
#pragma unroll 1
            for (int c = 0; c < 3; ++c) {
                if (!take()) return;
                const uint32_t dst = sbase + L::kOffRing + s * L::kSlot, full = full0 + 8 * s;
                if (leader) {
                    if (kPair) {
                        if (c < 2)
                            tma_load_3d_pair(dst, &tm_k, full, 64 * c, j0, seg_k.head, pol_kv);
                        else
                            tma_load_2d_pair(dst, &tm_kr, full, 0, j0, pol_kr);
                    } else {
                        if (c < 2)
                            tma_load_3d(dst, &tm_k, full, 64 * c, j0, seg_k.head, pol_kv);
                        else
                            tma_load_2d(dst, &tm_kr, full, 0, j0, pol_kr);
                    }
                }
                put();
            }
            ++g_k;
            if (++n_k == seg_k.cnt) {
                n_k = 0;
                ++seg_no_k;
                more_k = walk_k.next(p, seg_k);
            }
        };
        const auto keys_below = [&](int steps, int last_seg) {
            while (ok && more_k && g_k < steps && (n_k > 0 || seg_no_k <= last_seg)) load_k();
        };
        const auto load_v = [&](int j0) {
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
                if (!take()) return;
                const uint32_t dst = sbase + L::kOffRing + s * L::kSlot, full = full0 + 8 * s;
                if (leader) {
                    if (kPair) {
                        tma_load_3d_pair(dst, &tm_v, full, 64 * rank, j0 + 64 * c, seg.head, pol_kv);
                    } else {
                        tma_load_3d(dst, &tm_v, full, 0, j0 + 64 * c, seg.head, pol_kv);
                        tma_load_3d(dst + L::kSlot / 2, &tm_v, full, 64, j0 + 64 * c, seg.head, pol_kv);
                    }
                }
                put();
            }
        };
        if (leader) {
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_kr);
            tma_prefetch_desc(&tm_v);
        }
        keys_below(L::kScores, 1);
        for (int g = 0, n_seg = 0; ok && walk.next(p, seg); ++n_seg) {
            for (int n = 0; ok && n < seg.cnt; ++n, ++g) {
                load_v(first_key(seg, n));
                keys_below(g + 1 + L::kScores, n_seg + (n + 1 == seg.cnt ? 2 : 1));
            }
        }
        griddep_launch_dependents();  // the merge may be scheduled; it waits for this kernel's end
        // loads in flight land before the CTA can exit (in a pair both CTAs' complete on the even one's barriers)
        for (int k = r > L::kSlots ? r - L::kSlots : 0; rank == 0 && k < r; ++k)
            drain_phase(bar(L::kBarFull + k % L::kSlots), k / L::kSlots, w.timeout_ns);
    } else if (warp == 2) {
        griddep_wait();
        const bool leader = elect_lane();
        const uint64_t pol = l2_policy_evict_last();
        if (leader) {
            tma_prefetch_desc(&tm_qc);
            tma_prefetch_desc(&tm_qr);
        }
        int n = 0;
        while (walk.next(p, seg)) {
            const int b = n & 1;
            if (n >= 2 && !wait_all(bar(L::kBarQEmpty + b), (n >> 1) - 1, w)) break;
            if (kChunk && n >= 2 && !wait_all(bar(L::kBarStage + b), (n >> 1) - 1, w)) break;
            if (leader) {
                const uint32_t full = mma_bar(L::kBarQFull + b), q = sbase + b * L::kQ;
                const int row = seg.row0 + kTile * rank;
                if (rank == 0) mbar_arrive_expect_tx(bar(L::kBarQFull + b), (kPair ? 2 : 1) * L::kQ);
                if (kPair) {
                    tma_load_3d_pair(q, &tm_qc, full, 0, seg.head, row, pol);
                    tma_load_3d_pair(q + 16384, &tm_qc, full, 64, seg.head, row, pol);
                    tma_load_3d_pair(q + 2 * 16384, &tm_qr, full, 0, seg.head, row, pol);
                } else {
                    tma_load_3d(q, &tm_qc, full, 0, seg.head, row, pol);
                    tma_load_3d(q + 16384, &tm_qc, full, 64, seg.head, row, pol);
                    tma_load_3d(q + 2 * 16384, &tm_qr, full, 0, seg.head, row, pol);
                }
            }
            ++n;
        }
        for (int k = n > 2 ? n - 2 : 0; rank == 0 && k < n; ++k) drain_phase(bar(L::kBarQFull + (k & 1)), k >> 1, w.timeout_ns);
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr uint32_t idesc_qk0 = idesc_bf16(kPair ? 256 : 128, 0, false, false);
            uint32_t idesc_qk = 0;
            constexpr uint32_t idesc_pv = idesc_bf16(kPair ? 256 : 128, 128, false, true);
            const uint64_t q_desc = smem_desc(sbase, 16, 1024);
            const uint64_t k_desc = smem_desc(sbase + L::kOffRing, 16, 1024);
            const uint64_t v_desc = smem_desc(sbase + L::kOffRing, 8192, 1024);
            constexpr uint64_t kSlot16 = L::kSlot >> 4, kQChunk16 = 16384 >> 4;  // in the descriptors' 16-byte units
            const auto commit = [](uint32_t b) {
                if (kPair)
                    mma_commit_pair(b);
                else
                    mma_commit_one(b);
            };
            int s = 0, phase = 0, q_buf = 0;  // the next slot, the segment's query tile
            bool ok = true;
            const auto next_slot = [&]() {
                if (++s == L::kSlots) {
                    s = 0;
                    ++phase;
                }
            };
            // Scores into buffer b from the next three slots.
            const auto qk = [&](int b, int keys) {
                const uint32_t d = tmem + 128 * b;
                idesc_qk = idesc_qk0 | (uint32_t)(keys >> 3) << 17;
                const uint64_t a0 = q_desc + q_buf * 3 * kQChunk16;
#pragma unroll 1
                for (int c = 0; c < 3; ++c) {
                    if (!wait_all(bar(L::kBarFull + s), phase, w)) return ok = false;
                    tc_fence_after();
                    const uint64_t a = a0 + c * kQChunk16, k = k_desc + s * kSlot16;
                    slot_ss<kPair>(d, a, k, idesc_qk, c != 0 ? 1u : 0u, bar(L::kBarEmpty + s));
                    next_slot();
                }
                commit(bar(L::kBarSFull + b));
                return true;
            };
            // O from the P in buffer `buf` and the next two slots.
            const auto pv = [&](int buf, bool first, int keys) {
                const uint32_t pt = tmem + 128 * buf, d = tmem + L::kOCol;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    if (!wait_all(bar(L::kBarFull + s), phase, w)) return ok = false;
                    tc_fence_after();
                    const uint64_t b = v_desc + s * kSlot16;
                    const uint32_t a = pt + 32 * c;
                    slot_ts<kPair>(d, a, b, idesc_pv, first && c == 0 ? 0u : 1u, min(2, max(0, keys - 64 * c + 31) >> 5),
                                   bar(L::kBarEmpty + s));
                    next_slot();
                }
                return true;
            };
            // Two walks: the scores are up to three steps ahead of the outputs.  The first of a segment waits for its
            // query tile, whose buffer a chunk's outputs of the segment before the last left by: they need that
            // segment's products to have been issued.
            Walk<kChunk, kPair> walk_q(p);
            Segment seg_q;
            bool more_q = walk_q.next(p, seg_q);
            int n_q = 0, i_q = 0, g_q = 0, b_q = 0;  // its segment, step of the segment, step, score buffer
            const auto scores_below = [&](int steps, int last_seg) {
                while (more_q && g_q < steps && (i_q > 0 || n_q <= last_seg)) {
                    if (i_q == 0) {
                        q_buf = n_q & 1;
                        if (!(ok = wait_all(bar(L::kBarQFull + q_buf), n_q >> 1, w))) return false;
                    }
                    if (!qk(b_q, tile_keys(seg_q, i_q))) return false;
                    ++g_q;
                    b_q = b_q + 1 == L::kScores ? 0 : b_q + 1;
                    if (++i_q == seg_q.cnt) {
                        commit(bar(L::kBarQEmpty + q_buf));
                        i_q = 0;
                        ++n_q;
                        more_q = walk_q.next(p, seg_q);
                    }
                }
                return true;
            };
            scores_below(L::kScores, 1);
            int n_seg = 0, g = 0, b = 0, b_phase = 0;  // segments, steps, score buffer and its round
            while (ok && walk.next(p, seg)) {
                const int steps = seg.cnt;
                for (int i = 0; i < steps; ++i, ++g) {
                    if (!(ok = wait_all(bar(L::kBarPReady + b), b_phase, w))) break;
                    if (i == 0 && n_seg > 0 && !(ok = wait_all(bar(L::kBarOFree), n_seg - 1, w))) break;
                    tc_fence_after();
                    if (!pv(b, i == 0, tile_keys(seg, i))) break;
                    commit(bar(L::kBarPV + b));  // ahead of the next scores
                    if (++b == L::kScores) {
                        b = 0;
                        ++b_phase;
                    }
                    if (!scores_below(g + 1 + L::kScores, n_seg + (i + 1 == steps ? 2 : 1))) break;
                }
                ++n_seg;
            }
            commit(bar(L::kBarEnd));  // arrives when every MMA issued here has finished
        }
    } else {
        // softmax: warp (3..10) & 3 selects the TMEM lane quarter, a warp has 16 of its rows, a thread the
        // columns 8 k + 2 (lane & 3), + 1 of rows `row` and row + 8 (index 0 and 1 below)
        const int q4 = warp & 3, warp_row = 32 * q4 + 16 * ((warp - kSoftmaxWarp0) >> 2);
        const int row = warp_row + (lane >> 2), col = 2 * (lane & 3);
        const uint32_t lane_base = (uint32_t)warp_row << 16;
        const uint32_t r_ready = mma_bar(L::kBarPReady), r_free = mma_bar(L::kBarOFree);
        const auto arrive = [&](uint32_t at) {  // what it orders is in tensor memory
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (kPair)
                    mbar_arrive_remote_relaxed(at);
                else
                    mbar_arrive(at);
            }
        };
        int n_seg = 0, b = 0, b_phase = 0;  // segments, score buffer and its round
        int staged = -1;       // chunk: the buffer whose outputs are leaving
        const auto release = [&]() {
            if (lane == 0) {
                bulk_wait_read();
                mbar_arrive(bar(L::kBarStage + staged));
            }
            staged = -1;
        };
        bool ok = true;
        // The PV before the next step has finished (the scores of its step have been seen, so that the one three
        // steps ahead of it has, and the next needs the next step's P).
        const auto wait_pv = [&]() {
            return wait_all(bar(L::kBarPV + (b == 0 ? L::kScores - 1 : b - 1)), b == 0 ? b_phase - 1 : b_phase, w);
        };
        while (ok && walk.next(p, seg)) {
            const int steps = seg.cnt, tile_row = seg.row0 + kTile * rank;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // the running softmax
#pragma unroll 1
            for (int i = 0; i < steps; ++i) {
                const uint32_t t_s = tmem + lane_base + 128 * b;
                if (!(ok = wait_all(bar(L::kBarSFull + b), b_phase, w))) break;
                tc_fence_after();
                if (tile_row + warp_row < p.rows) {  // the warp has a row at all
                    uint32_t sr[64];
                    tmem_ld_16x128(t_s, sr);
                    tmem_wait_ld();
                    // Keys that a row does not see get -infinity.  A thread's 32 columns of a row in order are
                    // 0, 1, 8, 9, 16, ... from `col`; `upto` has a bit for each of them that is at most `c`.
                    const int j0 = first_key(seg, i);
                    const auto upto = [](int c) {
                        const int n = min(32, max(0, 2 * (c >> 3) + ((c & 7) ? 2 : 1)));
                        return c < 0 ? 0u : n == 32 ? 0xffffffffu : (1u << n) - 1u;
                    };
                    if (kChunk) {
                        // the first and the last row of the warp see every key: no row of it needs a mask
                        const int hi_first = p.hi0 + min(tile_row + warp_row, p.rows - 1);
                        const int hi_last = p.hi0 + min(tile_row + warp_row + 15, p.rows - 1);
                        if (j0 + kTile - 1 > hi_first || (j0 <= hi_last - p.window && j0 + kTile > p.sinks)) {
                            uint32_t sees[2];
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int hi = p.hi0 + min(tile_row + row + 8 * x, p.rows - 1), lo = hi - p.window + 1;
                                const int j = j0 + col;
                                sees[x] = upto(hi - j) & (~upto(lo - 1 - j) | upto(p.sinks - 1 - j));
                            }
#pragma unroll
                            for (int k = 0; k < 64; ++k)
                                if (!(sees[(k >> 1) & 1] >> (2 * (k >> 2) + (k & 1)) & 1u)) sr[k] = 0xff800000u;
                        }
                    } else if (j0 + kTile > p.keys) {
                        const uint32_t sees = upto(p.keys - 1 - j0 - col);
#pragma unroll
                        for (int k = 0; k < 64; ++k)
                            if (!(sees >> (2 * (k >> 2) + (k & 1)) & 1u)) sr[k] = 0xff800000u;
                    }
                    const uint64_t scale2 = pair(p.scale_log2, p.scale_log2);
                    uint32_t pk[2][16];
                    uint64_t sum[2];
                    const auto exponentials = [&]() {  // P and its sums with the maxima that there are
                        uint64_t neg2[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float neg = m[x] == -INFINITY ? 0.f : -m[x];
                            neg2[x] = pair(neg, neg);
                            sum[x] = 0;  // a pair of zeros
                        }
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const int x = k & 1;
                            float a, b;
                            unpair(fma2(pair(__uint_as_float(sr[2 * k]), __uint_as_float(sr[2 * k + 1])), scale2, neg2[x]), a, b);
                            a = ex2_approx(a);
                            b = ex2_approx(b);
                            sum[x] = add2(sum[x], pair(a, b));
                            pk[k >> 4][k & 15] = pack_bf16x2(a, b);
                        }
                    };
                    float mt[2];
                    bool beyond = i == 0;
                    if (i > 0) exponentials();
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float m2[2];  // two chains
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            m2[c] = fmaxf(__uint_as_float(sr[4 * c + 2 * x]), __uint_as_float(sr[4 * c + 2 * x + 1]));
#pragma unroll
                            for (int k = 2 + c; k < 16; k += 2)
                                m2[c] = max3(m2[c], __uint_as_float(sr[4 * k + 2 * x]), __uint_as_float(sr[4 * k + 2 * x + 1]));
                        }
                        mt[x] = fmaxf(m2[0], m2[1]) * p.scale_log2;
                        beyond = beyond || mt[x] > m[x] + kRescaleLog2;  // -infinity while a row has seen no key
                    }
                    if (__any_sync(0xffffffffu, beyond)) {
                        float f[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            mt[x] = fmaxf(mt[x], __shfl_xor_sync(0xffffffffu, mt[x], 1));
                            mt[x] = fmaxf(mt[x], __shfl_xor_sync(0xffffffffu, mt[x], 2));
                            const bool first = m[x] == -INFINITY, grow = mt[x] > m[x] + kRescaleLog2 || first;
                            f[x] = grow && !first ? ex2_approx(m[x] - mt[x]) : 1.f;
                            if (grow) m[x] = mt[x];
                            l[x] *= f[x];
                        }
                        if (i > 0 && __any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
                            if (!(ok = wait_pv())) break;
                            tc_fence_after();
                            const uint32_t t_o = tmem + lane_base + L::kOCol;
#pragma unroll 1
                            for (int c = 0; c < 4; ++c) {
                                uint32_t o[16];
                                tmem_ld_16x32(t_o + 32 * c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f[(k >> 1) & 1]);
                                tmem_st_16x32(t_o + 32 * c, o);
                            }
                        }
                        exponentials();
                    }
                    tmem_st_pairs(t_s, pk[0]);
                    tmem_st_pairs(t_s + 32, pk[1]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float a, b;
                        unpair(sum[x], a, b);
                        l[x] += a + b;
                    }
                    tmem_wait_st();
                }
                arrive(r_ready + 8 * b);
                if (++b == L::kScores) {
                    b = 0;
                    ++b_phase;
                }
                if (kChunk && staged >= 0) release();
            }
            if (!(ok = ok && wait_pv())) break;  // the segment's last
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // a quad has a row's sum
                l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
                l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
            }
            if (tile_row + warp_row < p.rows) {
                const int i = tile_row + row;
                float f[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    f[x] = 1.f / l[x];
                    if (!kChunk && i + 8 * x < p.rows && (lane & 3) == 0)
                        p.ws_lse[(int64_t)seg.slot * p.rows_cap + (i + 8 * x - seg.row0)] =
                            (m[x] + log2f(l[x])) * 0.69314718055994531f;
                }
                uint32_t o[64];
                tmem_ld_16x128(tmem + lane_base + L::kOCol, o);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 64; ++k)  // a row whose scores were all -infinity has no sum: zeros
                    o[k] = l[(k >> 1) & 1] == 0.f ? 0u : __float_as_uint(__uint_as_float(o[k]) * f[(k >> 1) & 1]);
                arrive(r_free);  // the next segment's products may start
                if (kChunk) {
                    // through shared memory and out by TMA, clipped at the last row: rows lie 32 KB apart, and 8 bytes a
                    // lane from registers took 2,100 cycles
                    uint8_t* stage = smem + (n_seg & 1) * L::kQ;
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int k = 0; k < 16; ++k) {  // columns 8 k + col, + 1: chunk k & 7 of 128-byte rows, swizzled
                            const int r = row + 8 * x;
                            *reinterpret_cast<uint32_t*>(stage + (k >> 3) * 16384 + r * 128 + (((k & 7) ^ (r & 7)) << 4) + 2 * col) =
                                pack_bf16x2(__uint_as_float(o[4 * k + 2 * x]), __uint_as_float(o[4 * k + 2 * x + 1]));
                        }
                    fence_proxy_async_cta();
                    __syncwarp();
                    if (lane == 0) {
                        const uint32_t from = smem_u32(stage) + warp_row * 128;
                        tma_store_3d(&tm_out, from, 0, seg.head, tile_row + warp_row);
                        tma_store_3d(&tm_out, from + 16384, 64, seg.head, tile_row + warp_row);
                        bulk_commit();
                    }
                } else {
                    // a quad's lanes write 32 bytes of a row side by side: whole sectors
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (i + 8 * x >= p.rows) continue;
                        float2* dst = reinterpret_cast<float2*>(
                            p.ws_o + ((int64_t)seg.slot * p.rows_cap + (i + 8 * x - seg.row0)) * 128 + col);
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            dst[4 * k] = make_float2(__uint_as_float(o[4 * k + 2 * x]), __uint_as_float(o[4 * k + 2 * x + 1]));
                    }
                }
            } else {
                arrive(r_free);
            }
            if (kChunk) staged = n_seg & 1;
            ++n_seg;
        }
        if (kChunk && lane == 0) bulk_wait_all();
    }
    // After a wait that ran out an odd CTA's loads may be in flight without a barrier of its own: they land in
    // microseconds, and it waits a millisecond.
    if (kPair && threadIdx.x == 0 && *abort_flag)
        for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 1000000;) {
        }
    // the last MMAs have finished before the tensor memory goes back
    if (warp == 1 && lane == 0 && rank == 0 && !(sbase & 1023u)) drain_phase(bar(L::kBarEnd), 0, w.timeout_ns);
    tc_fence_before();
    __syncthreads();
    if (kPair) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        if (kPair)
            tmem_dealloc_pair(tmem, kTmemCols);
        else
            tmem_dealloc(tmem, kTmemCols);
    }
    if (kPair) cluster_sync();  // no remote arrival at a CTA that has finished
}

struct Merge {
    const float* ws_o;
    const float* ws_lse;
    int rows, rows_cap, groups, group_rows, tiles, workers;  // as the attend kernel cut the units
    const __nv_bfloat16* own_out;  // [rows][128][128] or NULL
    const float* own_lse;          // [rows][128]
    __nv_bfloat16* out;            // may be own_out
    float* lse;                    // may be own_lse, or NULL
};

constexpr int kMergeWarps = 8;

// Joins the partials of the prefix (at most a few for one head and group) with the row's attention over
// its own tokens by log-sum-exp.  Half a warp per (row, head), eight columns a lane: bound by HBM and L2 (own
// outputs in, outputs out, partials from L2).  256 rows over 16,384 keys: 12 us for 54 MB (a warp of four columns a
// lane 17).
__global__ void __launch_bounds__(32 * kMergeWarps) prefix_merge_kernel(const __grid_constant__ Merge a)
{
    const int lane = threadIdx.x & 15;
    const int64_t id = (int64_t)blockIdx.x * (2 * kMergeWarps) + (threadIdx.x >> 4);
    if (id >= (int64_t)a.rows * 128) return;
    const int row = (int)(id >> 7), head = (int)(id & 127);
    const int group = row / a.group_rows, run = head * a.groups + group;
    const int64_t units = (int64_t)a.groups * 128 * a.tiles, u0 = (int64_t)run * a.tiles, u1 = u0 + a.tiles;
    // the workers with a unit of the run: c0 has the first, which lies at or after the quotient's
    int c0 = (int)(u0 * a.workers / units);
    while (c0 + 1 < a.workers && first_unit(c0 + 1, units, a.workers) <= u0) ++c0;
    int c1 = c0;
    while (c1 + 1 < a.workers && first_unit(c1 + 1, units, a.workers) < u1) ++c1;
    const int64_t at = row - group * a.group_rows;
    dev::griddep_wait();
    dev::griddep_launch_dependents();
    // The row's own part and the first three of the prefix (more only with more workers than runs) are requested
    // together, in one round trip.
    constexpr int kAtOnce = 3;
    const float own = a.own_lse ? a.own_lse[id] : -INFINITY;
    const uint4 own_o = a.own_out ? reinterpret_cast<const uint4*>(a.own_out + id * 128)[lane] : make_uint4(0, 0, 0, 0);
    float part_lse[kAtOnce];
    float4 part_o[kAtOnce][2];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
        const int64_t part = (int64_t)(min(c0 + k, c1) + run) * a.rows_cap + at;
        part_lse[k] = -INFINITY;
        if (c0 + k <= c1) {
            part_lse[k] = a.ws_lse[part];
            part_o[k][0] = reinterpret_cast<const float4*>(a.ws_o + part * 128)[2 * lane];
            part_o[k][1] = reinterpret_cast<const float4*>(a.ws_o + part * 128)[2 * lane + 1];
        }
    }
    float top = fmaxf(fmaxf(own, part_lse[0]), fmaxf(part_lse[1], part_lse[2]));
    for (int c = c0 + kAtOnce; c <= c1; ++c) top = fmaxf(top, a.ws_lse[(int64_t)(c + run) * a.rows_cap + at]);
    if (top == -INFINITY) top = 0.f;  // no part has seen a key: weights of zero, zeros out, a log-sum-exp of -infinity
    float total = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const auto add = [&](float part, const float4& o, const float4& q) {
        const float wgt = __expf(part - top);
        total += wgt;
        x[0] = fmaf(wgt, o.x, x[0]);
        x[1] = fmaf(wgt, o.y, x[1]);
        x[2] = fmaf(wgt, o.z, x[2]);
        x[3] = fmaf(wgt, o.w, x[3]);
        x[4] = fmaf(wgt, q.x, x[4]);
        x[5] = fmaf(wgt, q.y, x[5]);
        x[6] = fmaf(wgt, q.z, x[6]);
        x[7] = fmaf(wgt, q.w, x[7]);
    };
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
        if (c0 + k <= c1) add(part_lse[k], part_o[k][0], part_o[k][1]);
    for (int c = c0 + kAtOnce; c <= c1; ++c) {
        const int64_t part = (int64_t)(c + run) * a.rows_cap + at;
        const float4* o = reinterpret_cast<const float4*>(a.ws_o + part * 128) + 2 * lane;
        add(a.ws_lse[part], o[0], o[1]);
    }
    if (own != -INFINITY)  // a row without own tokens may hold anything
        add(own, make_float4(dev::bf16_lo(own_o.x), dev::bf16_hi(own_o.x), dev::bf16_lo(own_o.y), dev::bf16_hi(own_o.y)),
            make_float4(dev::bf16_lo(own_o.z), dev::bf16_hi(own_o.z), dev::bf16_lo(own_o.w), dev::bf16_hi(own_o.w)));
    const float inv = total == 0.f ? 0.f : 1.f / total;
    reinterpret_cast<uint4*>(a.out + id * 128)[lane] =
        make_uint4(dev::pack_bf16x2(x[0] * inv, x[1] * inv), dev::pack_bf16x2(x[2] * inv, x[3] * inv),
                   dev::pack_bf16x2(x[4] * inv, x[5] * inv), dev::pack_bf16x2(x[6] * inv, x[7] * inv));
    __syncwarp(__activemask());  // own_lse has been read by the half's lanes before lse, which may be it, is written
    if (lane == 0 && a.lse) a.lse[id] = top + logf(total);
}

}  // namespace attend
}  // namespace mla
