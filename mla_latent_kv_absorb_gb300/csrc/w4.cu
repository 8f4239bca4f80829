// w4.cu -- mla_linear_w4: out[r,h,n] = t * sum_k x[r,h,k] W[h,n,k] with W in 4 bits and a scale per
// group of k, and mla_w4_pack, which lays such weights out once (declared in include/mla.h).
//
// The weights are the M side of mma.sync m16n8k16 and eight rows of x its N side, so that a decode
// batch fills the instruction and every weight is unpacked once for all rows (up to 64).  At a few rows
// the product is bound by the weights' bytes and by unpacking; from some 25 to 40 rows on, where the
// MMAs take longer, the kernel of w4_rows.cuh, on tcgen05, is the faster one for weights of some size.
//
// A warp works on blocks of 32 n x 128 k: lane 4 g + t has the words (q, t), the eight k from 32 q + 8 t,
// q = 0..3, of rows g, g + 8, g + 16 and g + 24.  The packed layout keeps a block's 2 KB of codes in
// that order, its scales and zeros behind them, and the blocks of a thread block's four warps side by
// side, so that one bulk copy brings a step of all four (8 to 10 KB) and a lane reads its part in
// 16-byte pieces.  A ring of four or five steps covers the latency of HBM; x comes by cp.async, two
// steps at a time.  Unpacking is bound by the integer pipe, which runs at half the rate of the FMA
// pipes, so it is built from as few integer operations as there are.  A word has k 2 i and 2 i + 1 in
// nibbles i and i + 4:
//   int4: the bits (w & 0x000F000F) are, as a pair of bf16, code 2^-133 (subnormal bf16 is linear in
//         its bits, and still is one binade up, so (w & 0x00F000F0) is 16 code 2^-133); one bf16 FMA
//         with 2^127 or 2^123 and -zero / 64 makes (code - zero) / 64 exactly.  Five integer
//         operations and four FMAs a word.  The MMAs of a group start from zero, and the group's fp32
//         sums are scaled into the output's (the scale times a weight would round in bf16).
//   NVFP4: the code's bits moved to bf16's sign, two exponent bits and one mantissa bit are its value
//         times 2^-126; times scale 2^118 it is exact in bf16 (two times four significant bits).
// The powers of two left over, 2^6 and 2^8, go into the end's product.  Thread blocks of a cluster
// split k when there are few output tiles; the sums are joined in a fixed order through (distributed)
// shared memory, four outputs a thread.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/mla.h"
#include "launch.cuh"
#include "nvtx_range.h"
#include "ptx.cuh"

namespace mla::w4 {

constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kBlockN = 32, kBlockK = 128;          // of a packed block
constexpr int kCodeBytes = kBlockN * kBlockK / 2;   // its codes
constexpr int kRowTile = 8;                         // rows of x per MMA
constexpr int kMaxRowTiles = 8;
constexpr int kMaxGridZ = 65535;  // blocks of rows
constexpr int kRedPitch = kBlockN + 4;  // floats; the four lanes of a row hit different banks

// Bytes of a block's scales (int4: bf16 [g][j][group], NVFP4: e4m3 [g][t / 2][j][q]) and of its zeros
// (uint8 [g][j][group]), row 8 j + g of the block.
__host__ __device__ constexpr int scale_bytes(int group) { return group == 16 ? kBlockN * 8 : kBlockN * (kBlockK / group) * 2; }
__host__ __device__ constexpr int zero_bytes(int group) { return group == 16 ? 0 : kBlockN * (kBlockK / group); }

// How the four warps of a thread block share its outputs: all over n, so that x is brought for 128
// outputs at a time; two or all four over k where that leaves too few thread blocks for the SMs even
// with clusters of eight over k.  Goes by the weights alone, since they are packed for it.
__host__ inline int k_warps_of(const mla_w4_weight& w)
{
    const int64_t blocks_n = ((int64_t)w.n + kBlockN - 1) / kBlockN, blocks_k = ((int64_t)w.k + kBlockK - 1) / kBlockK;
    int k_warps = 1;
    while (k_warps < kWarps && blocks_k >= 4 * k_warps) {
        const int64_t tiles = (blocks_n * k_warps + kWarps - 1) / kWarps * w.heads, splits = blocks_k / k_warps / 2;
        if (tiles * (splits < 8 ? splits : 8) >= 2 * 152) break;
        k_warps *= 2;
    }
    return k_warps;
}

// The packed image: steps [h][n / (32 kWarps / k_warps)][k / (128 k_warps)] of four blocks, one for each
// warp of a thread block (warp w: w / k_warps over n, w % k_warps over k), each its codes, its scales
// and (has_zero) its zeros, a multiple of 16 bytes.
struct Layout {
    int k_warps;
    int64_t panels, steps;  // of one head
    int block_bytes;
    int64_t bytes;
};
__host__ inline Layout layout_of(const mla_w4_weight& w)
{
    Layout l;
    l.k_warps = k_warps_of(w);
    const int64_t panel_n = kBlockN * kWarps / l.k_warps, step_k = kBlockK * l.k_warps;
    l.panels = (w.n + panel_n - 1) / panel_n;
    l.steps = (w.k + step_k - 1) / step_k;
    l.block_bytes = kCodeBytes + scale_bytes(w.group) + (w.has_zero ? zero_bytes(w.group) : 0);
    l.bytes = l.panels * l.steps * w.heads * kWarps * l.block_bytes;
    return l;
}

// Where lane 4 g + t's 16 bytes of 32 are: lanes in order, and the four t of one g, or one t of eight g,
// hit different banks.
__device__ __forceinline__ int piece_of(int lane) { return lane ^ ((lane >> 3) & 3); }

struct PackArgs {
    const uint8_t* codes;
    const void* scale;
    const uint8_t* zero;
    uint8_t* packed;
    int n, k, group;
    int panels, steps, k_warps, block_bytes;
};

// One warp per packed block; n and k past the weights' are filled with zeros of scale zero.
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackArgs a)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, h = blockIdx.y;
    const int64_t b = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);  // of the head
    if (b >= (int64_t)a.panels * a.steps * kWarps) return;
    const int w = (int)(b % kWarps), step = (int)(b / kWarps % a.steps), panel = (int)(b / kWarps / a.steps);
    const int n0 = (panel * (kWarps / a.k_warps) + w / a.k_warps) * kBlockN, k0 = (step * a.k_warps + w % a.k_warps) * kBlockK;
    uint8_t* block = a.packed + ((int64_t)h * a.panels * a.steps * kWarps + b) * a.block_bytes;
    uint8_t* scales = block + kCodeBytes;
    uint8_t* zeros = scales + scale_bytes(a.group);
    const int groups = a.k / a.group;  // of a row
    const bool nv = a.group == 16;
    for (int j = 0; j < 4; ++j) {
        const int n = n0 + 8 * j + g;
        const int64_t row = (int64_t)h * a.n + n;
        uint32_t word[4];
        for (int q = 0; q < 4; ++q) {
            const int k = k0 + 32 * q + 8 * t;
            uint32_t to = 0;
            if (n < a.n && k < a.k) {
                const uint32_t v = *reinterpret_cast<const uint32_t*>(a.codes + row * (a.k / 2) + k / 2);
                for (int i = 0; i < 4; ++i)  // nibbles 2 i and 2 i + 1 to i and i + 4
                    to |= ((v >> (8 * i)) & 15u) << (4 * i) | ((v >> (8 * i + 4)) & 15u) << (4 * i + 16);
                // a negative scale's sign goes into its codes
                if (nv && (static_cast<const uint8_t*>(a.scale)[row * groups + k / 16] & 0x80u)) to ^= 0x88888888u;
            }
            word[q] = to;
        }
        *reinterpret_cast<uint4*>(block + j * 512 + piece_of(lane) * 16) = make_uint4(word[0], word[1], word[2], word[3]);
        if (nv) {
            if (t & 1) continue;
            uint32_t s = 0;
            for (int q = 0; q < 4; ++q) {
                const int k = k0 + 32 * q + 8 * t;
                if (n < a.n && k < a.k)
                    s |= (uint32_t)(static_cast<const uint8_t*>(a.scale)[row * groups + k / 16] & 0x7Fu) << (8 * q);
            }
            *reinterpret_cast<uint32_t*>(scales + (g * 2 + (t >> 1)) * 16 + j * 4) = s;
        } else {
            const int count = kBlockK / a.group;
            if (t >= count) continue;
            const int k = k0 + t * a.group;
            const bool in = n < a.n && k < a.k;
            const int at = (g * 4 + j) * count + t;
            reinterpret_cast<uint16_t*>(scales)[at] =
                in ? static_cast<const uint16_t*>(a.scale)[row * groups + k / a.group] : (uint16_t)0;
            if (a.zero) zeros[at] = in ? a.zero[row * groups + k / a.group] : (uint8_t)8;
        }
    }
}

struct Args {
    const __nv_bfloat16* x;
    int64_t x_row, x_head;
    const uint8_t* packed;
    int block_bytes;
    uint32_t zero_mask;  // all ones, or 0: every zero is 8
    __nv_bfloat16* out;
    int64_t out_row, out_head;
    float tensor_scale;
    int rows, n, k;
    int steps;    // of 128 k_warps k
    int k_warps;  // warps of a thread block over k; the others over n
    int splits;   // thread blocks of a cluster, over k
    int ring_off, bars_off;  // in shared memory
    bool out_quads;  // four outputs are one aligned 8-byte store
    bool early;      // kernels behind this one may start before it ends (they wait for `out` themselves)
};

__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Four floats of a block of the cluster (after a cluster barrier; not volatile, so that loads from
// several blocks are under way at once).
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr)
{
    float4 v;
    asm("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// `bytes` (a multiple of 16) from global to this block's shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// bf16 pairs of powers of two
constexpr uint32_t k2p127 = 0x7F007F00u, k2p123 = 0x7D007D00u, k2p111 = 0x77007700u, kMinus2p127 = 0xFF00FF00u;

// -zero / 64 in both halves, of byte i of z
__device__ __forceinline__ uint32_t minus_zero(uint32_t z, int i)
{
    return mul_bf16x2(__byte_perm(z, 0u, 0x4040u | i | (i << 8)), kMinus2p127);
}

// The pairs (2 i, 2 i + 1), i = 0..3, of a word of eight int4 codes: (code - zero) / 64.
__device__ __forceinline__ void unpack_int4(uint32_t w, uint32_t z, uint32_t (&v)[4])
{
    const uint32_t u = w >> 8;
    v[0] = fma_bf16x2(w & 0x000F000Fu, k2p127, z);
    v[1] = fma_bf16x2(w & 0x00F000F0u, k2p123, z);
    v[2] = fma_bf16x2(u & 0x000F000Fu, k2p127, z);
    v[3] = fma_bf16x2(u & 0x00F000F0u, k2p123, z);
}

// The same pairs of e2m1 codes times s (scale 2^118 in both halves): values times scale 2^-8.  Left
// shifts only, which the FMA pipe does as products.
__device__ __forceinline__ void unpack_e2m1(uint32_t w, uint32_t s, uint32_t (&v)[4])
{
    const uint32_t u = w >> 8;
    v[0] = mul_bf16x2(((w << 12) & 0x80008000u) | ((w << 6) & 0x01C001C0u), s);
    v[1] = mul_bf16x2(((w << 8) & 0x80008000u) | ((w << 2) & 0x01C001C0u), s);
    v[2] = mul_bf16x2(((u << 12) & 0x80008000u) | ((u << 6) & 0x01C001C0u), s);
    v[3] = mul_bf16x2((w & 0x80008000u) | ((u << 2) & 0x01C001C0u), s);
}

// e4m3 byte i (no sign) of `bytes` as bf16 scale 2^118 in both halves: the byte's bits at bf16's
// exponent and mantissa are scale 2^-120 (subnormals too); two exact products raise it.
__device__ __forceinline__ uint32_t e4m3_scale(uint32_t bytes, int i)
{
    const uint32_t b = __byte_perm(bytes, 0u, 0x4040u | i | (i << 8));
    return mul_bf16x2(mul_bf16x2(b << 4, k2p127), k2p111);
}

// What a lane holds of a block: the codes of its four rows, their scales and zeros.
template <int kGroup>
struct Held {
    static constexpr int kScale = kGroup == 128 ? 2 : kGroup == 32 ? 8 : 4;  // 32-bit words
    static constexpr int kZero = kGroup >= 32 ? 128 / kGroup : 1;
    uint4 c[4];
    uint32_t s[kScale];
    uint32_t z[kZero];

    template <int N>
    static __device__ __forceinline__ void words(uint32_t (&to)[N], const uint8_t* from)
    {
        if constexpr (N == 1) {
            to[0] = *reinterpret_cast<const uint32_t*>(from);
        } else if constexpr (N == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(from);
            to[0] = v.x, to[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const uint4 v = reinterpret_cast<const uint4*>(from)[i];
                to[4 * i] = v.x, to[4 * i + 1] = v.y, to[4 * i + 2] = v.z, to[4 * i + 3] = v.w;
            }
        }
    }
    // from the block's image in shared memory; without zeros the bytes read for them are not used
    __device__ __forceinline__ void load(const uint8_t* image, int lane)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = reinterpret_cast<const uint4*>(image)[32 * j + piece_of(lane)];
        const uint8_t* scales = image + kCodeBytes;
        words(s, scales + (kGroup == 16 ? lane >> 1 : lane >> 2) * (4 * kScale));
        if constexpr (kGroup >= 32) words(z, scales + scale_bytes(kGroup) + (lane >> 2) * (4 * kZero));
    }
    // int4: scale and zero of group i of row 8 j + g
    __device__ __forceinline__ float scale(int j, int i) const
    {
        const int e = j * (kBlockK / kGroup) + i;
        return e & 1 ? dev::bf16_hi(s[e / 2]) : dev::bf16_lo(s[e / 2]);
    }
    __device__ __forceinline__ uint32_t zero64(const Args& a, int j, int i) const
    {
        const int e = j * (kBlockK / kGroup) + i;
        return minus_zero((z[e / 4] & a.zero_mask) | (~a.zero_mask & 0x08080808u), e & 3);
    }
};

// What a thread holds of one row of a block, row 8 j + g for lane 8 j + g.
template <int kGroup>
struct RowOfBlock {
    static constexpr int kCount = kGroup == 16 ? 1 : kBlockK / kGroup;  // groups
    uint4 c[4];     // [t], its words q
    uint32_t s[2];  // NVFP4: scales [t / 2], byte q; int4: zeros in s[0]

    __device__ __forceinline__ void load(const uint8_t* block, int lane)
    {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            c[t] = *reinterpret_cast<const uint4*>(block + lane * 64 + ((t ^ ((lane >> 1) & 3)) << 4));
        const int j = lane >> 3, g = lane & 7;
        const uint8_t* scales = block + kCodeBytes;
        if constexpr (kGroup == 16) {
#pragma unroll
            for (int i = 0; i < 2; ++i) s[i] = *reinterpret_cast<const uint32_t*>(scales + (g * 2 + i) * 16 + j * 4);
        } else {
            const uint8_t* z = scales + scale_bytes(kGroup) + (g * 4 + j) * kCount;
            s[0] = kCount == 1 ? *z : kCount == 2 ? *reinterpret_cast<const uint16_t*>(z) : *reinterpret_cast<const uint32_t*>(z);
        }
    }
    static __device__ __forceinline__ void scales(float (&to)[kCount], const uint8_t* block, int lane)
    {
        const uint16_t* at = reinterpret_cast<const uint16_t*>(block + kCodeBytes) + ((lane & 7) * 4 + (lane >> 3)) * kCount;
#pragma unroll
        for (int i = 0; i < kCount; ++i) to[i] = __uint_as_float((uint32_t)at[i] << 16);
    }
    // The 32 k of q, in pairs.
    __device__ __forceinline__ void unpack(uint32_t zero_mask, int q, uint32_t (&v)[16]) const
    {
        uint32_t zero = 0u;
        if constexpr (kGroup >= 32)
            zero = minus_zero((s[0] & zero_mask) | (~zero_mask & 0x08080808u), q / (kGroup / 32));
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint32_t word = q == 0 ? c[t].x : q == 1 ? c[t].y : q == 2 ? c[t].z : c[t].w;
            uint32_t o[4];
            if constexpr (kGroup >= 32)
                unpack_int4(word, zero, o);
            else
                unpack_e2m1(word, e4m3_scale(s[t >> 1], q), o);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * t + i] = o[i];
        }
    }
};

// Thread blocks per SM, which sets the registers of a thread: 128, 168 or 255.  Three at four and five
// row tiles only where the sums of a group fit without spilling (33 rows, groups of 64: 46 us with
// three and spills, 42 with two; groups of 128: 40 with three, 41 with two).
template <int kGroup, int RT>
__host__ __device__ constexpr int blocks_per_sm()
{
    return RT <= 2 ? 4 : RT == 3 || (RT == 4 && kGroup != 32) || (RT == 5 && (kGroup == 128 || kGroup == 16)) ? 3 : 2;
}

// Shared memory: x's two stages of kStageSteps steps of k_warps pieces of 128 k; a ring of steps'
// packed blocks, with a barrier a slot; afterwards, in the same place, the sums.  A step is one bulk
// copy of 8 to 10 KB: an SM's copy engine takes about the same time for any size (2 KB blocks, a copy
// each, stopped at 5 TB/s with nothing done to them).
constexpr int kStageSteps = 2;
constexpr int kXPiece = kRowTile * kBlockK * 2;  // bytes of 128 k of one row tile
template <int kGroup, int RT>
struct Shared {
    static constexpr int kBlock = kCodeBytes + scale_bytes(kGroup) + zero_bytes(kGroup);
    // as many as leave room for those thread blocks
    static constexpr int kSlots = (RT == 1 && kGroup != 32) || RT == 3 ? 5 : 4;
    static constexpr int kBars = (kSlots + 1) * 8;
    // of a thread block that takes `steps` steps
    static __host__ constexpr int x_bytes(int k_warps, int steps)
    {
        return (steps < 2 * kStageSteps ? steps : 2 * kStageSteps) * k_warps * RT * kXPiece;
    }
    static __host__ constexpr int bytes(int k_warps, int steps)
    {
        const int sums = kWarps * RT * kRowTile * kRedPitch * 4;
        const int rings = x_bytes(k_warps, steps) + kWarps * (steps < kSlots ? steps : kSlots) * kBlock;
        return (sums > rings ? sums : rings) + kBars;
    }
    // thread blocks that an SM holds
    static __host__ constexpr int resident(int k_warps, int steps)
    {
        const int fit = 228 * 1024 / (bytes(k_warps, steps) + 1024);
        return fit < blocks_per_sm<kGroup, RT>() ? fit : blocks_per_sm<kGroup, RT>();
    }
};

// kGroup 32, 64, 128: int4; 16: NVFP4.
template <int kGroup, int RT>
__global__ void __launch_bounds__(kThreads, blocks_per_sm<kGroup, RT>()) linear_w4_kernel(const __grid_constant__ Args a)
{
    using namespace dev;
    constexpr bool kInt4 = kGroup >= 32;
    constexpr int kQ = kInt4 ? kGroup / 32 : 1;  // q's of a group
    using S = Shared<kGroup, RT>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int n_warps = kWarps / a.k_warps, wk = warp % a.k_warps;
    const int rank = (int)blockIdx.x % a.splits, tile = (int)blockIdx.x / a.splits;
    const int h = blockIdx.y, r0 = (int)blockIdx.z * (RT * kRowTile);
    const int begin = (int)((int64_t)a.steps * rank / a.splits), end = (int)((int64_t)a.steps * (rank + 1) / a.splits);
    const int steps = end - begin, stages = (steps + kStageSteps - 1) / kStageSteps;

    // the ring of steps
    const uint32_t sbase = smem_u32(smem);
    const int ring_off = a.ring_off, bars_off = a.bars_off;
    const uint32_t bars = sbase + bars_off;
    volatile int* abort = reinterpret_cast<volatile int*>(smem + bars_off + S::kSlots * 8);
    const WaitCtx wait{kTimeoutNs, abort, nullptr};
    const int step_bytes = kWarps * a.block_bytes;
    const uint8_t* source = a.packed + (((int64_t)h * (gridDim.x / a.splits) + tile) * a.steps + begin) * step_bytes;
    const auto bring = [&](int i) {  // thread 0: step i of this thread block
        const int slot = i % S::kSlots;
        mbar_arrive_expect_tx(bars + 8 * slot, step_bytes);
        bulk_load(sbase + ring_off + slot * (kWarps * S::kBlock), source + (int64_t)i * step_bytes, step_bytes, bars + 8 * slot);
    };
    if (tid == 0) {
        *abort = 0;
        for (int i = 0; i < S::kSlots; ++i) mbar_init(bars + 8 * i, 1);
        fence_barrier_init();
        // Bringing weights to L2 is no read of them: it may come before the kernel ahead has ended,
        // even one that writes them.
        prefetch_l2(source, (steps < S::kSlots ? steps : S::kSlots) * step_bytes);
    }
    griddep_wait();
    if (a.early) griddep_launch_dependents();
    if (tid == 0)
        for (int i = 0; i < S::kSlots && i < steps; ++i) bring(i);

    const __nv_bfloat16* xhead = a.x + (int64_t)h * a.x_head;
    float acc[2][RT][4] = {};
    // a block in w, its x at `ring`
    const auto work = [&](const Held<kGroup>& w, const uint8_t* ring) {
        float part[2][RT][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint4 b[RT];  // piece (q, t) of rows g + 8 rt
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                b[rt] = *reinterpret_cast<const uint4*>(ring + rt * kXPiece + g * (kBlockK * 2) +
                                                        (((4 * q + t) ^ ((g & 1) << 2)) << 4));
            if (kInt4 && q % kQ == 0) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) part[m][rt][e] = 0.f;
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                uint32_t v[2][4];  // rows g and g + 8 of the m tile
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int j = 2 * m + half;
                    const uint32_t word = q == 0 ? w.c[j].x : q == 1 ? w.c[j].y : q == 2 ? w.c[j].z : w.c[j].w;
                    if constexpr (kInt4)
                        unpack_int4(word, w.zero64(a, j, q / kQ), v[half]);
                    else
                        unpack_e2m1(word, e4m3_scale(w.s[j], q), v[half]);
                }
                const uint32_t a0[4] = {v[0][0], v[1][0], v[0][1], v[1][1]}, a1[4] = {v[0][2], v[1][2], v[0][3], v[1][3]};
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    mma(kInt4 ? part[m][rt] : acc[m][rt], a0, b[rt].x, b[rt].y);
                    mma(kInt4 ? part[m][rt] : acc[m][rt], a1, b[rt].z, b[rt].w);
                }
            }
            if (kInt4 && q % kQ == kQ - 1) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const float sc[2] = {w.scale(2 * m, q / kQ), w.scale(2 * m + 1, q / kQ)};
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[m][rt][e] += sc[e >> 1] * part[m][rt][e];
                }
            }
        }
    };
    // x: this thread brings 16 bytes, piece tid % 16 of rows tid / 16 + 8 rt; what is not there is zero
    const int xrow = tid >> 4, xpiece = tid & 15;
    const uint32_t xdst = sbase + xrow * (kBlockK * 2) + ((xpiece ^ ((xrow & 1) << 2)) << 4);
    const __nv_bfloat16* xsrc = xhead + (int64_t)(r0 + xrow) * a.x_row + xpiece * 8;
    const auto load_x = [&](int stage) {
        const int left = steps - stage * kStageSteps, pieces = (left < kStageSteps ? left : kStageSteps) * a.k_warps;
        const uint32_t dst = xdst + (stage & 1) * (kStageSteps * a.k_warps) * (RT * kXPiece);
        for (int i = 0; i < pieces; ++i) {
            const int k = ((begin + stage * kStageSteps) * a.k_warps + i) * kBlockK;
            const bool k_ok = k + xpiece * 8 < a.k;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const bool ok = k_ok && r0 + xrow + 8 * rt < a.rows;
                cp_async16_or_zero(dst + (i * RT + rt) * kXPiece, ok ? xsrc + (int64_t)rt * 8 * a.x_row + k : a.x, ok);
            }
        }
        cp_async_commit();
    };
    load_x(0);
    int slot = 0, phase = 0, taken = 0;
    bool ok = true;
    for (int stage = 0; stage < stages; ++stage) {
        cp_async_wait<0>();
        __syncthreads();  // the stage's x has landed, and every warp has left the stage before
        if (stage + 1 < stages) load_x(stage + 1);
        if (tid == 0 && stage > 0 && ok)  // the slots of the stage before take other steps
            for (int i = taken - kStageSteps + S::kSlots; i < taken + S::kSlots && i < steps; ++i) bring(i);
        const uint8_t* xat = smem + ((stage & 1) * kStageSteps * a.k_warps + wk) * (RT * kXPiece);
#pragma unroll
        for (int sub = 0; sub < kStageSteps; ++sub) {
            if (taken >= steps || !ok) break;
            ok = wait_warp(bars + 8 * slot, phase, wait);
            if (!ok) break;
            Held<kGroup> w;
            w.load(smem + ring_off + slot * (kWarps * S::kBlock) + warp * a.block_bytes, lane);
            ++taken;
            if (++slot == S::kSlots) slot = 0, phase ^= 1;
            work(w, xat + sub * a.k_warps * (RT * kXPiece));
        }
    }
    if (!ok) {  // given up: the outputs say so
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][rt][e] = __uint_as_float(0x7FFFFFFFu);
    }
    if (!ok && tid == 0)  // and what is in flight lands first
        for (int i = taken; i < steps && i < taken + S::kSlots; ++i)
            drain_phase(bars + 8 * (i % S::kSlots), i / S::kSlots, kTimeoutNs);
    cp_async_wait<0>();
    __syncthreads();  // every warp has left the rings: their memory takes the sums, [warp][row][kRedPitch]
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[(warp * RT * kRowTile + rt * kRowTile + 2 * t + (e & 1)) * kRedPitch + 16 * m + 8 * (e >> 1) + g] =
                    acc[m][rt][e];
    __syncwarp();
    if (a.splits > 1)
        cluster_sync();
    else
        __syncthreads();
    // Four outputs a thread; the sums of the k warps and of the cluster's blocks are added in the order
    // of k.
    const int rows = a.rows - r0 < RT * kRowTile ? a.rows - r0 : RT * kRowTile;
    const int quads = n_warps * (kBlockN / 4);
    const int n0 = tile * n_warps * kBlockN;
    constexpr int kWarpSums = RT * kRowTile * kRedPitch;
    for (int e = rank * kThreads + tid; e < rows * quads; e += a.splits * kThreads) {
        const int r = e / quads, c = e % quads * 4, n = n0 + c;
        if (n >= a.n) continue;
        const int at = ((c / kBlockN) * a.k_warps * RT * kRowTile + r) * kRedPitch + c % kBlockN;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        const auto add = [&](const float4& v) { sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w; };
        if (a.splits > 1) {
            for (int i = 0; i < a.k_warps; ++i) {
                float4 v[8];
#pragma unroll
                for (int p = 0; p < 8; ++p)
                    if (p < a.splits) v[p] = ld_cluster_f32x4(map_to_cta(sbase + (at + i * kWarpSums) * 4, p));
#pragma unroll
                for (int p = 0; p < 8; ++p)
                    if (p < a.splits) add(v[p]);
            }
        } else {
            for (int i = 0; i < a.k_warps; ++i) add(*reinterpret_cast<const float4*>(red + at + i * kWarpSums));
        }
        const float scale = kInt4 ? 64.f : 256.f;
        const auto to_bf16 = [&](float f) { return __float2bfloat16_rn(f * scale * a.tensor_scale); };
        alignas(8) const __nv_bfloat16 v[4] = {to_bf16(sum.x), to_bf16(sum.y), to_bf16(sum.z), to_bf16(sum.w)};
        __nv_bfloat16* out = a.out + (int64_t)(r0 + r) * a.out_row + (int64_t)h * a.out_head + n;
        if (a.out_quads && n + 4 <= a.n) {
            *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(v);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < a.n) out[i] = v[i];
        }
    }
    __syncwarp();
    if (a.splits > 1) cluster_sync();  // no block leaves while another reads its sums
}

constexpr int kLimit = 227 * 1024;  // shared memory of a thread block

template <int kGroup, int RT>
mla_status launch(Args a, int heads, int64_t panels, void* stream)
{
    using S = Shared<kGroup, RT>;
    const auto kernel = linear_w4_kernel<kGroup, RT>;
    const int row_blocks = (a.rows + RT * kRowTile - 1) / (RT * kRowTile);
    if (row_blocks > kMaxGridZ) return MLA_ERR_UNSUPPORTED;
    const int64_t tiles = panels * heads * row_blocks;
    // Thread blocks of a cluster over k: as many as still start at once (clusters leave some of the
    // places on the SMs empty: nine tenths are counted on), with four steps or more for each.
    a.splits = 1;
    for (const int s : {8, 6, 4, 2}) {
        if (a.steps < 4 * s || tiles * s * 10 > 9 * 152 * S::resident(a.k_warps, (a.steps + s - 1) / s)) continue;
        a.splits = s;
        break;
    }
    const int steps = (a.steps + a.splits - 1) / a.splits, bytes = S::bytes(a.k_warps, steps);
    if (bytes > kLimit) return MLA_ERR_UNSUPPORTED;
    a.ring_off = S::x_bytes(a.k_warps, steps);
    a.bars_off = bytes - S::kBars;
    // The kernel's limit is the process's: set to the same value by every call, the most that any asks
    // for (full rings, four warps over k), so that no thread lowers it between another's set and launch.
    constexpr int kFull = S::bytes(kWarps, 2 * kStageSteps + S::kSlots), kMost = kFull < kLimit ? kFull : kLimit;
    const mla_status st = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost),
                                      "cudaFuncSetAttribute(max dynamic shared memory)");
    if (st != MLA_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(panels * a.splits), (unsigned)heads, (unsigned)row_blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
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
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, a), "4-bit product kernel launch");
}

}  // namespace mla::w4

#include "w4_rows.cuh"

namespace mla::w4 {

template <int kGroup>
mla_status launch_rows(const Args& a, const mla_w4_weight& w, const Layout& l, void* stream)
{
    const int heads = w.heads;
    const int64_t panels = l.panels;
    if (rows::faster<kGroup>(a, w, l)) return rows::launch<kGroup>(a, w, l, stream);
    int row_tiles = (a.rows + kRowTile - 1) / kRowTile;
    // with four warps over k, x of more than 40 rows does not fit the shared memory: two thread blocks
    if (a.k_warps == kWarps && row_tiles > 5) row_tiles = row_tiles <= 6 ? 3 : 4;
    switch (row_tiles) {
        case 1: return launch<kGroup, 1>(a, heads, panels, stream);
        case 2: return launch<kGroup, 2>(a, heads, panels, stream);
        case 3: return launch<kGroup, 3>(a, heads, panels, stream);
        case 4: return launch<kGroup, 4>(a, heads, panels, stream);
        case 5: return launch<kGroup, 5>(a, heads, panels, stream);
        case 6: return launch<kGroup, 6>(a, heads, panels, stream);
        default: return launch<kGroup, 8>(a, heads, panels, stream);
    }
}

}  // namespace mla::w4

namespace {

using mla::is_aligned;

// Format, sizes and group of a weight.
mla_status check_shape(const mla_w4_weight* w)
{
    if (!w || (w->format != MLA_W4_INT4 && w->format != MLA_W4_NVFP4)) return MLA_ERR_INVALID_ARG;
    const bool int4 = w->format == MLA_W4_INT4;
    if (w->heads < 1 || w->n < 1 || w->k < 1 || !std::isfinite(w->tensor_scale)) return MLA_ERR_INVALID_ARG;
    if (int4 ? (w->group != 32 && w->group != 64 && w->group != 128) : w->group != 16) return MLA_ERR_INVALID_ARG;
    if (w->k % w->group || w->k % 32 || (w->has_zero != 0 && w->has_zero != 1) || (!int4 && w->has_zero))
        return MLA_ERR_INVALID_ARG;
    // outputs fit 32 bits with those that fill up a pair of tiles (256)
    if (w->heads > 65535 || (int64_t)w->heads * w->n > ((int64_t)1 << 31) - 256 || w->k > (1 << 30)) return MLA_ERR_UNSUPPORTED;
    const mla::w4::Layout l = mla::w4::layout_of(*w);
    if (l.panels * l.steps * mla::w4::kWarps >= ((int64_t)1 << 31)) return MLA_ERR_UNSUPPORTED;
    return MLA_OK;
}

mla_status linear_w4(int32_t rows, const void* x, int64_t x_row_stride, int64_t x_head_stride, const mla_w4_weight* w,
                     void* out, int64_t out_row_stride, int64_t out_head_stride, bool early, void* stream)
{
    using namespace mla::w4;
    constexpr int64_t kMaxStride = (int64_t)1 << 40;
    const auto stride_ok = [](int64_t s) { return s >= 0 && s <= kMaxStride; };
    if (rows < 0) return MLA_ERR_INVALID_ARG;
    const mla_status shape = check_shape(w);
    if (shape != MLA_OK) return shape;
    if (!stride_ok(x_row_stride) || !stride_ok(x_head_stride) || !stride_ok(out_row_stride) || !stride_ok(out_head_stride))
        return MLA_ERR_INVALID_ARG;
    if (rows == 0) return MLA_OK;
    if (!x || !out || !w->packed || x == out) return MLA_ERR_INVALID_ARG;
    if (!mla::distinct_elements(rows, out_row_stride, w->heads, out_head_stride, w->n)) return MLA_ERR_INVALID_ARG;
    if (!is_aligned(x, 16) || !is_aligned(w->packed, 16) || !is_aligned(out, 2) || (rows > 1 && x_row_stride % 8) ||
        (w->heads > 1 && x_head_stride % 8))
        return MLA_ERR_ALIGNMENT;
    if (rows > kMaxGridZ * kMaxRowTiles * kRowTile) return MLA_ERR_UNSUPPORTED;  // of 64 rows a thread block
    const Layout l = layout_of(*w);
    Args a = {};
    a.x = static_cast<const __nv_bfloat16*>(x);
    a.x_row = x_row_stride;
    a.x_head = x_head_stride;
    a.packed = static_cast<const uint8_t*>(w->packed);
    a.block_bytes = l.block_bytes;
    a.zero_mask = w->has_zero ? 0xFFFFFFFFu : 0u;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.out_row = out_row_stride;
    a.out_head = out_head_stride;
    a.tensor_scale = w->tensor_scale;
    a.rows = rows;
    a.n = w->n;
    a.k = w->k;
    a.steps = (int)l.steps;
    a.k_warps = l.k_warps;
    a.early = early;
    a.out_quads = is_aligned(out, 8) && (rows == 1 || out_row_stride % 4 == 0) && (w->heads == 1 || out_head_stride % 4 == 0);
    switch (w->group) {
        case 16: return launch_rows<16>(a, *w, l, stream);
        case 32: return launch_rows<32>(a, *w, l, stream);
        case 64: return launch_rows<64>(a, *w, l, stream);
        default: return launch_rows<128>(a, *w, l, stream);
    }
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

extern "C" MLA_API size_t mla_w4_packed_bytes(const mla_w4_weight* w)
{
    return check_shape(w) == MLA_OK ? (size_t)mla::w4::layout_of(*w).bytes : 0;
}

extern "C" MLA_API mla_status mla_w4_pack(const mla_w4_weight* w, const void* codes, const void* scale,
                                          const void* zero, void* packed, void* stream)
{
    const mla::NvtxRange nvtx_range("mla_w4_pack");
    const mla_status shape = check_shape(w);
    if (shape != MLA_OK) return shape;
    if (!codes || !scale || !packed || (w->has_zero != 0) != (zero != nullptr)) return MLA_ERR_INVALID_ARG;
    if (!is_aligned(codes, 16) || !is_aligned(packed, 16) || (w->format == MLA_W4_INT4 && !is_aligned(scale, 2)))
        return MLA_ERR_ALIGNMENT;
    const mla::w4::Layout l = mla::w4::layout_of(*w);
    mla::w4::PackArgs a = {};
    a.codes = static_cast<const uint8_t*>(codes);
    a.scale = scale;
    a.zero = static_cast<const uint8_t*>(zero);
    a.packed = static_cast<uint8_t*>(packed);
    a.n = w->n;
    a.k = w->k;
    a.group = w->group;
    a.panels = (int)l.panels;
    a.steps = (int)l.steps;
    a.k_warps = l.k_warps;
    a.block_bytes = l.block_bytes;
    const dim3 grid((unsigned)((l.panels * l.steps * mla::w4::kWarps + 7) / 8), (unsigned)w->heads);
    mla::w4::pack_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return mla::cuda_status(cudaGetLastError(), "4-bit pack kernel launch");
}
