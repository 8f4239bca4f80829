// w4.cu -- mla_linear_w4: out[r,h,n] = t * sum_k x[r,h,k] W[h,n,k] with W in 4 bits and a scale per
// group of k, and mla_w4_pack, which lays such weights out once (declared in include/mla.h).
//
// The weights are the M side of mma.sync m16n8k16 and eight rows of x its N side, so that a decode
// batch fills the instruction and every weight is unpacked once for all rows (up to 64).  tcgen05
// would want the unpacked weights in shared memory and a group's scale cannot be applied inside its
// accumulator; at these row counts the product is bound by the weights' bytes, then by unpacking.
//
// A warp works on blocks of 32 n x 128 k, which the packed layout keeps in 2 KB: lane 4 g + t finds
// its words (q, t), the eight k from 32 q + 8 t, q = 0..3, of rows g, g + 8, g + 16 and g + 24 in four
// 16-byte pieces, so that the codes go from memory to the registers that unpack them, the next
// block's while this one's are worked on, and no barrier is in the loop.  (Codes by cp.async through
// shared memory with a barrier a stage took 34 us where this takes TIME1, at one row, N 8192, K
// 16384.)  Unpacking is bound by the integer pipe, which runs at half the rate of the FMA pipes, so
// it is built from as few integer operations as there are.  A word has k 2 i and 2 i + 1 in nibbles i
// and i + 4:
//   int4: the bits (w & 0x000F000F) are, as a pair of bf16, code 2^-133 (subnormal bf16 is linear in
//         its bits, and still is one binade up, so (w & 0x00F000F0) is 16 code 2^-133); one bf16 FMA
//         with 2^127 or 2^123 and -zero / 64 makes (code - zero) / 64 exactly.  Five integer
//         operations and four FMAs a word.  The MMAs of a group start from zero, and the group's fp32
//         sums are scaled into the output's (the scale times a weight would round in bf16).
//   NVFP4: the code's bits moved to bf16's sign, two exponent bits and one mantissa bit are its value
//         times 2^-126; times scale 2^118 it is exact in bf16 (two times four significant bits).
// The powers of two left over, 2^6 and 2^8, go into the end's product.  x is read as it lies, through
// L1, where the warps of an SM find each other's pieces.  The warps of a block split k (and n, when
// there is little k), and so do the blocks of a cluster when there are few output tiles; the sums are
// joined in a fixed order through (distributed) shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/mla.h"
#include "launch.cuh"
#include "nvtx_range.h"
#include "ptx.cuh"

namespace mla::w4 {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kBlockN = 32, kBlockK = 128;          // of a packed block
constexpr int kBlockBytes = kBlockN * kBlockK / 2;  // its codes
constexpr int kRowTile = 8;                         // rows of x per MMA
constexpr int kMaxRowTiles = 8;
constexpr int kRedPitch = kBlockN + 4;  // floats; the four lanes of a row hit different banks

// Bytes of a block's scales (int4: bf16 [g][j][group], NVFP4: e4m3 [g][t / 2][j][q]) and of its zeros
// (uint8 [g][j][group]), row 8 j + g of the block.
__host__ __device__ constexpr int scale_bytes(int group) { return group == 16 ? kBlockN * 8 : kBlockN * (kBlockK / group) * 2; }
__host__ __device__ constexpr int zero_bytes(int group) { return kBlockN * (kBlockK / group); }

// The packed image: all blocks' codes [h][n / 32][k / 128], then their scales, then their zeros.
struct Layout {
    int64_t blocks_n, blocks_k;  // of one head
    int64_t scale_off, zero_off, bytes;
};
__host__ inline Layout layout_of(const mla_w4_weight& w)
{
    Layout l;
    l.blocks_n = ((int64_t)w.n + kBlockN - 1) / kBlockN;
    l.blocks_k = ((int64_t)w.k + kBlockK - 1) / kBlockK;
    const int64_t blocks = l.blocks_n * l.blocks_k * w.heads;
    l.scale_off = blocks * kBlockBytes;
    l.zero_off = l.scale_off + blocks * scale_bytes(w.group);
    l.bytes = l.zero_off + (w.has_zero ? blocks * zero_bytes(w.group) : 0);
    return l;
}

struct PackArgs {
    const uint8_t* codes;
    const void* scale;
    const uint8_t* zero;
    uint8_t* packed;
    int64_t scale_off, zero_off;
    int n, k, group;
    int blocks_n, blocks_k;
};

// One warp per packed block; n and k past the weights' are filled with zeros of scale zero.
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackArgs a)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, h = blockIdx.y;
    const int64_t b = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (b >= (int64_t)a.blocks_n * a.blocks_k) return;
    const int n0 = (int)(b / a.blocks_k) * kBlockN, k0 = (int)(b % a.blocks_k) * kBlockK;
    const int64_t block = (int64_t)h * a.blocks_n * a.blocks_k + b;
    const int groups = a.k / a.group;  // of a row
    const bool nv = a.group == 16;
    for (int j = 0; j < 4; ++j) {
        const int n = n0 + 8 * j + g;
        const int64_t row = (int64_t)h * a.n + n;
        uint32_t word[4];
        for (int q = 0; q < 4; ++q) {
            const int k = k0 + 32 * q + 8 * t;
            uint32_t w = 0;
            if (n < a.n && k < a.k) {
                const uint32_t v = *reinterpret_cast<const uint32_t*>(a.codes + row * (a.k / 2) + k / 2);
                for (int i = 0; i < 4; ++i)  // nibbles 2 i and 2 i + 1 to i and i + 4
                    w |= ((v >> (8 * i)) & 15u) << (4 * i) | ((v >> (8 * i + 4)) & 15u) << (4 * i + 16);
                // a negative scale's sign goes into its codes
                if (nv && (static_cast<const uint8_t*>(a.scale)[row * groups + k / 16] & 0x80u)) w ^= 0x88888888u;
            }
            word[q] = w;
        }
        *reinterpret_cast<uint4*>(a.packed + block * kBlockBytes + j * 512 + lane * 16) =
            make_uint4(word[0], word[1], word[2], word[3]);
        if (nv) {
            if (t & 1) continue;
            uint32_t s = 0;
            for (int q = 0; q < 4; ++q) {
                const int k = k0 + 32 * q + 8 * t;
                if (n < a.n && k < a.k)
                    s |= (uint32_t)(static_cast<const uint8_t*>(a.scale)[row * groups + k / 16] & 0x7Fu) << (8 * q);
            }
            *reinterpret_cast<uint32_t*>(a.packed + a.scale_off + block * scale_bytes(16) + (g * 2 + (t >> 1)) * 16 + j * 4) = s;
        } else {
            const int count = kBlockK / a.group;
            if (t >= count) continue;
            const int k = k0 + t * a.group;
            const bool in = n < a.n && k < a.k;
            const int at = (g * 4 + j) * count + t;
            reinterpret_cast<uint16_t*>(a.packed + a.scale_off + block * scale_bytes(a.group))[at] =
                in ? static_cast<const uint16_t*>(a.scale)[row * groups + k / a.group] : (uint16_t)0;
            if (a.zero)
                (a.packed + a.zero_off + block * zero_bytes(a.group))[at] =
                    in ? a.zero[row * groups + k / a.group] : (uint8_t)8;
        }
    }
}

struct Args {
    const __nv_bfloat16* x;
    int64_t x_row, x_head;
    const uint8_t* codes;
    const uint8_t* scale;
    const uint8_t* zero;  // NULL: 8
    __nv_bfloat16* out;
    int64_t out_row, out_head;
    float tensor_scale;
    int rows, n, k;
    int blocks_n, blocks_k;
    int k_warps;  // warps of a thread block over k; the others over n
    int splits;   // thread blocks of a cluster, over k
    bool early;   // kernels behind this one may start before it ends (they wait for `out` themselves)
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void prefetch_l2_bulk(const void* p, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
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

// What a lane holds of a block: the codes of its four rows, and their scales and zeros.
template <int kGroup>
struct Held {
    static constexpr int kScale = kGroup == 128 ? 2 : kGroup == 32 ? 8 : 4;  // 32-bit words
    static constexpr int kZero = kGroup >= 32 ? 128 / kGroup : 1;
    uint4 c[4];
    uint32_t s[kScale];
    uint32_t z[kZero];

    // Through L2 only what is read once; the scales' sectors are shared by the four lanes of a row.
    __device__ __forceinline__ void load(const Args& a, int64_t block, int lane)
    {
        const uint4* p = reinterpret_cast<const uint4*>(a.codes + block * kBlockBytes) + lane;
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = __ldcg(p + 32 * j);
        const int g = lane >> 2;
        const uint8_t* ps = a.scale + block * scale_bytes(kGroup);
        if constexpr (kGroup == 16) {
            const uint4 v = __ldcg(reinterpret_cast<const uint4*>(ps) + (lane >> 1));
            s[0] = v.x, s[1] = v.y, s[2] = v.z, s[3] = v.w;
        } else if constexpr (kGroup == 128) {
            const uint2 v = __ldcg(reinterpret_cast<const uint2*>(ps) + g);
            s[0] = v.x, s[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < kScale / 4; ++i) {
                const uint4 v = __ldcg(reinterpret_cast<const uint4*>(ps) + g * (kScale / 4) + i);
                s[4 * i] = v.x, s[4 * i + 1] = v.y, s[4 * i + 2] = v.z, s[4 * i + 3] = v.w;
            }
        }
        if constexpr (kGroup >= 32) {
#pragma unroll
            for (int i = 0; i < kZero; ++i) z[i] = 0x08080808u;
            if (a.zero) {
                const uint8_t* pz = a.zero + block * zero_bytes(kGroup);
                if constexpr (kZero == 1) {
                    z[0] = __ldcg(reinterpret_cast<const uint32_t*>(pz) + g);
                } else if constexpr (kZero == 2) {
                    const uint2 v = __ldcg(reinterpret_cast<const uint2*>(pz) + g);
                    z[0] = v.x, z[1] = v.y;
                } else {
                    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(pz) + g);
                    z[0] = v.x, z[1] = v.y, z[2] = v.z, z[3] = v.w;
                }
            }
        }
    }
    // int4: scale and zero of group i of row 8 j + g
    __device__ __forceinline__ float scale(int j, int i) const
    {
        const int e = j * (kBlockK / kGroup) + i;
        return e & 1 ? dev::bf16_hi(s[e / 2]) : dev::bf16_lo(s[e / 2]);
    }
    __device__ __forceinline__ uint32_t zero64(int j, int i) const
    {
        const int e = j * (kBlockK / kGroup) + i;
        return minus_zero(z[e / 4], e & 3);
    }
};

// x of a block's k: piece (q, t) of rows g + 8 rt
template <int RT>
struct XPieces {
    uint4 v[RT];
};

template <int RT>
__host__ __device__ constexpr int blocks_per_sm()
{
    return RT <= 2 ? 4 : RT <= 5 ? 3 : 2;
}

// kGroup 32, 64, 128: int4; 16: NVFP4.
template <int kGroup, int RT>
__global__ void __launch_bounds__(kThreads, blocks_per_sm<RT>()) linear_w4_kernel(const __grid_constant__ Args a)
{
    using namespace dev;
    constexpr bool kInt4 = kGroup >= 32;
    constexpr int kQ = kInt4 ? kGroup / 32 : 1;  // q's of a group
    extern __shared__ __align__(16) float red[];  // [warp][row][kRedPitch]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int n_warps = kWarps / a.k_warps, wk = warp % a.k_warps, wn = warp / a.k_warps;
    const int rank = (int)blockIdx.x % a.splits, tile = (int)blockIdx.x / a.splits;
    const int bn = tile * n_warps + wn;
    const int h = blockIdx.y, r0 = (int)blockIdx.z * (RT * kRowTile);
    const int first = (int)((int64_t)a.blocks_k * rank / a.splits) + wk;
    const int last = bn < a.blocks_n ? (int)((int64_t)a.blocks_k * (rank + 1) / a.splits) : 0;
    const int64_t row_blocks = ((int64_t)h * a.blocks_n + bn) * a.blocks_k;

    constexpr int kFar = 4;  // blocks of this warp from HBM to L2 ahead
    // Bringing the weights to L2 is no read of them: it may come before the kernel ahead has ended.
    if (lane < kFar && first + lane * a.k_warps < last)
        prefetch_l2_bulk(a.codes + (row_blocks + first + lane * a.k_warps) * kBlockBytes, kBlockBytes);
    griddep_wait();
    if (a.early) griddep_launch_dependents();

    const __nv_bfloat16* xsrc = a.x + (int64_t)(r0 + g) * a.x_row + (int64_t)h * a.x_head + 8 * t;
    const auto load_x = [&](int block, int q, XPieces<RT>& p) {
        const int k = block * kBlockK + 32 * q;
        const bool k_ok = k + 8 * t < a.k;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            p.v[rt] = make_uint4(0u, 0u, 0u, 0u);
            if (k_ok && r0 + g + 8 * rt < a.rows)
                p.v[rt] = __ldca(reinterpret_cast<const uint4*>(xsrc + (int64_t)rt * 8 * a.x_row + k));
        }
    };

    float acc[2][RT][4] = {};
    const auto work = [&](const Held<kGroup>& w, int block, int after) {
        if (lane == 0 && block + kFar * a.k_warps < last)
            prefetch_l2_bulk(a.codes + (row_blocks + block + kFar * a.k_warps) * kBlockBytes, kBlockBytes);
        float part[2][RT][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            XPieces<RT> b;
            load_x(block, q, b);
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
                        unpack_int4(word, w.zero64(j, q / kQ), v[half]);
                    else
                        unpack_e2m1(word, e4m3_scale(w.s[j], q), v[half]);
                }
                const uint32_t a0[4] = {v[0][0], v[1][0], v[0][1], v[1][1]}, a1[4] = {v[0][2], v[1][2], v[0][3], v[1][3]};
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    mma(kInt4 ? part[m][rt] : acc[m][rt], a0, b.v[rt].x, b.v[rt].y);
                    mma(kInt4 ? part[m][rt] : acc[m][rt], a1, b.v[rt].z, b.v[rt].w);
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
    if (first < last) {
        Held<kGroup> even, odd;  // the block worked on and the next one
        even.load(a, row_blocks + first, lane);
        for (int block = first; block < last; block += 2 * a.k_warps) {
            const int second = block + a.k_warps, third = second + a.k_warps;
            if (second < last) odd.load(a, row_blocks + second, lane);
            work(even, block, second);
            if (third < last) even.load(a, row_blocks + third, lane);
            if (second < last) work(odd, second, third);
        }
    }

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
    const int rows = a.rows - r0 < RT * kRowTile ? a.rows - r0 : RT * kRowTile;
    const int width = n_warps * kBlockN, n0 = tile * width;
    const uint32_t rbase = smem_u32(red);
    for (int e = rank * kThreads + tid; e < rows * width; e += a.splits * kThreads) {
        const int r = e / width, c = e % width, n = n0 + c;
        if (n >= a.n) continue;
        const int at = ((c / kBlockN) * a.k_warps * RT * kRowTile + r) * kRedPitch + c % kBlockN;
        float sum = 0.f;
        for (int p = 0; p < a.splits; ++p) {
            const uint32_t peer = a.splits > 1 ? map_to_cta(rbase + at * 4, p) : 0u;
            for (int i = 0; i < a.k_warps; ++i)
                sum += a.splits > 1 ? ld_cluster_f32(peer + i * (RT * kRowTile * kRedPitch * 4))
                                    : red[at + i * (RT * kRowTile * kRedPitch)];
        }
        a.out[(int64_t)(r0 + r) * a.out_row + (int64_t)h * a.out_head + n] =
            __float2bfloat16_rn(sum * (kInt4 ? 64.f : 256.f) * a.tensor_scale);
    }
    __syncwarp();
    if (a.splits > 1) cluster_sync();  // no block leaves while another reads its sums
}

template <int kGroup, int RT>
mla_status launch(const Args& a, int heads, void* stream)
{
    const auto kernel = linear_w4_kernel<kGroup, RT>;
    constexpr int kBytes = kWarps * RT * kRowTile * kRedPitch * 4;
    if (kBytes > 48 * 1024) {
        const mla_status st = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes),
                                          "cudaFuncSetAttribute(max dynamic shared memory)");
        if (st != MLA_OK) return st;
    }
    const int n_warps = kWarps / a.k_warps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.blocks_n + n_warps - 1) / n_warps * a.splits), (unsigned)heads,
                       (unsigned)((a.rows + RT * kRowTile - 1) / (RT * kRowTile)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kBytes;
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

template <int kGroup>
mla_status launch_rows(const Args& a, int heads, void* stream)
{
    switch ((a.rows + kRowTile - 1) / kRowTile) {
        case 1: return launch<kGroup, 1>(a, heads, stream);
        case 2: return launch<kGroup, 2>(a, heads, stream);
        case 3: return launch<kGroup, 3>(a, heads, stream);
        case 4: return launch<kGroup, 4>(a, heads, stream);
        case 5: return launch<kGroup, 5>(a, heads, stream);
        case 6: return launch<kGroup, 6>(a, heads, stream);
        default: return launch<kGroup, 8>(a, heads, stream);
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
    if (w->heads > 65535 || (int64_t)w->heads * w->n >= ((int64_t)1 << 31) || w->k > (1 << 30)) return MLA_ERR_UNSUPPORTED;
    const mla::w4::Layout l = mla::w4::layout_of(*w);
    if (l.blocks_n * l.blocks_k >= ((int64_t)1 << 31)) return MLA_ERR_UNSUPPORTED;
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
    if (rows > 65535 * kMaxRowTiles * kRowTile) return MLA_ERR_UNSUPPORTED;
    const Layout l = layout_of(*w);
    const uint8_t* packed = static_cast<const uint8_t*>(w->packed);
    Args a = {};
    a.x = static_cast<const __nv_bfloat16*>(x);
    a.x_row = x_row_stride;
    a.x_head = x_head_stride;
    a.codes = packed;
    a.scale = packed + l.scale_off;
    a.zero = w->has_zero ? packed + l.zero_off : nullptr;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.out_row = out_row_stride;
    a.out_head = out_head_stride;
    a.tensor_scale = w->tensor_scale;
    a.rows = rows;
    a.n = w->n;
    a.k = w->k;
    a.blocks_n = (int)l.blocks_n;
    a.blocks_k = (int)l.blocks_k;
    a.early = early;
    // As many of a block's warps over k as have two blocks each; the others over n.
    a.k_warps = 1;
    while (a.k_warps < kWarps && a.blocks_k >= 2 * a.k_warps) a.k_warps *= 2;
    // Blocks of a cluster over k: doubled while there are too few for three per SM and every warp
    // keeps two of the packed blocks.
    const int64_t row_blocks = (rows + kMaxRowTiles * kRowTile - 1) / (kMaxRowTiles * kRowTile);
    const int64_t tiles = l.blocks_n * a.k_warps / kWarps * w->heads * row_blocks;
    a.splits = 1;
    while (a.splits < 8 && tiles * a.splits < 3 * 152 && a.blocks_k >= 4 * a.k_warps * a.splits) a.splits *= 2;
    switch (w->group) {
        case 16: return launch_rows<16>(a, w->heads, stream);
        case 32: return launch_rows<32>(a, w->heads, stream);
        case 64: return launch_rows<64>(a, w->heads, stream);
        default: return launch_rows<128>(a, w->heads, stream);
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
    a.scale_off = l.scale_off;
    a.zero_off = l.zero_off;
    a.n = w->n;
    a.k = w->k;
    a.group = w->group;
    a.blocks_n = (int)l.blocks_n;
    a.blocks_k = (int)l.blocks_k;
    const dim3 grid((unsigned)((l.blocks_n * l.blocks_k + 7) / 8), (unsigned)w->heads);
    mla::w4::pack_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return mla::cuda_status(cudaGetLastError(), "4-bit pack kernel launch");
}
