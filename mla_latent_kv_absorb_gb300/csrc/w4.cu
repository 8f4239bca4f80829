// w4.cu -- mla_linear_w4: out[r,h,n] = t * sum_k x[r,h,k] W[h,n,k] with W in 4 bits and a scale per
// group of k (declared in include/mla.h).
//
// The weights are the M side of mma.sync m16n8k16 and eight rows of x its N side, so that a decode
// batch fills the instruction and every weight is unpacked once for all rows (up to 64).  tcgen05
// would want the unpacked weights in shared memory and a group's scale cannot be applied inside its
// accumulator; at these row counts the product is bound by the weights' bytes, then by unpacking.
//
// A block takes 128 outputs of one head: eight warps, four over n (32 each) and two over k.  A stage
// is 256 k: 16 KB of codes, brought by cp.async into a ring, and 4 KB of x per eight rows, which the
// threads bring through registers one stage ahead.  Of a warp's 128 k, lane 4 g + t holds word (q,
// t), the eight k from 32 q + 8 t, of rows g and g + 8.  Unpacking is bound by the integer pipe,
// which runs at half the rate of the FMA pipes (measured: 54 % of it busy where the FMA pipes were
// at 12 %), so it is built from as few integer operations as there are:
//   int4: the bits (w & 0x000F000F) are, as a pair of bf16, code 2^-133 for k i and i + 4 (subnormal
//         bf16 is linear in its bits, and still is one binade up, so (w & 0x00F000F0) is 16 code
//         2^-133); one bf16 FMA with 2^127 or 2^123 and -zero / 64 makes (code - zero) / 64 exactly.
//         Five integer operations and four FMAs a word.  The MMAs of a group start from zero, and
//         the group's fp32 sums are scaled into the output's (the scale times a weight would round
//         in bf16).
//   NVFP4: the code's bits moved to bf16's sign, two exponent bits and one mantissa bit are its value
//         times 2^-126; times scale 2^118 it is exact in bf16 (two times four significant bits).
// The powers of two left over, 2^6 and 2^8, go into the end's product.  x is stored in the order of
// k that the words have, (0, 4), (1, 5), (2, 6), (3, 7).  Blocks of a cluster split k when there are
// few output tiles; their sums, and the two k warps', are joined in a fixed order through
// (distributed) shared memory.
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

constexpr int kThreads = 256;
constexpr int kTileN = 128;
constexpr int kStageK = 256;
constexpr int kCodeBytes = kTileN * kStageK / 2;
constexpr int kRowTile = 8;                       // rows of x per MMA
constexpr int kXBytes = kRowTile * kStageK * 2;   // of one row tile
constexpr int kRedPitch = kTileN + 4;             // floats; the four lanes of a row hit different banks
constexpr int kMaxRowTiles = 8;

template <int RT>
struct Ring {
    // two blocks per SM up to three row tiles, one above
    static constexpr int kBlocks = RT <= 3 ? 2 : 1;
    static constexpr int kStages = RT <= 2 ? 6 : RT == 3 ? 5 : RT <= 5 ? 8 : RT == 6 ? 7 : 6;
    static constexpr int kXOff = kStages * kCodeBytes;
    static constexpr int kXSlot = RT * kXBytes;
    static constexpr int kBytes = kXOff + 2 * kXSlot;
    static_assert((kBytes + 1024) * kBlocks <= 228 * 1024, "shared memory of an SM");
    static_assert(2 * RT * kRowTile * kRedPitch * 4 <= kBytes, "the sums are joined in the ring's memory");
};

struct Args {
    const __nv_bfloat16* x;
    int64_t x_row, x_head;
    const uint8_t* codes;
    const void* scale;
    const uint8_t* zero;
    __nv_bfloat16* out;
    int64_t out_row, out_head;
    float tensor_scale;
    int rows, n, k;
    int splits;   // blocks of a cluster, over k
    bool packed;  // the scales (and zeros) of 128 k are one aligned word
    bool early;   // kernels behind this one may start before it ends (they wait for `out` themselves)
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes of zeros where !valid (src is then not read)
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

__device__ __forceinline__ uint32_t lds32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
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

// -zero / 64 in both halves, of byte j of z
__device__ __forceinline__ uint32_t minus_zero(uint32_t z, int j)
{
    return mul_bf16x2(__byte_perm(z, 0u, 0x4040u | j | (j << 8)), kMinus2p127);
}

// The pairs (i, i + 4), i = 0..3, of a word of eight int4 codes: (code - zero) / 64.
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

// An e4m3 byte of `bytes` as bf16 scale 2^118 in both halves; `sel` places it in bytes 0 and 2.  The
// byte's bits at bf16's exponent and mantissa are scale 2^-120 (subnormals too); two exact products
// raise it.
__device__ __forceinline__ uint32_t e4m3_scale(uint32_t bytes, uint32_t sel)
{
    const uint32_t b = __byte_perm(bytes, 0u, sel);
    return mul_bf16x2(mul_bf16x2(((b << 4) & 0x07F007F0u) | ((b << 8) & 0x80008000u), k2p127), k2p111);
}

// The scales (int4: up to four bf16; NVFP4: eight e4m3) and zeros of one row's 128 k from k0, packed;
// groups at or past k read as 0.  `g` is the row's first scale.
template <int kGroup>
__device__ __forceinline__ void load_scales(const Args& a, int64_t g, int k0, uint2& s, uint32_t& z)
{
    s = make_uint2(0u, 0u);
    z = 0x08080808u;
    g += k0 / kGroup;
    if constexpr (kGroup >= 32) {
        const uint16_t* p = static_cast<const uint16_t*>(a.scale) + g;
        const uint8_t* pz = a.zero + (a.zero ? g : 0);
        if (a.packed) {
            if constexpr (kGroup == 128) {
                s.x = __ldca(p);
                if (a.zero) z = __ldca(pz);
            } else if constexpr (kGroup == 64) {
                s.x = __ldca(reinterpret_cast<const uint32_t*>(p));
                if (a.zero) z = __ldca(reinterpret_cast<const uint16_t*>(pz));
            } else {
                s = __ldca(reinterpret_cast<const uint2*>(p));
                if (a.zero) z = __ldca(reinterpret_cast<const uint32_t*>(pz));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 128 / kGroup; ++i) {
                if (k0 + i * kGroup >= a.k) break;
                (i < 2 ? s.x : s.y) |= (uint32_t)__ldca(p + i) << (16 * (i & 1));
                if (a.zero) z = (z & ~(0xFFu << (8 * i))) | ((uint32_t)__ldca(pz + i) << (8 * i));
            }
        }
    } else {
        const uint8_t* p = static_cast<const uint8_t*>(a.scale) + g;
        if (a.packed) {
            s = __ldca(reinterpret_cast<const uint2*>(p));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (k0 + 16 * i >= a.k) break;
                (i < 4 ? s.x : s.y) |= (uint32_t)__ldca(p + i) << (8 * (i & 3));
            }
        }
    }
}

// kGroup 32, 64, 128: int4; 16: NVFP4.
template <int kGroup, int RT>
__global__ void __launch_bounds__(kThreads, Ring<RT>::kBlocks) linear_w4_kernel(const __grid_constant__ Args a)
{
    using R = Ring<RT>;
    using namespace dev;
    constexpr bool kInt4 = kGroup >= 32;
    constexpr int kQ = kInt4 ? kGroup / 32 : 1;  // q's of a group
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wn = warp & 3, wk = warp >> 2, g = lane >> 2, t = lane & 3;
    const int rank = (int)blockIdx.x % a.splits, n0 = (int)blockIdx.x / a.splits * kTileN;
    const int h = blockIdx.y, r0 = (int)blockIdx.z * (RT * kRowTile);
    const int total = (a.k + kStageK - 1) / kStageK;
    const int first = (int)((int64_t)total * rank / a.splits), last = (int)((int64_t)total * (rank + 1) / a.splits);

    // Codes of a stage: this thread brings 16-byte piece tid % 8 of rows tid / 8 + 32 j.  Rows past n
    // repeat row n - 1 (their sums go nowhere); pieces past k are zeros.
    const int crow = tid >> 3, cpiece = tid & 7;
    const uint8_t* csrc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int n = n0 + crow + 32 * j;
        csrc[j] = a.codes + ((int64_t)h * a.n + (n < a.n ? n : a.n - 1)) * (a.k / 2) + (int64_t)first * (kStageK / 2) +
                  cpiece * 16;
    }
    const uint32_t cdst = sbase + crow * 128 + ((cpiece ^ (crow & 7)) << 4);
    const auto load_codes = [&](int stage, uint32_t slot) {
        if ((stage + 1) * kStageK <= a.k) {
#pragma unroll
            for (int j = 0; j < 4; ++j) cp_async16(cdst + slot * kCodeBytes + j * 32 * 128, csrc[j]);
        } else {
            const bool ok = stage * kStageK + cpiece * 32 < a.k;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                cp_async16_or_zero(cdst + slot * kCodeBytes + j * 32 * 128, ok ? csrc[j] : a.codes, ok);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) csrc[j] += kStageK / 2;
    };
    // x of a stage: piece tid % 32 of rows tid / 32 + 8 j; rows and pieces that are not there are zeros
    const int xrow = tid >> 5, xpiece = tid & 31;
    const __nv_bfloat16* xsrc = a.x + (int64_t)(r0 + xrow) * a.x_row + (int64_t)h * a.x_head + xpiece * 8;
    const uint32_t xdst = sbase + R::kXOff + xrow * 512 + ((xpiece ^ ((xrow & 1) << 2)) << 4);
    uint4 xv[RT];
    const auto load_x = [&](int stage) {
        const bool k_ok = stage * kStageK + xpiece * 8 < a.k;
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            xv[j] = make_uint4(0u, 0u, 0u, 0u);
            if (k_ok && r0 + xrow + 8 * j < a.rows)
                xv[j] = __ldca(reinterpret_cast<const uint4*>(xsrc + (int64_t)j * 8 * a.x_row + stage * kStageK));
        }
    };
    const auto store_x = [&](int slot) {
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            const uint4 v = xv[j];
            sts128(xdst + slot * R::kXSlot + j * kXBytes,
                   make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                              __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632)));
        }
    };
    constexpr int kAhead = R::kStages - 1;
    if (a.early) {  // the step's weights do not depend on the kernel before this one
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (first + i < last) load_codes(first + i, i);
    }
    griddep_wait();
    if (a.early) griddep_launch_dependents();
    load_x(first);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        if (!a.early && first + i < last) load_codes(first + i, i);
        cp_async_commit();
    }
    store_x(0);
    if (first + 1 < last) load_x(first + 1);

    float acc[2][RT][4] = {};
    // first scale of the four rows (m, half); rows past n as above
    const int groups = a.k / kGroup;
    int64_t srow[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = n0 + 32 * wn + 8 * i + g;
        srow[i] = ((int64_t)h * a.n + (n < a.n ? n : a.n - 1)) * groups;
    }
    uint32_t crd[4], xrd[4];  // word (q, t) of row 32 wn + g, and x's
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        crd[q] = sbase + (32 * wn + g) * 128 + (((4 * wk + q) ^ g) << 4) + 4 * t;
        xrd[q] = sbase + R::kXOff + g * 512 + (((16 * wk + 4 * q + t) ^ ((g & 1) << 2)) << 4);
    }
    const uint32_t sel0 = 0x4040u | (t >> 1) | ((t >> 1) << 8), sel1 = sel0 + 0x0202u;  // NVFP4: even and odd q

    uint32_t slot = 0, next = kAhead;
    for (int stage = first, i = 0; stage < last; ++stage, ++i) {
        const int k0 = stage * kStageK + wk * 128;
        const bool busy = k0 < a.k;
        uint2 s[4];
        uint32_t z[4];
        if (busy) {
#pragma unroll
            for (int j = 0; j < 4; ++j) load_scales<kGroup>(a, srow[j], k0, s[j], z[j]);
        }
        cp_async_wait<kAhead - 1>();
        __syncthreads();  // this stage has landed, and every warp has left the one before
        if (stage + kAhead < last) load_codes(stage + kAhead, next);
        cp_async_commit();
        if (stage + 1 < last) store_x((i + 1) & 1);
        if (stage + 2 < last) load_x(stage + 2);
        const uint32_t cat = slot * kCodeBytes, xat = (i & 1) * R::kXSlot;
        slot = slot + 1 == R::kStages ? 0 : slot + 1;
        next = next + 1 == R::kStages ? 0 : next + 1;
        if (!busy) continue;
        float part[2][RT][4];
        uint32_t mz[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint4 b[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) b[rt] = lds128(xrd[q] + xat + rt * kXBytes);
            if (kInt4 && q % kQ == 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) mz[j] = minus_zero(z[j], q / kQ);
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) part[m][rt][e] = 0.f;
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                uint32_t lo[4], hi[4];  // rows g and g + 8
                const uint32_t w0 = lds32(crd[q] + cat + (16 * m) * 128), w1 = lds32(crd[q] + cat + (16 * m + 8) * 128);
                if constexpr (kInt4) {
                    unpack_int4(w0, mz[2 * m], lo);
                    unpack_int4(w1, mz[2 * m + 1], hi);
                } else {
                    const uint32_t sel = q & 1 ? sel1 : sel0;
                    unpack_e2m1(w0, e4m3_scale(q < 2 ? s[2 * m].x : s[2 * m].y, sel), lo);
                    unpack_e2m1(w1, e4m3_scale(q < 2 ? s[2 * m + 1].x : s[2 * m + 1].y, sel), hi);
                }
                const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    mma(kInt4 ? part[m][rt] : acc[m][rt], a0, b[rt].x, b[rt].y);
                    mma(kInt4 ? part[m][rt] : acc[m][rt], a1, b[rt].z, b[rt].w);
                }
            }
            if (kInt4 && q % kQ == kQ - 1) {
                constexpr int kHalf = 2;
                const int j = q / kQ;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float sc[kHalf];
#pragma unroll
                    for (int half = 0; half < kHalf; ++half) {
                        const uint32_t w = j < 2 ? s[2 * m + half].x : s[2 * m + half].y;
                        sc[half] = j & 1 ? bf16_hi(w) : bf16_lo(w);
                    }
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[m][rt][e] += sc[e >> 1] * part[m][rt][e];
                }
            }
        }
    }

    cp_async_wait<0>();
    __syncthreads();  // every warp has left the ring: its memory takes the sums, [wk][row][n]
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[(wk * RT * kRowTile + rt * kRowTile + 2 * t + (e & 1)) * kRedPitch + 32 * wn + 16 * m + 8 * (e >> 1) + g] =
                    acc[m][rt][e];
    __syncwarp();
    if (a.splits > 1)
        cluster_sync();
    else
        __syncthreads();
    const int rows = a.rows - r0 < RT * kRowTile ? a.rows - r0 : RT * kRowTile;
    for (int e = rank * kThreads + tid; e < rows * kTileN; e += a.splits * kThreads) {
        const int r = e / kTileN, n = e % kTileN;
        if (n0 + n >= a.n) continue;
        const uint32_t at = sbase + (r * kRedPitch + n) * 4, other = RT * kRowTile * kRedPitch * 4;
        float sum = 0.f;
        if (a.splits > 1) {
            for (int p = 0; p < a.splits; ++p) {
                const uint32_t peer = map_to_cta(at, p);
                sum += ld_cluster_f32(peer) + ld_cluster_f32(peer + other);
            }
        } else {
            sum = red[r * kRedPitch + n] + red[(RT * kRowTile + r) * kRedPitch + n];
        }
        a.out[(int64_t)(r0 + r) * a.out_row + (int64_t)h * a.out_head + n0 + n] = 
            __float2bfloat16_rn(sum * (kInt4 ? 64.f : 256.f) * a.tensor_scale);
    }
    __syncwarp();
    if (a.splits > 1) cluster_sync();  // no block leaves while another reads its sums
}

template <int kGroup, int RT>
mla_status launch(const Args& a, int heads, void* stream)
{
    const auto kernel = linear_w4_kernel<kGroup, RT>;
    const mla_status st = cuda_status(
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<RT>::kBytes),
        "cudaFuncSetAttribute(max dynamic shared memory)");
    if (st != MLA_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.n + kTileN - 1) / kTileN * a.splits), (unsigned)heads,
                       (unsigned)((a.rows + RT * kRowTile - 1) / (RT * kRowTile)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Ring<RT>::kBytes;
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
    if (w->heads > 65535 || (int64_t)w->heads * w->n >= ((int64_t)1 << 31) || rows > 65535 * kMaxRowTiles * kRowTile)
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
    a.early = early;
    a.packed = w->k % 128 == 0 && is_aligned(w->scale, 8) && is_aligned(w->zero, 4);
    // blocks of a cluster over k: doubled while there are too few tiles for two blocks per SM and
    // every block keeps two stages
    const int64_t row_blocks = (rows + kMaxRowTiles * kRowTile - 1) / (kMaxRowTiles * kRowTile);
    const int64_t tiles = (int64_t)((w->n + kTileN - 1) / kTileN) * w->heads * row_blocks;
    const int stages = (w->k + kStageK - 1) / kStageK;
    a.splits = 1;
    while (a.splits < 8 && tiles * a.splits < 2 * 152 && stages >= 4 * a.splits) a.splits *= 2;
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
