// Products of microscaled 4-bit or 16-bit operands on the tensor cores, dense or one per expert over
// ragged row groups:
//   C[m][n] = act(a_scale[m] * b_scale[e][n] * sum_k A[m][k] B[e][n][k] + bias[e][n]) + residual[m][n].
//
// As in prefill_kernel.cuh the product is computed transposed, D[n][m] = sum_k B[n][k] A[m][k]: the
// weight's 128 channels are the MMA's 128 rows, and the activation rows its N, which the instruction
// takes in steps of 16. So a group of a few rows costs a few columns, not a padded tile, and one
// kernel serves single tokens and long prompts. The 4-bit formats are multiplied as they are
// (kind::mxf4 / mxf4nvf4: 64 of K per instruction, the block scales applied inside), so nothing is
// dequantized anywhere.
//
// A thread block runs through output tiles (128 channels x up to BN rows of one group). Roles:
//   warp 0      TMA: per pipeline stage 128 bytes of K (256 values in 4 bits, 64 in 16) of the tile's
//               weight rows and activation rows (128-byte swizzle), and the weight's scale tiles, which
//               are stored in the order the tensor cores take them;
//   warps 2, 3  the activations' scales, stored row by row because a group may start at any row, brought
//               into that same order through registers;
//   warp 1      one lane copies a stage's scales to tensor memory (tcgen05.cp; copies and MMAs of one
//               thread run in issue order) and issues its MMAs, accumulating in tensor memory;
//   warps 4-11  read the accumulator, apply the epilogue and store. The next tile's MMAs run meanwhile
//               in a second accumulator. Two of 256 columns do not fit beside the scales: they overlap in
//               32 (MXFP4) or 48 columns, which the epilogue reads first.
// Groups are found in the kernel from the offsets (the host never reads them): each block sums the
// groups' tile counts once, and finds a tile's group by binary search.
//
// SPLIT: with too few tiles to fill the GPU, the blocks of a cluster share a tile, each taking a part
// of K. Each block is sent its share of the channels' partial sums by all of them (asynchronous stores to
// distributed shared memory, counted by a barrier: no fence between blocks) and adds them in rank
// order. Tiles of up to 32 rows store their sums one by one; larger ones (4 bytes at a time they
// took 4 us for 64 rows) turn them in shared memory and send one bulk copy to each block, which for
// a few rows takes 0.5 us longer. No workspace, no atomics, one launch. A cluster has one tile at most.
//
// What bounds it, and what it measured (bf16 output, no bias or activation, calls in a graph):
//   few rows    the weight's bytes from HBM, once: 64 rows of 32 experts, 2560 x 9728, MXFP4: 49 us,
//               6.3 TB/s (NVFP4 50 us). With fewer tiles than SMs the SMs that work: 1 x 4096 x 11008 is 86
//               blocks of 16 stages, 6.8 us (3.3 TB/s; NVFP4 7.3). For the smallest the launch, the first
//               loads and the join: 16 x 4096 x 4096 5.1 us;
//   many rows   16 bits: the tensor cores (2048 x 4096 x 14336 122 us, 1970 TFLOPS). 4 bits: an MMA of a
//               pair takes 97 cycles, six times the 16-bit rate, and a stage's four MMAs no longer cover what
//               goes on beside them: 36 KB from L2 to each SM, the scale copies and the epilogue. Each of
//               these left out makes about a fifth; tiles of 240 rows, whose accumulators share no
//               columns, make nothing (44 us and 161 -> 167 below). MXFP4 2048 x 4096 x 14336 41 us (5.8
//               PFLOPS; tensor pipe 57 %, HBM 14 %; 42.8 with SiLU, 46 to 47 with SiLU and bias on inputs that
//               change from call to call), SwiGLU over 32768 rows of 32 experts, 2560 x 5120, 160 us (5.4
//               PFLOPS; 171 to 173 on changing inputs). NVFP4 has twice the scales to copy: 56 us and 207
//               to 215.
//
// Every wait is bounded (see ptx.cuh); after an abort the copies and MMAs in flight are waited for,
// and a cluster's blocks leave together.
#pragma once

#include <type_traits>

#include "epilogue.cuh"
#include "experts.cuh"
#include "fp4.cuh"
#include "group_plan.h"
#include "ptx.cuh"

namespace qg {
namespace gg {

constexpr int kThreads = 384;
constexpr int kEpiWarp = 4, kEpiWarps = 8, kEpiThreads = kEpiWarps * 32;
constexpr int kScaleWarp = 2;
constexpr int kRowBytes = 128;                     // K bytes of a row per stage
constexpr int kMaxStages = 10;
constexpr long long kDrainNs = 20000000;           // limit of a wait for copies in flight after an abort
constexpr size_t kSmemMax = 232448;
constexpr int kTail = 1024;                        // barriers

// Operand forms: 16-bit, or 4-bit with 2 (MXFP4) or 4 (NVFP4) scale tiles per stage.
enum Form { HALF = 0, MX = 1, NV = 2 };
// Blocks and tiles: one block a tile; a cluster that shares a tile's K; two blocks a tile of 256 channels.
enum Mode { SOLO = 0, SPLIT = 1, PAIR = 2 };
template <int F, int BN, int MODE>
struct Plan {
    static constexpr int kChunks = F == HALF ? 0 : (F == MX ? 2 : 4);      // scale tiles (128 rows x 4) per stage
    static constexpr int kHalves = (BN + 127) / 128;                       // ... of the activations, per 128 rows
    static constexpr int kTileCh = MODE == PAIR ? 2 * kCh : kCh;            // channels of a tile
    static constexpr int kBRows = MODE == PAIR ? BN / 2 : BN;              // activation rows in this block's stage
    static constexpr int kA = kCh * kRowBytes, kB = kBRows * kRowBytes;
    static constexpr int kSA = kChunks * 512, kSB = kChunks * kHalves * 512;
    static constexpr int kStage = kA + kB + kSA + kSB;
    static constexpr int kRed = MODE == SPLIT ? kCh * BN * 4 : 0;          // partial sums received, [block][row][channel of the share]
    static constexpr int kTables = 2 * (1024 + 1) * 4;                     // group starts and tile counts
    static constexpr int kRoom = (int)kSmemMax - kTail - kTables - kRed;
    static constexpr int kStages = kRoom / kStage < kMaxStages ? kRoom / kStage : kMaxStages;
    static constexpr size_t kSmem = (size_t)kStages * kStage + kRed + kTail + kTables;
    static constexpr int kBoxRows = BN == 32 ? 16 : 64;                 // rows of one activation box
    // tensor-memory columns: two accumulators, then the scales of a stage
    static constexpr int kScaleCols = kChunks * (1 + kHalves) * 4;
    static constexpr bool kOverlap = 2 * BN + kScaleCols > 512;
    static constexpr int kAcc1 = kOverlap ? (512 - kScaleCols - BN) / 16 * 16 : BN;
    static constexpr int kSaCol = kAcc1 + BN, kSbCol = kSaCol + 4 * kChunks;
    static constexpr int kWide = BN == 32 ? 16 : 32;                       // columns of an epilogue chunk
    static constexpr int kShared = kOverlap ? (BN - kAcc1 + kWide - 1) / kWide : 0;      // chunks with shared columns
    static_assert(kStage % 1024 == 0, "stages keep the 128-byte swizzle's alignment");
    static_assert(kStages >= 4, "ring");
    static_assert(kAcc1 + BN + kScaleCols <= 512, "tensor memory");
};

struct Params {
    int M, E, K, N, cols;      // cols: C's columns (N, or N / 2 for SwiGLU)
    int n_tiles, stages;       // channel tiles; stages of K
    int ch_tiles;              // 128-channel tiles of the weight's scales
    int bf16;                  // HALF: bf16 (else f16)
    int split;                 // blocks of a cluster (1, 2 for PAIR)
    const int32_t* offsets;
    const uint8_t* As;
    int pitch;                 // bytes of a row of As
    int ktiles;                // the weight's scale tiles along K
    const float* a_scale;
    const float* b_scale;
    const float* bias;
    const void* residual;
    void* C;
    int act, c_dtype;
    unsigned int* status;
    long long wait_ns;
    int stall;
};
struct Maps {
    CUtensorMap a;             // activations [M][row bytes]
    CUtensorMap b;             // weights [E][N][row bytes]
    CUtensorMap sb;            // the weights' scale tiles [E x channel tiles x K tiles][512 bytes]
};

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptors, the high words: K-major rows of 128 bytes with the 128-byte
// swizzle (8-row atoms 1024 bytes apart), and a 32 x 16-byte scale tile without swizzle (8-row groups 128
// bytes apart). The low word is the address in units of 16 bytes (14 bits, so that adding offsets
// inside shared memory never carries) and, for the rows, a leading offset of 1.
constexpr uint32_t kRowsHi = (1024u >> 4) | (1u << 14) | (2u << 29), kScaleHi = (128u >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t rows_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t scale_lo(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4; }
// Scale tile (512 bytes) to four tensor-memory columns, in all four lane quarters (PAIR: each block's
// own tile to its own columns).
template <int MODE>
__device__ __forceinline__ void copy_scales(uint32_t tcol, uint32_t lo) {
    if constexpr (MODE == PAIR)
        asm volatile("{\n\t.reg .pred e;\n\t.reg .b64 x;\n\tmov.b64 x, {%1, %2};\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], x;\n\t}" ::"r"(tcol), "r"(lo), "n"(kScaleHi)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred e;\n\t.reg .b64 x;\n\tmov.b64 x, {%1, %2};\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], x;\n\t}" ::"r"(tcol), "r"(lo), "n"(kScaleHi)
                     : "memory");
}
// Instruction descriptors for m rows (128, PAIR: 256) and n columns. 16-bit: float32 D, A and B
// both f16 (0) or bf16 (1). 4-bit: A and B e2m1, scales e4m3 (0) or e8m0 (1 at bit 23), and which of a
// column's four scale bytes come first (sf: A's at bit 29, B's at bit 4).
template <int F>
__device__ __forceinline__ uint32_t inst_desc(int m, int n, int bf16) {
    if constexpr (F == HALF)
        return (1u << 4) | ((uint32_t)bf16 << 7) | ((uint32_t)bf16 << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((F == MX ? 1u : 0u) << 23) | ((uint32_t)(m >> 7) << 27);
}
// One MMA over 32 bytes of K, issued by one elected lane of the warp: D (+)= A x B, both from shared
// memory (PAIR: each block holds its 128 rows of A and D and half of B's columns). a, b: low words.
#define QG_MMA(GROUP, KIND, ...)                                                                               \
    asm volatile(                                                                                               \
        "{\n\t.reg .pred p, e;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"               \
        "setp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t@e tcgen05.mma.cta_group::" GROUP "." KIND ", p;\n\t}" ::"r"(d), \
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kRowsHi), ##__VA_ARGS__                                        \
        : "memory")
template <int F, int MODE>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t acc) {
    if constexpr (F == HALF) {
        if constexpr (MODE == PAIR) QG_MMA("2", "kind::f16 [%0], x, y, %3");
        else QG_MMA("1", "kind::f16 [%0], x, y, %3");
    } else if constexpr (F == MX) {
        if constexpr (MODE == PAIR) QG_MMA("2", "kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %3, [%6], [%7]", "r"(sa), "r"(sb));
        else QG_MMA("1", "kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %3, [%6], [%7]", "r"(sa), "r"(sb));
    } else {
        if constexpr (MODE == PAIR) QG_MMA("2", "kind::mxf4nvf4.block_scale.scale_vec::4X [%0], x, y, %3, [%6], [%7]", "r"(sa), "r"(sb));
        else QG_MMA("1", "kind::mxf4nvf4.block_scale.scale_vec::4X [%0], x, y, %3, [%6], [%7]", "r"(sa), "r"(sb));
    }
}
#undef QG_MMA
// One arrival on `bar` (PAIR: in both blocks) once the copies and MMAs issued so far are done.
template <int MODE>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    if constexpr (MODE == PAIR)
        asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
                     "h"((uint16_t)3)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
                     : "memory");
}
// Tiled TMA loads into this block's shared memory; with PAIR, `bar` may be the other block's.
template <int MODE>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    if constexpr (MODE == PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        ptx::tma_load_2d(dst, map, x, y, bar);
}
template <int MODE>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    if constexpr (MODE == PAIR)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        ptx::tma_load_3d(dst, map, x, y, z, bar);
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// (relaxed: the barrier orders lifetimes; what the blocks exchange is ordered by mbarriers, and the
// mbarriers' initialization by its own fence. A release would wait for the thread's memory accesses.)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// Address of this block's shared-memory location in the cluster's block `rank`.
__device__ __forceinline__ uint32_t peer(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
// An arrival on a barrier of another block. By itself it orders execution at cluster scope, which with
// tcgen05.fence on both sides is what tensor memory needs.
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Makes the arrival after it release this block's shared memory to the cluster (the waits acquire at that
// scope). Shared memory alone: an arrival that releases all memory waits for every load of the thread in
// flight, and takes a few thousand cycles even from a thread that has none (2048 x 4096 x 14336: 99 and
// 112 us instead of 41).
__device__ __forceinline__ void release_shared() {
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
}
// A value to another block's shared memory, counted in bytes by a barrier of that block.
__device__ __forceinline__ void peer_store(uint32_t addr, float v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(addr), "f"(v), "r"(bar) : "memory");
}
// Bulk copy of this block's shared memory into another's, counted in bytes by a barrier of that block.
__device__ __forceinline__ void peer_copy(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "r"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
// ptx.cuh's waits for barriers that other blocks of the cluster arrive on.
__device__ __forceinline__ bool cluster_bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool cluster_bar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned int* status,
                                                 long long limit_ns) {
    if (cluster_bar_try(bar, parity)) return true;
    return ptx::mbar_wait(bar, parity, abort_flag, status, limit_ns) && cluster_bar_try(bar, parity);
}
// A look that never suspends the warp.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// True in one lane of the (converged) warp. The instructions that a single thread issues (TMA,
// tcgen05.mma, tcgen05.cp) take their operands from warp-wide registers; elect.sync tells the
// compiler that one lane is active (under `lane == 0` each of them measured 88 cycles).
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

struct Tile {
    int e, n0, m0, rows;       // expert, first channel (of this block), first row, rows
};

// Two neighbouring channels' values of the chunk's 2 W rows, exchanged between the lanes of a pair: the
// even lane ends with both channels of the first W rows (first[i], second[i]), the odd lane of the rest.
template <int W>
__device__ __forceinline__ void pair_up(const float (&v)[2 * W], float (&first)[W], float (&second)[W], bool odd) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + W], 1);
        first[i] = odd ? got : v[i];
        second[i] = odd ? v[i + W] : got;
    }
}

// v * sigmoid(v), for the tensor-core tiles: the exponential and the reciprocal without the handling
// of subnormal numbers, which cannot show in 1 + e^-v (half the instructions of epilogue.cuh's form, the
// same few units in the last place).
__device__ __forceinline__ float silu(float v) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return v * r;
}
// max(v, 0) that keeps a NaN: an operand's NaN scale marks its row or channel of C behind every
// activation (fmaxf would make it 0).
__device__ __forceinline__ float relu(float v) {
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
    return r;
}
template <int ACT, int W>
__device__ __forceinline__ void act_all(float (&v)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = ACT == ACT_SILU ? silu(v[i]) : (ACT == ACT_RELU ? relu(v[i]) : act_fixed<ACT>(v[i]));
}

template <int CDT>
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
    uint32_t w;
    if constexpr (CDT == DT_F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}
// Of two words that hold two rows (halves) of one channel each, exchanged between lanes `mask` apart:
// both channels of the first row (lower lane) or of the second (upper lane).
__device__ __forceinline__ uint32_t both_channels(uint32_t own, int mask, bool upper) {
    return __byte_perm(own, __shfl_xor_sync(0xffffffffu, own, mask), upper ? 0x3276u : 0x5410u);
}

// The rest of the epilogue for 2 W rows from m on (the first `live` of them; FULL: all) of channel n:
// activation, residual, rounding, stores. One choice of activation and type per chunk, none per value;
// the number of instructions here is what bounds tiles of short K. 16-bit outputs are rounded two rows to
// a word and leave as pairs of channels (64 contiguous bytes a row), of the first W rows from the even
// lanes and the others from the odd ones; SwiGLU pairs become one channel the same way, and channels of
// neighbouring pairs leave together.
template <int CDT, int W, bool FULL>
__device__ __forceinline__ void store_chunk(const Params& p, float (&v)[2 * W], int n, int m, int live, int lane) {
    constexpr size_t kEsz = CDT == DT_F32 ? 4 : 2;
    switch (p.act) {
        case ACT_RELU: act_all<ACT_RELU>(v); break;
        case ACT_SILU: act_all<ACT_SILU>(v); break;
        case ACT_GELU_TANH: act_all<ACT_GELU_TANH>(v); break;
        default: break;
    }
    const bool glu = p.act == ACT_SWIGLU, odd = lane & 1;
    const size_t step = (size_t)p.cols * kEsz;
    // `count` values of one channel in consecutive rows
    auto column = [&](float* y, int row, int col, int rows, auto count) {
        constexpr int kCount = decltype(count)::value;
        const size_t at = (size_t)row * p.cols + col;
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < kCount; ++i)
                if (i < rows) y[i] += load_as_float<CDT>(p.residual, at + (size_t)i * p.cols);
        }
        uint8_t* out = static_cast<uint8_t*>(p.C) + at * kEsz;
#pragma unroll
        for (int i = 0; i < kCount; ++i, out += step)
            if (i < rows) store_out_rt(out, 0, y[i], CDT);
    };
    const int half = odd ? W : 0;      // this lane's rows after an exchange with its neighbour
    if (glu) {
        float a[W], b[W];
        pair_up<W>(v, a, b, odd);
#pragma unroll
        for (int i = 0; i < W; ++i) a[i] = silu(a[i]) * b[i];
        if (CDT != DT_F32 && !p.residual && (p.cols & 1) == 0) {
            const int second = (lane >> 1) & 1;
            uint8_t* out = static_cast<uint8_t*>(p.C) + ((size_t)(m + half + second) * p.cols + ((n >> 1) & ~1)) * kEsz;
#pragma unroll
            for (int i = 0; i < W; i += 2, out += 2 * step) {
                const uint32_t w = both_channels(round2<CDT>(a[i], a[i + 1]), 2, second);
                if (n < p.N && (FULL || half + second + i < live)) *reinterpret_cast<uint32_t*>(out) = w;
            }
        } else if (n < p.N) {
            column(a, m + half, n >> 1, live - half, std::integral_constant<int, W>());
        }
    } else if (CDT != DT_F32 && (p.N & 1) == 0) {
        const size_t at = ((size_t)(m + half) * p.cols + (n & ~1)) * kEsz;
        uint8_t* out = static_cast<uint8_t*>(p.C) + at;
        if (!p.residual) {
#pragma unroll
            for (int i = 0; i < W; ++i, out += step) {
                const uint32_t w = both_channels(round2<CDT>(v[i], v[i + W]), 1, odd);
                if (n < p.N && (FULL || half + i < live)) *reinterpret_cast<uint32_t*>(out) = w;
            }
            return;
        }
        float a[W], b[W];
        pair_up<W>(v, a, b, odd);
        if (n >= p.N) return;              // (N is even here: both lanes of a pair)
        uint32_t r[W];
#pragma unroll
        for (int i = 0; i < W; ++i)
            r[i] = half + i < live ? load(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.residual) + at + i * step)) : 0u;
#pragma unroll
        for (int i = 0; i < W; ++i, out += step) {
            float2 f;
            if constexpr (CDT == DT_F16) f = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
            else f = make_float2(__uint_as_float(r[i] << 16), __uint_as_float(r[i] & 0xFFFF0000u));
            if (half + i < live) *reinterpret_cast<uint32_t*>(out) = round2<CDT>(a[i] + f.x, b[i] + f.y);
        }
    } else if (n < p.N) {
        column(v, m, n, live, std::integral_constant<int, 2 * W>());
    }
}
template <int CDT, int W>
__device__ __forceinline__ void store_chunk(const Params& p, float (&v)[2 * W], int n, int m, int live, int lane) {
    if (W == 16 && live == 2 * W) store_chunk<CDT, W, W == 16>(p, v, n, m, live, lane);
    else store_chunk<CDT, W, false>(p, v, n, m, live, lane);
}

__device__ __forceinline__ float element(const void* p, size_t i, int dt) {
    return dt == DT_F32 ? load_as_float<DT_F32>(p, i) : (dt == DT_F16 ? load_as_float<DT_F16>(p, i) : load_as_float<DT_BF16>(p, i));
}
// Scales, bias and the rest of the epilogue for channels n .. n + 3 of expert e in C's row m (SPLIT).
__device__ __forceinline__ void finish4(const Params& p, float (&y)[4], int e, size_t m, int n) {
    const size_t en = (size_t)e * p.N + n;
    const int live = min(4, p.N - n);
    const float as = p.a_scale ? load(p.a_scale + m) : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float ws = p.b_scale && i < live ? load(p.b_scale + en + i) : 1.f;
        const float bias = p.bias && i < live ? load(p.bias + en + i) : 0.f;
        y[i] = fmaf(y[i] * as, ws, bias);
    }
    const bool glu = p.act == ACT_SWIGLU;
    if (glu) {
        y[0] = act_fixed<ACT_SILU>(y[0]) * y[1];
        y[1] = act_fixed<ACT_SILU>(y[2]) * y[3];
    } else if (p.act != ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = act_apply(p.act, y[i]);
            y[i] = isnan(y[i]) ? y[i] : v;       // (kept behind ReLU, as everywhere)
        }
    }
    const int count = glu ? live >> 1 : live;
    const size_t at = m * p.cols + (glu ? n >> 1 : n);
    if (p.residual) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < count) y[i] += element(p.residual, at + i, p.c_dtype);
    }
    if (count == 4 && (p.cols & 3) == 0) {
        if (p.c_dtype == DT_F32) {
            *reinterpret_cast<float4*>(static_cast<float*>(p.C) + at) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (p.c_dtype == DT_F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(y[2 * i + 1]), "f"(y[2 * i]));
                else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(y[2 * i + 1]), "f"(y[2 * i]));
            }
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.C) + at) = make_uint2(w[0], w[1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < count) store_out_rt(p.C, at + i, y[i], p.c_dtype);
    }
}

template <int F, int BN, int MODE>
__global__ void __launch_bounds__(kThreads, 1) group_gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    using P = Plan<F, BN, MODE>;
    constexpr int S = P::kStages;
    constexpr bool kPair = MODE == PAIR, kCluster = MODE != SOLO, kDirect = MODE == SPLIT && BN == 32;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * P::kStage + P::kRed);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 10);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int32_t* start = reinterpret_cast<int32_t*>(smem + S * P::kStage + P::kRed + kTail);   // group starts, held to [0, M]
    int32_t* before = start + p.E + 1;                                                      // tiles before each group
    const uint32_t ring = ptx::smem_u32(smem), red = ring + S * P::kStage;
    auto bar = [&](int i) { return ptx::smem_u32(bars + i); };
    auto full = [&](int s) { return bar(s); };                        // the stage's copies landed, the scales are in place
    auto empty = [&](int s) { return bar(kMaxStages + s); };          // the stage's MMAs are done
    auto acc_full = [&](int b) { return bar(2 * kMaxStages + b); };   // the accumulator's MMAs are done
    auto acc_empty = [&](int b) { return bar(2 * kMaxStages + 2 + b); };   // the epilogue has read what the next MMAs overwrite
    const uint32_t drain = bar(2 * kMaxStages + 4), stall_bar = bar(2 * kMaxStages + 5);
    const uint32_t parts = bar(2 * kMaxStages + 6);       // SPLIT: the partial sums of this block's channels arrived
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp: known to be uniform
    auto wait = [&](uint32_t b, uint32_t parity) {
        return kPair ? cluster_bar_wait(b, parity, abort_flag, p.status, p.wait_ns)
                     : ptx::mbar_wait(b, parity, abort_flag, p.status, p.wait_ns);
    };
    const uint32_t rank = kCluster ? cluster_rank() : 0u;
    const int worker = kCluster ? (int)blockIdx.x / p.split : (int)blockIdx.x;
    const int workers = kCluster ? (int)gridDim.x / p.split : (int)gridDim.x;
    // this block's stages of every tile
    const int ks0 = MODE == SPLIT ? (int)((long long)p.stages * rank / p.split) : 0;
    const int nks = MODE == SPLIT ? (int)((long long)p.stages * (rank + 1) / p.split) - ks0 : p.stages;
    // PAIR: block 0's barriers gather both blocks' copies, scales and epilogues for the MMAs it issues
    auto lead = [&](uint32_t b) { return kPair ? peer(b, 0) : b; };

    const int dense_m = (p.M + BN - 1) / BN;
    // the MMA's columns for a tile of `rows` rows
    auto columns = [](int rows) { return kPair ? (rows + 31) / 32 * 32 : (rows + 15) / 16 * 16; };
    // Tile t: groups in order, in a group the row tiles of a channel tile side by side (they share its
    // weights).
    auto tile_of = [&](int t) {
        Tile x;
        int lo = 0, hi = p.M, mt = dense_m;
        x.e = 0;
        if (p.offsets) {
            int a = 0, b = p.E;            // before[a] <= t < before[b]
            while (b - a > 1) {
                const int c = (a + b) >> 1;
                if (before[c] <= t) a = c;
                else b = c;
            }
            x.e = a;
            t -= before[a];
            lo = start[a];
            hi = start[a + 1];
            mt = (hi - lo + BN - 1) / BN;
        }
        x.n0 = t / mt * P::kTileCh + (kPair ? (int)rank * kCh : 0);      // this block's channels
        x.m0 = lo + t % mt * BN;
        x.rows = min(BN, hi - x.m0);
        return x;
    };

    // Stage i of this block's part of tile x into slot s.
    auto issue = [&](const Tile& x, int i, int s) {
        // PAIR: each block brings the rows of its half of the MMA's columns
        const int mine = kPair ? columns(x.rows) / 2 : x.rows, first = x.m0 + (kPair ? (int)rank * mine : 0);
        const int boxes = (mine + P::kBoxRows - 1) / P::kBoxRows;
        const int k = ks0 + i, kx = k * (F == HALF ? 64 : kRowBytes);
        const uint32_t st = ring + (uint32_t)s * P::kStage, done = lead(full(s));
        if (rank == 0 || !kPair)
            ptx::mbar_expect_tx(full(s), (uint32_t)(P::kA + boxes * P::kBoxRows * kRowBytes + P::kSA) * (kPair ? 2u : 1u));
        load_3d<MODE>(st, &maps.b, kx, x.n0, x.e, done);
        for (int b = 0; b < boxes; ++b)
            load_2d<MODE>(st + P::kA + b * (P::kBoxRows * kRowBytes), &maps.a, kx, first + b * P::kBoxRows, done);
        // (a stage past the channels' last scale tile brings tiles that no MMA uses)
        if (F != HALF)
            load_2d<MODE>(st + P::kA + P::kB, &maps.sb, 0, (x.e * p.ch_tiles + x.n0 / kCh) * p.ktiles + k * P::kChunks, done);
    };

    bool sent = false;   // SPLIT: this thread has waited for the peers' barriers
    if (warp == 0 && elect_one()) {
        for (int s = 0; s < S; ++s) {
            // the TMA warp, and one scale warp (PAIR: one a half in both blocks)
            ptx::mbar_init(full(s), F == HALF ? 1 : (kPair ? 5 : 2));
            ptx::mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(acc_full(b), 1);
            ptx::mbar_init(acc_empty(b), kPair ? 2 * kEpiWarps : kEpiWarps);
        }
        ptx::mbar_init(drain, 1);
        ptx::mbar_init(stall_bar, 1);
        ptx::mbar_init(parts, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        ptx::prefetch_tmap(&maps.a);
        ptx::prefetch_tmap(&maps.b);
        if (F != HALF) ptx::prefetch_tmap(&maps.sb);
    }
    if (warp == 1) {
        // (one block fits an SM, so the columns are free; PAIR: both blocks take part)
        if constexpr (kPair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_u32(tmem_slot)), "r"(512) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_u32(tmem_slot)), "r"(512) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    grid_wait();      // the earlier kernels' results (offsets, operands) are there, and C may be written
    grid_release();
    if (p.offsets && warp == 2) {
        // Group starts and the tiles before each group. An entry is held to [0, M] and to the largest
        // before it, so that groups never overlap and have no more tiles than the launch allowed for.
        int carry = 0, reached = 0;
        for (int e0 = 0; e0 <= p.E; e0 += 32) {
            const int e = e0 + lane;
            int lo = max(min(max(e <= p.E ? load(p.offsets + e) : 0, 0), p.M), reached);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, lo, o);
                if (lane >= o) lo = max(lo, y);
            }
            // the group's end: the next lane's start, or for the last lane the next entry
            int hi = __shfl_down_sync(0xffffffffu, lo, 1);
            if (lane == 31 && e < p.E) hi = max(min(max(load(p.offsets + e + 1), 0), p.M), lo);
            const int tiles = e < p.E ? (hi - lo + BN - 1) / BN * p.n_tiles : 0;
            int sum = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            if (e <= p.E) {
                start[e] = lo;
                before[e] = carry + sum - tiles;
            }
            carry += __shfl_sync(0xffffffffu, sum, 31);
            reached = __shfl_sync(0xffffffffu, lo, 31);
        }
    }
    tc_fence_before();
    // the peers' barriers are initialized before anyone arrives on them (SPLIT: the wait comes later)
    if constexpr (kCluster) cluster_arrive();
    if constexpr (kPair) cluster_wait();
    // The block barrier. The TMA warp only reports that it has initialized the barriers, and goes on to
    // its first loads, where it needs neither the tile table nor another block.
    if (warp == 0 && !kPair && !p.offsets) asm volatile("bar.arrive 2, %0;" ::"n"(kThreads) : "memory");
    else asm volatile("bar.sync 2, %0;" ::"n"(kThreads) : "memory");
    tc_fence_after();
    const int total = p.offsets ? before[p.E] : dense_m * p.n_tiles;
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);       // (not for the TMA warp)
    if (warp == 0) {
        // ---------------- TMA
        if (elect_one()) {
            int g = 0, s = 0;
            uint32_t ph = 0;
            bool stop = false;
            for (int t = worker; t < total && !stop; t += workers) {
                const Tile x = tile_of(t);
                for (int i = 0; i < nks; ++i) {
                    if (*abort_flag || (g >= S && !wait(empty(s), ph ^ 1u))) {
                        stop = true;
                        break;
                    }
                    issue(x, i, s);
                    ++g;
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
            // PAIR: the last reports of finished stages have arrived here before the block leaves
            if (kPair && !stop)
                for (int i = max(0, g - S); i < g; ++i) wait(empty(i % S), (uint32_t)(i / S) & 1u);
            if (*abort_flag && (rank == 0 || !kPair))
                // the copies issued land before the block (PAIR: the cluster, whose copies report here) exits;
                // the scale warps, or the other block, may have left some of these phases open, so the
                // wait is short
                for (int i = max(0, g - S); i < (kPair ? max(0, g - S) + S : g); ++i) {
                    volatile int never = 0;
                    ptx::mbar_wait(full(i % S), (uint32_t)(i / S) & 1u, &never, p.status, kDrainNs);
                }
        }
    } else if (warp == kScaleWarp || warp == kScaleWarp + 1) {
        // ---------------- the activations' scales
        // A lane takes the 16-byte pieces (two stages' scales in MXFP4, one's in NVFP4) of the four rows
        // r, r + 32, r + 64, r + 96 of a half of the tile and writes each scale tile's four words of its
        // rows, which lie side by side there, as 16 bytes. (Bringing the words in one by one with 4-byte
        // asynchronous copies took as long as the stage's MMAs: each touches another line of the cache.)
        // The loads run as far ahead as the ring's, behind whose copies they queue, across tiles, in sets
        // of registers taken in turn (passing them on from set to set would wait for them). The warps
        // take a half each (PAIR), or every other piece.
        if constexpr (F != HALF) {
            constexpr bool kTurns = !kPair;
            constexpr int kStep = kTurns ? 2 : 1, kPer = F == MX ? 2 : 1;      // pieces, stages per piece
            const int w = warp - kScaleWarp, half = kTurns ? 0 : w;
            int first = ks0 / kPer;
            const int last = (ks0 + nks - 1) / kPer;
            if (kTurns && (first & 1) != w) ++first;
            // the next loads: piece qf of tile tf
            int tf = first <= last ? worker : total, qf = first, rows = 0;
            const uint8_t* src = nullptr;
            auto open_tile = [&]() {
                if (tf >= total) return;
                const Tile x = tile_of(tf);
                rows = x.rows - 128 * half - lane;           // row 32 j of this lane is the tile's while 32 j < rows
                src = p.As + (size_t)(x.m0 + 128 * half + lane) * p.pitch;
            };
            auto fetch = [&](uint4 (&v)[4]) {
                if (tf >= total) return;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = 32 * j < rows ? load(reinterpret_cast<const uint4*>(src + (size_t)(32 * j) * p.pitch) + qf) : make_uint4(0, 0, 0, 0);
                qf += kStep;
                if (qf > last) {
                    qf = first;
                    tf += workers;
                    open_tile();
                }
            };
            // the next pieces written: q of tile tu, whose first stage is the block's gb-th
            int tu = tf, q = first, gb = 0;
            auto write = [&](uint4 (&v)[4]) {
                if (tu >= total) return false;
                // a piece's stages together: one wait, one fence
                bool go = true;
                int slot[kPer];
#pragma unroll
                for (int d = 0; d < kPer; ++d) {
                    const int i = q * kPer + d - ks0, g = gb + i;
                    slot[d] = i < 0 || i >= nks ? -1 : g % S;
                    if (slot[d] >= 0 && g >= S) go = go && wait(empty(slot[d]), (uint32_t)(g / S - 1) & 1u);
                }
                if (!__all_sync(0xffffffffu, go)) return false;
#pragma unroll
                for (int d = 0; d < kPer; ++d) {
                    if (slot[d] < 0) continue;
                    const uint32_t dst = ring + (uint32_t)slot[d] * P::kStage + P::kA + P::kB + P::kSA + half * 512 + lane * 16;
#pragma unroll
                    for (int c = 0; c < P::kChunks; ++c) {
                        constexpr int kWords = P::kChunks;       // words of a row per stage
                        auto word = [&](const uint4& x) {
                            const int i4 = d * kWords + c;
                            return i4 == 0 ? x.x : (i4 == 1 ? x.y : (i4 == 2 ? x.z : x.w));
                        };
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + c * P::kHalves * 512), "r"(word(v[0])),
                                     "r"(word(v[1])), "r"(word(v[2])), "r"(word(v[3]))
                                     : "memory");
                    }
                }
                ptx::fence_proxy_async_smem();       // visible to the tensor core's copies
                __syncwarp();
                if (lane < kPer) {
                    const int s = kPer == 2 && lane == 1 ? slot[kPer - 1] : slot[0];
                    if (s >= 0) {
                        if constexpr (kPair) {
                            release_shared();
                            peer_arrive(lead(full(s)));
                        } else {
                            ptx::mbar_arrive(full(s));
                        }
                    }
                }
                fetch(v);
                q += kStep;
                if (q > last) {
                    q = first;
                    tu += workers;
                    gb += nks;
                }
                return true;
            };
            constexpr int kSets = F == MX ? 4 : 6;
            uint4 sets[kSets][4];
            open_tile();
#pragma unroll
            for (int i = 0; i < kSets; ++i) fetch(sets[i]);
            for (bool more = true; more;) {
#pragma unroll
                for (int i = 0; i < kSets; ++i) more = more && write(sets[i]);
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA. The whole warp runs through this, so that the operands stay in warp-wide
        // registers; each instruction elects its lane.
        if (rank == 0 || !kPair) {
            auto wait_all = [&](uint32_t b, uint32_t parity) {       // one answer for the warp
                return __all_sync(0xffffffffu, wait(b, parity));
            };
            int s = 0, tj = 0;
            uint32_t ph = 0;
            bool stop = false, issued = false;
            // A stage's MMAs run in groups that share a scale tile: two MMAs in MXFP4, one in NVFP4 (16-bit:
            // the whole stage). Copies and MMAs execute in the order of issue, and a copy issued just
            // before the MMA that needs it leaves the tensor cores idle meanwhile, so each group's copies
            // are issued ahead of the previous group's MMAs. Rows and halves past the tile's are copied
            // too, whatever they hold: their columns are not read.
            constexpr int kGroups = F == HALF ? 1 : P::kChunks;
            const uint32_t wdesc = rows_lo(ring), adesc = rows_lo(ring + P::kA), sdesc = scale_lo(ring + P::kA + P::kB);
            auto copy_group = [&](int slot, int c) {
                if constexpr (F != HALF) {
                    const uint32_t at = sdesc + (uint32_t)(slot * (P::kStage >> 4));
                    copy_scales<MODE>(tmem + P::kSaCol + 4 * c, at + c * 32);
#pragma unroll
                    for (int h = 0; h < P::kHalves; ++h)
                        copy_scales<MODE>(tmem + P::kSbCol + 4 * (c * P::kHalves + h), at + (P::kChunks + c * P::kHalves + h) * 32);
                }
            };
            if (p.stall) wait_all(stall_bar, 0u);      // diagnostic: runs out
            const int kbytes = F == HALF ? 2 * p.K : p.K / 2;
            for (int t = worker; t < total && !stop; t += workers, ++tj) {
                const int rows = __shfl_sync(0xffffffffu, tile_of(t).rows, 0);
                const uint32_t idesc = inst_desc<F>(P::kTileCh, columns(rows), p.bf16);
                const uint32_t acc = tmem + ((tj & 1) ? (uint32_t)P::kAcc1 : 0u);
                // overlapping accumulators: the last tile's shared columns have been read; else: the
                // accumulator's tile before the last has been read
                if (P::kOverlap ? (tj >= 1 && !wait_all(acc_empty(0), (uint32_t)(tj - 1) & 1u))
                                : (tj >= 2 && !wait_all(acc_empty(tj & 1), (uint32_t)((tj >> 1) - 1) & 1u)))
                    break;
                bool copied = false;       // the stage is in place and its first scales are on their way
                for (int i = 0; i < nks; ++i) {
                    if (!copied) {
                        if (!wait_all(full(s), ph)) {
                            stop = true;
                            break;
                        }
                        tc_fence_after();
                        issued = true;
                        copy_group(s, 0);
                    }
                    const uint32_t at = (uint32_t)(s * (P::kStage >> 4));     // the stage, in descriptor units
                    const int steps = min(4, (kbytes - (ks0 + i) * kRowBytes) / 32);     // 32 bytes of K per MMA
                    const int s1 = s + 1 == S ? 0 : s + 1;
                    const uint32_t ph1 = s + 1 == S ? ph ^ 1u : ph;
#pragma unroll
                    for (int gr = 0; gr < kGroups; ++gr) {
                        // the next group's scales before this group's MMAs
                        if (gr + 1 < kGroups) {
                            copy_group(s, gr + 1);
                        } else if (F != HALF) {
                            copied = i + 1 < nks && __all_sync(0xffffffffu, bar_test(full(s1), ph1));
                            if (copied) {
                                tc_fence_after();
                                copy_group(s1, 0);
                            }
                        }
#pragma unroll
                        for (int kk = gr * (4 / kGroups); kk < (gr + 1) * (4 / kGroups); ++kk) {
                            if (kk >= steps) break;
                            const uint32_t add = (i | kk) != 0;
                            const uint32_t sf = F == MX ? 2u * (kk & 1) : 0u;
                            mma<F, MODE>(acc, wdesc + at + 2 * kk, adesc + at + 2 * kk, idesc | sf << 29 | sf << 4,
                                         tmem + P::kSaCol + 4 * gr, tmem + P::kSbCol + 4 * gr * P::kHalves, add);
                        }
                    }
                    mma_commit<MODE>(empty(s));
                    s = s1;
                    ph = ph1;
                }
                if (!stop) mma_commit<MODE>(acc_full(tj & 1));
            }
            if (__any_sync(0xffffffffu, *abort_flag) && issued) {   // the MMAs issued finish before their tensor memory is released
                volatile int never = 0;
                mma_commit<MODE>(drain);
                ptx::mbar_wait(drain, 0u, &never, p.status);
            }
        }
    } else {
        // ---------------- epilogue
        const int q = warp & 3, h = (warp - kEpiWarp) >> 2;
        const float* const part = reinterpret_cast<const float*>(smem + S * P::kStage);
        int tj = 0;
        for (int t = worker; t < total; t += workers, ++tj) {
            const Tile x = tile_of(t);
            if (!__all_sync(0xffffffffu, wait(acc_full(tj & 1), (uint32_t)(tj >> 1) & 1u))) break;
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + ((tj & 1) ? (uint32_t)P::kAcc1 : 0u);
            constexpr int kParts = BN / 32;      // chunks of 16 columns of each column half
            if constexpr (MODE == SPLIT) {
                // the partial sums arrive as [block][row][channel of the share]
                const int share = kCh / p.split, ch = 32 * q + lane, held = x.rows * share * 4;
                if (threadIdx.x == kEpiWarp * 32) ptx::mbar_expect_tx(parts, (uint32_t)(p.split * held));
                if constexpr (kDirect) {
                    cluster_wait();
                    sent = true;
                    const uint32_t to = peer(red + rank * held + (uint32_t)(ch % share) * 4, ch / share), to_bar = peer(parts, ch / share);
                    const int c0 = 16 * h;
                    if (c0 < x.rows) {
                        float v[16];
                        tmem_ld(acc + (uint32_t)c0, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (c0 + i < x.rows) peer_store(to + (uint32_t)((c0 + i) * share) * 4, v[i], to_bar);
                    }
                    __syncwarp();
                } else {
                    // turned where the ring was (its MMAs are done)
                    float* const own = reinterpret_cast<float*>(smem) + (size_t)(ch / share) * x.rows * share + ch % share;
                    for (int j = 0; j < kParts; ++j) {
                        const int c0 = 16 * (kParts * h + j);
                        if (c0 >= x.rows) break;
                        float v[16];
                        tmem_ld(acc + (uint32_t)c0, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (c0 + i < x.rows) own[(c0 + i) * share] = v[i];
                        __syncwarp();
                    }
                    ptx::fence_proxy_async_smem();
                    asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory");
                    cluster_wait();
                    sent = true;
                    if (threadIdx.x == kEpiWarp * 32)
                        for (int r = 0; r < p.split; ++r)
                            peer_copy(peer(red + rank * held, r), ring + r * held, (uint32_t)held, peer(parts, r));
                }
                if (!__all_sync(0xffffffffu, cluster_bar_wait(parts, 0u, abort_flag, p.status, p.wait_ns))) break;
                // this block's share of the channels (a power of two from 16 up), all rows, four channels a thread
                const int lg = 31 - __clz(share >> 2), step = x.rows * share;
#pragma unroll 1
                for (int i = threadIdx.x - kEpiWarp * 32; i < step / 4; i += kEpiThreads) {
                    const int row = i >> lg, n = x.n0 + (int)rank * share + 4 * (i - (row << lg));
                    if (n >= p.N) continue;
                    float4 v[kMaxSplit];
#pragma unroll
                    for (int r = 0; r < kMaxSplit; ++r)
                        if (r < p.split) v[r] = *reinterpret_cast<const float4*>(part + r * step + 4 * i);
                    float y[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
                    for (int r = 1; r < kMaxSplit; ++r)
                        if (r < p.split) {
                            y[0] += v[r].x;
                            y[1] += v[r].y;
                            y[2] += v[r].z;
                            y[3] += v[r].w;
                        }
                    finish4(p, y, x.e, (size_t)(x.m0 + row), n);
                }
            } else {
                const int n = x.n0 + 32 * q + lane;
                const size_t en = (size_t)x.e * p.N + min(n, p.N - 1);
                const float ws = p.b_scale ? load(p.b_scale + en) : 1.f;
                const float bias = p.bias ? load(p.bias + en) : 0.f;
                constexpr int kWide = P::kWide, kMine = BN / (2 * kWide);     // chunks of a column half
#pragma unroll 1
                for (int j = 0; j < kMine; ++j) {
                    // chunks alternate between the halves; overlapping accumulators share the first one's
                    // last columns and the second one's first: those go first
                    const int i2 = 2 * j + h, c0 = kWide * (P::kOverlap && !(tj & 1) ? 2 * kMine - 1 - i2 : i2);
                    const int live = min(kWide, x.rows - c0);       // rows of this chunk (none: <= 0)
                    float v[kWide];
                    __syncwarp();
                    if (live > 0) tmem_ld(acc + (uint32_t)c0, v);
                    if (j == (P::kOverlap ? (P::kShared + 1) / 2 - 1 : kMine - 1)) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            const uint32_t b = acc_empty(P::kOverlap ? 0 : tj & 1);
                            if constexpr (kPair) peer_arrive(lead(b));
                            else ptx::mbar_arrive(b);
                        }
                    }
                    if (live <= 0) continue;
                    const int m = x.m0 + c0;
                    if (p.a_scale) {
                        const float as = load(p.a_scale + m + min(lane & (kWide - 1), live - 1));
#pragma unroll
                        for (int i = 0; i < kWide; ++i) v[i] *= __shfl_sync(0xffffffffu, as, i);
                    }
                    if (p.b_scale || p.bias) {
#pragma unroll
                        for (int i = 0; i < kWide; ++i) v[i] = fmaf(v[i], ws, bias);
                    }
                    if (p.c_dtype == DT_BF16) store_chunk<DT_BF16, kWide / 2>(p, v, n, m, live, lane);
                    else if (p.c_dtype == DT_F16) store_chunk<DT_F16, kWide / 2>(p, v, n, m, live, lane);
                    else store_chunk<DT_F32, kWide / 2>(p, v, n, m, live, lane);
                }
                __syncwarp();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // No block leaves while a peer may still reach its memory, or a copy may still read it. (With its sums,
    // each stored by its sender, a block has heard the last of its peers; one that gave up waits until
    // they have left or given up too.)
    if (kCluster && (!kDirect || *abort_flag)) {
        if (MODE == SPLIT && !sent) cluster_wait();        // the first phase, where it was not waited for
        cluster_arrive();
        cluster_wait();
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if constexpr (kPair) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ---------------------------------------------------------------- host side
// Operand rows of row_bytes as a 2-D (activations) or 3-D (weights of E experts) tensor; boxes of 128
// bytes x box_rows rows with the 128-byte swizzle; bytes, rows and experts past the end read 0.
inline cudaError_t make_map(CUtensorMap* map, const void* base, int form, int bf16, int K, int rows, int E, int box_rows) {
    EncodeTiledFn enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t row_bytes = form == HALF ? (cuuint64_t)K * 2 : (cuuint64_t)K / 2;
    const cuuint64_t dims[3] = {form == HALF ? (cuuint64_t)K : row_bytes, (cuuint64_t)rows, (cuuint64_t)E};
    const cuuint64_t strides[2] = {row_bytes, row_bytes * rows};
    const cuuint32_t box[3] = {(cuuint32_t)(form == HALF ? 64 : kRowBytes), (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUtensorMapDataType dt = form != HALF ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : (bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16);
    return enc(map, dt, E > 0 ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// The weights' scale tiles as a 2-D tensor of 512-byte rows; boxes of a stage's tiles.
inline cudaError_t make_scale_map(CUtensorMap* map, const void* base, size_t tiles, int chunks) {
    EncodeTiledFn enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {128, (cuuint64_t)tiles};
    const cuuint64_t strides[1] = {512};
    const cuuint32_t box[2] = {128, (cuuint32_t)chunks};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// The launch for a tile height and cluster size; tiles: at least as many as the call has.
template <int F, int BN, int MODE>
cudaError_t launch(const GroupGemmArgs& a, int fmt, int split, long long tiles, cudaStream_t s) {
    using P = Plan<F, BN, MODE>;
    const int bf16 = fmt == GF_BF16, block = F == MX ? 32 : 16;
    Maps maps;
    cudaError_t e = make_map(&maps.a, a.A, F, bf16, a.K, a.M, 0, P::kBoxRows);
    if (e == cudaSuccess) e = make_map(&maps.b, a.B, F, bf16, a.K, a.N, a.E, kCh);
    const int ch_tiles = (a.N + kCh - 1) / kCh, ktiles = F == HALF ? 0 : fp4::scale_ktiles(a.K, block);
    if (F == HALF) maps.sb = maps.b;   // unused
    else if (e == cudaSuccess) e = make_scale_map(&maps.sb, a.Bs, (size_t)a.E * ch_tiles * ktiles, P::kChunks);
    if (e != cudaSuccess) return e;
    Params p{};
    p.M = a.M; p.E = a.E; p.K = a.K; p.N = a.N;
    p.cols = a.act == ACT_SWIGLU ? a.N / 2 : a.N;
    p.n_tiles = (a.N + P::kTileCh - 1) / P::kTileCh;
    p.ch_tiles = ch_tiles;
    p.stages = F == HALF ? a.K / 64 : (a.K + 255) / 256;
    p.bf16 = bf16;
    p.split = split;
    p.offsets = a.offsets;
    p.As = static_cast<const uint8_t*>(a.As);
    p.pitch = F == HALF ? 0 : fp4::scale_pitch(a.K, block);
    p.ktiles = ktiles;
    p.a_scale = a.a_scale; p.b_scale = a.b_scale; p.bias = a.bias;
    p.residual = a.residual;
    p.C = a.C;
    p.act = a.act; p.c_dtype = a.c_dtype;
    p.status = status_word_address();
    if (!p.status) return cudaErrorUnknown;
    p.wait_ns = option_wait_ns();
    p.stall = option_stall();
    auto kern = group_gemm_kernel<F, BN, MODE>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)P::kSmem);
    if (e != cudaSuccess) return e;
    const long long most = kTargetSms / split;
    return launch_behind(kern, dim3((unsigned)((tiles < most ? tiles : most) * split)), dim3(kThreads), P::kSmem, (unsigned)split, s, maps, p);
}

template <int F>
cudaError_t launch_form(const GroupGemmArgs& a, int fmt, cudaStream_t s) {
    const Choice c = choose(a, fmt);       // (the call's checks have refused more tiles than can be counted)
    if (c.bn == 32) return c.split > 1 ? launch<F, 32, SPLIT>(a, fmt, c.split, c.tiles, s) : launch<F, 32, SOLO>(a, fmt, 1, c.tiles, s);
    if (c.bn == 128) return c.split > 1 ? launch<F, 128, SPLIT>(a, fmt, c.split, c.tiles, s) : launch<F, 128, SOLO>(a, fmt, 1, c.tiles, s);
    return launch<F, 256, PAIR>(a, fmt, 2, c.tiles, s);
}

}  // namespace gg
}  // namespace qg
