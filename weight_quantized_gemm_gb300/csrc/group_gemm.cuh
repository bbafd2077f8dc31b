// Products of microscaled 4-bit or 16-bit operands on the tensor cores, dense or one per expert over
// ragged row groups:
//   C[m][n] = act(a_scale[m] * b_scale[e][n] * sum_k A[m][k] B[e][n][k] + bias[e][n]) + residual[m][n].
//
// As in prefill_kernel.cuh the product is computed transposed, D[n][m] = sum_k B[n][k] A[m][k]: the
// weight's 128 channels are the MMA's 128 rows, and the activation rows its N, which the instruction
// takes in steps of 16. So a group of a few rows costs a few columns, not a padded tile, and one
// kernel serves single tokens and long prompts. The 4-bit formats are multiplied as they are
// (kind::mxf4 / mxf4nvf4: 64 of K per instruction, four times the 16-bit rate, the block scales
// applied inside), so nothing is dequantized anywhere.
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
//               48 columns, which the epilogue reads first.
// Groups are found in the kernel from the offsets (the host never reads them): each block sums the
// groups' tile counts once, and finds a tile's group by binary search.
//
// SPLIT: with too few tiles to fill the GPU, the blocks of a cluster share a tile, each taking a part
// of K; partial sums meet in distributed shared memory, where every block adds its part of the
// channels over the blocks in rank order. No workspace, no atomics, one launch.
//
// Every wait is bounded (see ptx.cuh); after an abort the copies and MMAs in flight are waited for,
// and a cluster's blocks leave together.
#pragma once

#include <type_traits>

#include "epilogue.cuh"
#include "fp4.cuh"
#include "ptx.cuh"

namespace qg {
namespace gg {

constexpr int kThreads = 384;
constexpr int kEpiWarp = 4, kEpiWarps = 8, kEpiThreads = kEpiWarps * 32;
constexpr int kScaleWarp = 2;
constexpr int kRowBytes = 128;                     // K bytes of a row per stage
constexpr int kCh = 128;                           // channels per tile
constexpr int kMaxSplit = 8;
constexpr int kMaxStages = 10;
constexpr size_t kSmemMax = 232448;
constexpr int kTail = 1024;                        // barriers

// Operand forms: 16-bit, or 4-bit with 2 (MXFP4) or 4 (NVFP4) scale tiles per stage.
enum Form { HALF = 0, MX = 1, NV = 2 };
template <int F, int BN, bool SPLIT>
struct Plan {
    static constexpr int kChunks = F == HALF ? 0 : (F == MX ? 2 : 4);      // scale tiles (128 rows x 4) per stage
    static constexpr int kHalves = (BN + 127) / 128;                       // ... of the activations, per 128 rows
    static constexpr int kA = kCh * kRowBytes, kB = BN * kRowBytes;
    static constexpr int kSA = kChunks * 512, kSB = kChunks * kHalves * 512;
    static constexpr int kStage = kA + kB + kSA + kSB;
    static constexpr int kRed = SPLIT ? BN * kCh * 4 : 0;                  // this block's partial sums
    static constexpr int kTables = 2 * (1024 + 1) * 4;                     // group starts and tile counts
    static constexpr int kRoom = (int)kSmemMax - kTail - kTables - kRed;
    static constexpr int kStages = kRoom / kStage < kMaxStages ? kRoom / kStage : kMaxStages;
    static constexpr size_t kSmem = (size_t)kStages * kStage + kRed + kTail + kTables;
    static constexpr int kBoxRows = BN == 32 ? 16 : BN / 2;                // rows of one activation box
    static constexpr bool kOverlap = F != HALF && BN == 256;
    static constexpr int kAcc1 = kOverlap ? 208 : BN;                      // second accumulator's column
    static constexpr int kSaCol = kOverlap ? 464 : 2 * BN;                 // scale columns
    static constexpr int kSbCol = kSaCol + 16;
    static_assert(kStage % 1024 == 0, "stages keep the 128-byte swizzle's alignment");
    static_assert(kStages >= 4, "ring");
    static_assert(F == HALF ? 2 * BN <= 512 : kSbCol + kChunks * kHalves * 4 <= 512, "tensor memory");
};

struct Params {
    int M, E, K, N, cols;      // cols: C's columns (N, or N / 2 for SwiGLU)
    int n_tiles, stages;       // channel tiles; stages of K
    int bf16;                  // HALF: bf16 (else f16)
    int split;                 // blocks of a cluster that share a tile
    const int32_t* offsets;
    const uint8_t* As;
    int pitch;                 // bytes of a row of As
    const uint8_t* Bs;
    int ktiles;                // scale tiles along K of one channel tile of Bs
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
};

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptors: K-major rows of 128 bytes with the 128-byte swizzle (8-row atoms
// 1024 bytes apart), and a 32 x 16-byte scale tile without swizzle (8-row groups 128 bytes apart).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
// Scale tile (512 bytes) to four tensor-memory columns, in all four lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t tcol, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tcol), "l"(desc) : "memory");
}
// Instruction descriptors for n columns (a multiple of 16) and 128 rows. 16-bit: float32 D, A and B
// both f16 (0) or bf16 (1). 4-bit: A and B e2m1, scales e4m3 (0) or e8m0 (1 at bit 23), and which of a
// column's four scale bytes come first (sf: A's at bit 29, B's at bit 4).
template <int F>
__device__ __forceinline__ uint32_t inst_desc(int n, int bf16) {
    if constexpr (F == HALF)
        return (1u << 4) | ((uint32_t)bf16 << 7) | ((uint32_t)bf16 << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kCh >> 4) << 24);
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((F == MX ? 1u : 0u) << 23) | ((uint32_t)(kCh >> 7) << 27);
}
__device__ __forceinline__ void mma_half(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a),
        "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
template <int F>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t acc) {
    if constexpr (F == MX)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d), "l"(a), "l"(b),
            "r"(idesc), "r"(acc), "r"(sa), "r"(sb)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d), "l"(a),
            "l"(b), "r"(idesc), "r"(acc), "r"(sa), "r"(sb)
            : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
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
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Address of this block's shared-memory location in the cluster's block `rank`.
__device__ __forceinline__ uint32_t peer(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float peer_load(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
// mbar_wait (ptx.cuh) for a barrier that other blocks of the cluster arrive on.
__device__ __forceinline__ bool cluster_bar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned int* status,
                                                 long long limit_ns) {
    if (!ptx::mbar_wait(bar, parity, abort_flag, status, limit_ns)) return false;
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
    return true;
}
// True in one lane of the (converged) warp. The instructions that a single thread issues (TMA,
// tcgen05.mma, tcgen05.cp) take their operands from warp-wide registers; under this predicate the
// compiler knows that one lane is active and moves them there directly, under `lane == 0` it loops.
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

struct Tile {
    int e, n0, m0, rows;       // expert, first channel, first row, rows (0: none)
};

// Two neighbouring channels' values of the chunk's 16 rows, exchanged between the lanes of a pair: the
// even lane ends with both channels of rows 0-7 (first[i], second[i]), the odd lane with rows 8-15.
__device__ __forceinline__ void pair_up(const float (&v)[16], float (&first)[8], float (&second)[8], bool odd) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 8], 1);
        first[i] = odd ? got : v[i];
        second[i] = odd ? v[i + 8] : got;
    }
}

template <int ACT>
__device__ __forceinline__ void act16(float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = act_fixed<ACT>(v[i]);
}

// The rest of the epilogue for 16 rows m .. m + 15 (the first `live` of them) of channel n: activation,
// residual, rounding, stores. One choice of activation and type per chunk, none per value. 16-bit
// outputs leave as pairs of channels (64 contiguous bytes a row), of rows 0-7 from the even lanes
// and 8-15 from the odd ones; SwiGLU pairs become one channel the same way.
template <int CDT>
__device__ __forceinline__ void store_chunk(const Params& p, float (&v)[16], int n, int m, int live, bool odd) {
    constexpr size_t kEsz = CDT == DT_F32 ? 4 : 2;
    switch (p.act) {
        case ACT_RELU: act16<ACT_RELU>(v); break;
        case ACT_SILU: act16<ACT_SILU>(v); break;
        case ACT_GELU_TANH: act16<ACT_GELU_TANH>(v); break;
        default: break;
    }
    const bool glu = p.act == ACT_SWIGLU;
    const size_t step = (size_t)p.cols * kEsz;
    // `count` values of one channel in consecutive rows
    auto column = [&](float* y, int row, int col, int rows, auto count) {
        constexpr int kCount = decltype(count)::value;
        const size_t at = (size_t)row * p.cols + col;
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < kCount; ++i)
                if (i < rows) y[i] += load_c<CDT>(p.residual, at + (size_t)i * p.cols);
        }
        uint8_t* out = static_cast<uint8_t*>(p.C) + at * kEsz;
#pragma unroll
        for (int i = 0; i < kCount; ++i)
            if (i < rows) store_out_rt(out + i * step, 0, y[i], CDT);
    };
    if (glu || (CDT != DT_F32 && (p.N & 1) == 0)) {
        float a[8], b[8];
        pair_up(v, a, b, odd);
        const int row = m + (odd ? 8 : 0), rows = live - (odd ? 8 : 0);
        if (n >= p.N) return;              // (N is even here: both lanes of a pair)
        if (glu) {
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = act_fixed<ACT_SILU>(a[i]) * b[i];
            column(a, row, n >> 1, rows, std::integral_constant<int, 8>());
        } else if constexpr (CDT != DT_F32) {
            const size_t at = ((size_t)row * p.cols + (n & ~1)) * kEsz;
            if (p.residual) {
                uint32_t r[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    r[i] = i < rows ? __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.residual) + at + i * step)) : 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if constexpr (CDT == DT_F16) {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
                        a[i] += f.x;
                        b[i] += f.y;
                    } else {
                        a[i] += __uint_as_float(r[i] << 16);
                        b[i] += __uint_as_float(r[i] & 0xFFFF0000u);
                    }
                }
            }
            uint8_t* out = static_cast<uint8_t*>(p.C) + at;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t w;
                if constexpr (CDT == DT_F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b[i]), "f"(a[i]));
                else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b[i]), "f"(a[i]));
                if (i < rows) *reinterpret_cast<uint32_t*>(out + i * step) = w;
            }
        }
    } else if (n < p.N) {
        column(v, m, n, live, std::integral_constant<int, 16>());
    }
}

template <int F, int BN, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) group_gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    using P = Plan<F, BN, SPLIT>;
    constexpr int S = P::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * P::kStage + P::kRed);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * kMaxStages + 10);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int32_t* start = reinterpret_cast<int32_t*>(smem + S * P::kStage + P::kRed + kTail);   // group starts, held to [0, M]
    int32_t* before = start + p.E + 1;                                                      // tiles before each group
    const uint32_t ring = ptx::smem_u32(smem), red = ring + S * P::kStage;
    auto bar = [&](int i) { return ptx::smem_u32(bars + i); };
    auto full = [&](int s) { return bar(s); };                        // the stage's TMA copies landed
    auto full_sc = [&](int s) { return bar(kMaxStages + s); };        // the activations' scales are in place
    auto empty = [&](int s) { return bar(2 * kMaxStages + s); };      // the stage's MMAs are done
    auto acc_full = [&](int b) { return bar(3 * kMaxStages + b); };   // the accumulator's MMAs are done
    auto acc_empty = [&](int b) { return bar(3 * kMaxStages + 2 + b); };   // the epilogue has read what the next MMAs overwrite
    const uint32_t drain = bar(3 * kMaxStages + 4), stall_bar = bar(3 * kMaxStages + 5);
    const uint32_t parts_ready = bar(3 * kMaxStages + 6), parts_taken = bar(3 * kMaxStages + 7);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto wait = [&](uint32_t b, uint32_t parity) { return ptx::mbar_wait(b, parity, abort_flag, p.status, p.wait_ns); };
    const uint32_t rank = SPLIT ? cluster_rank() : 0u;
    const int worker = SPLIT ? (int)blockIdx.x / p.split : (int)blockIdx.x;
    const int workers = SPLIT ? (int)gridDim.x / p.split : (int)gridDim.x;
    // this block's stages of every tile
    const int ks0 = SPLIT ? (int)((long long)p.stages * rank / p.split) : 0;
    const int nks = SPLIT ? (int)((long long)p.stages * (rank + 1) / p.split) - ks0 : p.stages;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(full_sc(s), BN == 256 ? 2 : 1);   // one warp, or one a half
            ptx::mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(acc_full(b), 1);
            ptx::mbar_init(acc_empty(b), kEpiWarps);
        }
        ptx::mbar_init(drain, 1);
        ptx::mbar_init(stall_bar, 1);
        ptx::mbar_init(parts_ready, SPLIT ? kEpiWarps * p.split : 1);
        ptx::mbar_init(parts_taken, SPLIT ? kEpiWarps * p.split : 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        ptx::prefetch_tmap(&maps.a);
        ptx::prefetch_tmap(&maps.b);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_u32(tmem_slot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (p.offsets && warp == 2) {
        // group starts and the tiles before each group
        int carry = 0;
        for (int e0 = 0; e0 <= p.E; e0 += 32) {
            const int e = e0 + lane;
            const int lo = e <= p.E ? min(max(__ldg(p.offsets + e), 0), p.M) : 0;
            const int hi = e < p.E ? max(min(max(__ldg(p.offsets + e + 1), 0), p.M), lo) : lo;
            const int tiles = (hi - lo + BN - 1) / BN * p.n_tiles;
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
        }
    }
    tc_fence_before();
    if constexpr (SPLIT) cluster_sync();   // the peers' barriers are initialized before anyone arrives on them
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int dense_m = (p.M + BN - 1) / BN;
    const int total = p.offsets ? before[p.E] : dense_m * p.n_tiles;
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
            hi = max(start[a + 1], lo);
            mt = (hi - lo + BN - 1) / BN;
        }
        x.n0 = t / mt * kCh;
        x.m0 = lo + t % mt * BN;
        x.rows = min(BN, hi - x.m0);
        return x;
    };

    if (warp == 0) {
        // ---------------- TMA
        if (elect_one()) {
            int g = 0, s = 0;
            uint32_t ph = 0;
            bool stop = false;
            for (int t = worker; t < total && !stop; t += workers) {
                const Tile x = tile_of(t);
                const int boxes = (x.rows + P::kBoxRows - 1) / P::kBoxRows;
                const uint8_t* bs = F == HALF ? nullptr : p.Bs + ((size_t)x.e * p.n_tiles + x.n0 / kCh) * p.ktiles * 512;
                for (int i = 0; i < nks; ++i) {
                    if (*abort_flag || (g >= S && !wait(empty(s), ph ^ 1u))) {
                        stop = true;
                        break;
                    }
                    const int k = ks0 + i;
                    const uint32_t st = ring + (uint32_t)s * P::kStage;
                    const int chunks = min(P::kChunks, p.ktiles - k * P::kChunks);     // (16-bit: none)
                    const uint32_t sbytes = F == HALF ? 0u : (uint32_t)chunks * 512u;
                    ptx::mbar_expect_tx(full(s), (uint32_t)P::kA + (uint32_t)(boxes * P::kBoxRows * kRowBytes) + sbytes);
                    const int kx = k * (F == HALF ? 64 : kRowBytes);
                    ptx::tma_load_3d(st, &maps.b, kx, x.n0, x.e, full(s));
                    for (int b = 0; b < boxes; ++b)
                        ptx::tma_load_2d(st + P::kA + b * (P::kBoxRows * kRowBytes), &maps.a, kx, x.m0 + b * P::kBoxRows, full(s));
                    if (F != HALF) ptx::bulk_load(st + P::kA + P::kB, bs + (size_t)k * P::kSA, sbytes, full(s));
                    ++g;
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
            if (*abort_flag)   // the copies issued land before the block exits
                for (int i = max(0, g - S); i < g; ++i) {
                    volatile int never = 0;
                    ptx::mbar_wait(full(i % S), (uint32_t)(i / S) & 1u, &never, p.status);
                }
        }
    } else if (warp == kScaleWarp || warp == kScaleWarp + 1) {
        // ---------------- the activations' scales
        // A lane takes the 16-byte pieces (two stages' scales in MXFP4, one's in NVFP4) of the four rows
        // r, r + 32, r + 64, r + 96 of a half of the tile, the next pieces while it writes these, and writes
        // each scale tile's four words of its rows, which lie side by side there, as 16 bytes. (Bringing
        // the words in one by one with 4-byte asynchronous copies took as long as the stage's MMAs:
        // each touches another line of the cache.) The warps take a half each, or turns.
        if constexpr (F != HALF) {
            constexpr bool kTurns = BN < 256;
            constexpr int kStep = kTurns ? 2 : 1;
            const int w = warp - kScaleWarp, half = kTurns ? 0 : w;
            int s = 0, g = 0;
            uint32_t ph = 0;
            bool stop = false;
            for (int t = worker; t < total && !stop; t += workers) {
                const Tile x = tile_of(t);
                uint4 now[4], next[4];
                const uint8_t* src = p.As + (size_t)(x.m0 + 128 * half + lane) * p.pitch;
                auto fetch = [&](int piece, uint4 (&v)[4]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = 128 * half + 32 * j + lane < x.rows
                                   ? __ldg(reinterpret_cast<const uint4*>(src + (size_t)(32 * j) * p.pitch) + piece)
                                   : make_uint4(0, 0, 0, 0);
                };
                const int last = (ks0 + nks - 1) / (F == MX ? 2 : 1);
                int have = -1;
                for (int i = 0; i < nks; ++i) {
                    const int k = ks0 + i, piece = F == MX ? k >> 1 : k;
                    if (!kTurns || (piece & 1) == w) {
                        if (piece != have) {
                            if (have < 0) fetch(piece, now);
                            else
#pragma unroll
                                for (int j = 0; j < 4; ++j) now[j] = next[j];
                            have = piece;
                            if (piece + kStep <= last) fetch(piece + kStep, next);
                        }
                        const bool go = !*abort_flag && (g < S || wait(empty(s), ph ^ 1u));
                        if (!__all_sync(0xffffffffu, go)) {
                            stop = true;
                            break;
                        }
                        const uint32_t dst = ring + (uint32_t)s * P::kStage + P::kA + P::kB + P::kSA + lane * 16;
                        const bool second = F == MX && (k & 1);
#pragma unroll
                        for (int c = 0; c < P::kChunks; ++c) {
                            auto word = [&](const uint4& v) {
                                if (F == MX) return c == 0 ? (second ? v.z : v.x) : (second ? v.w : v.y);
                                return c == 0 ? v.x : (c == 1 ? v.y : (c == 2 ? v.z : v.w));
                            };
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (c * P::kHalves + half) * 512),
                                         "r"(word(now[0])), "r"(word(now[1])), "r"(word(now[2])), "r"(word(now[3]))
                                         : "memory");
                        }
                        ptx::fence_proxy_async_smem();       // visible to the tensor core's copies
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(full_sc(s));
                    }
                    ++g;
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA
        if (elect_one()) {
            int s = 0, tj = 0;
            uint32_t ph = 0;
            bool stop = false, issued = false;
            if (p.stall) wait(stall_bar, 0u);      // diagnostic: runs out
            const int kbytes = F == HALF ? 2 * p.K : p.K / 2;
            const uint64_t wdesc = sw128_desc(ring), adesc = sw128_desc(ring + P::kA), sdesc = scale_desc(ring + P::kA + P::kB);
            for (int t = worker; t < total && !stop; t += workers, ++tj) {
                const Tile x = tile_of(t);
                const uint32_t idesc = inst_desc<F>((x.rows + 15) / 16 * 16, p.bf16);
                const uint32_t acc = tmem + ((tj & 1) ? (uint32_t)P::kAcc1 : 0u);
                // overlapping accumulators: the last tile's shared columns have been read; else: the
                // accumulator's tile before the last has been read
                if (P::kOverlap ? (tj >= 1 && !wait(acc_empty(0), (uint32_t)(tj - 1) & 1u))
                                : (tj >= 2 && !wait(acc_empty(tj & 1), (uint32_t)((tj >> 1) - 1) & 1u)))
                    break;
                for (int i = 0; i < nks; ++i) {
                    if (!wait(full(s), ph) || (F != HALF && !wait(full_sc(s), ph))) {
                        stop = true;
                        break;
                    }
                    tc_fence_after();
                    issued = true;
                    const uint64_t at = (uint64_t)(s * (P::kStage >> 4));     // the stage, in descriptor units
                    const int steps = min(4, (kbytes - (ks0 + i) * kRowBytes) / 32);     // 32 bytes of K per MMA
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (kk >= steps) break;
                        const uint32_t add = (i | kk) != 0;
                        if constexpr (F == HALF) {
                            mma_half(acc, wdesc + at + 2 * kk, adesc + at + 2 * kk, idesc, add);
                        } else {
                            // a scale tile serves two MMAs (MXFP4) or one; rows and halves past the tile's
                            // are copied too, whatever they hold: their columns are not read
                            const int c = F == MX ? kk >> 1 : kk;
                            if (F == NV || (kk & 1) == 0) {
                                copy_scales(tmem + P::kSaCol + 4 * c, sdesc + at + c * 32);
#pragma unroll
                                for (int h = 0; h < P::kHalves; ++h)
                                    copy_scales(tmem + P::kSbCol + 4 * (c * P::kHalves + h),
                                                sdesc + at + (P::kChunks + c * P::kHalves + h) * 32);
                            }
                            const uint32_t sf = F == MX ? 2u * (kk & 1) : 0u;
                            mma_fp4<F>(acc, wdesc + at + 2 * kk, adesc + at + 2 * kk, idesc | sf << 29 | sf << 4,
                                       tmem + P::kSaCol + 4 * c, tmem + P::kSbCol + 4 * c * P::kHalves, add);
                        }
                    }
                    mma_commit(empty(s));
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
                if (!stop) mma_commit(acc_full(tj & 1));
            }
            if (*abort_flag && issued) {   // the MMAs issued finish before their tensor memory is released
                volatile int never = 0;
                mma_commit(drain);
                ptx::mbar_wait(drain, 0u, &never, p.status);
            }
        }
    } else {
        // ---------------- epilogue
        const int q = warp & 3, h = (warp - kEpiWarp) >> 2;
        const bool odd = lane & 1, glu = p.act == ACT_SWIGLU;
        float* const part = reinterpret_cast<float*>(smem + S * P::kStage);
        auto cluster_wait = [&](uint32_t b, uint32_t parity) {
            return cluster_bar_wait(b, parity, abort_flag, p.status, p.wait_ns);
        };
        auto store_one = [&](size_t at, float y) {
            if (p.residual)
                y += p.c_dtype == DT_F32 ? load_c<DT_F32>(p.residual, at)
                                         : (p.c_dtype == DT_F16 ? load_c<DT_F16>(p.residual, at) : load_c<DT_BF16>(p.residual, at));
            store_out_rt(p.C, at, y, p.c_dtype);
        };
        int tj = 0;
        for (int t = worker; t < total; t += workers, ++tj) {
            const Tile x = tile_of(t);
            if (!__all_sync(0xffffffffu, wait(acc_full(tj & 1), (uint32_t)(tj >> 1) & 1u))) break;
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + ((tj & 1) ? (uint32_t)P::kAcc1 : 0u);
            constexpr int kParts = BN / 32;      // chunks of 16 columns of each column half
            if constexpr (SPLIT) {
                // this block's partial sums [row][channel], once the peers have read the last tile's
                if (tj > 0 && !__all_sync(0xffffffffu, cluster_wait(parts_taken, (uint32_t)(tj - 1) & 1u))) break;
                for (int j = 0; j < kParts; ++j) {
                    const int c0 = 16 * (kParts * h + j);
                    if (c0 >= x.rows) break;
                    float v[16];
                    tmem_ld16(acc + (uint32_t)c0, v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) part[(c0 + i) * kCh + 32 * q + lane] = v[i];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(acc_empty(tj & 1));
                    for (int r = 0; r < p.split; ++r) peer_arrive(peer(parts_ready, r));
                }
                if (!__all_sync(0xffffffffu, cluster_wait(parts_ready, (uint32_t)tj & 1u))) break;
                // this block's share of the channels (a multiple of 16), all rows
                const int share = kCh / p.split, count = x.rows * share;
                for (int i0 = threadIdx.x - kEpiWarp * 32; i0 < (count + 31) / 32 * 32; i0 += kEpiThreads) {
                    const int i = min(i0, count - 1), c = (int)rank * share + i % share, m = x.m0 + i / share, n = x.n0 + c;
                    float v[kMaxSplit];
#pragma unroll
                    for (int r = 0; r < kMaxSplit; ++r)
                        v[r] = r < p.split ? peer_load(peer(red + (uint32_t)((i / share) * kCh + c) * 4, r)) : 0.f;
#pragma unroll
                    for (int r = 1; r < kMaxSplit; ++r) v[0] += v[r];
                    const size_t en = (size_t)x.e * p.N + min(n, p.N - 1);
                    float y = v[0];
                    if (p.a_scale) y *= __ldg(p.a_scale + m);
                    if (p.b_scale) y *= __ldg(p.b_scale + en);
                    if (p.bias) y += __ldg(p.bias + en);
                    if (glu) {
                        const float up = __shfl_xor_sync(0xffffffffu, y, 1);
                        y = act_fixed<ACT_SILU>(y) * up;
                        if (i0 < count && n < p.N && !odd) store_one((size_t)m * p.cols + (n >> 1), y);
                    } else {
                        y = act_apply(p.act, y);
                        if (i0 < count && n < p.N) store_one((size_t)m * p.cols + n, y);
                    }
                }
                __syncwarp();          // (the loads above are complete: their values were used)
                if (lane == 0)
                    for (int r = 0; r < p.split; ++r) peer_arrive(peer(parts_taken, r));
            } else {
                // (x is in registers of every lane; its chunk's rows are x.m0 + c0 + i)
                const int n = x.n0 + 32 * q + lane;
                const size_t en = (size_t)x.e * p.N + min(n, p.N - 1);
                const float ws = p.b_scale ? __ldg(p.b_scale + en) : 1.f;
                const float bias = p.bias ? __ldg(p.bias + en) : 0.f;
#pragma unroll 1
                for (int j = 0; j < kParts; ++j) {
                    // the shared columns of overlapping accumulators first: half 0 upwards, half 1 downwards
                    const int c0 = 16 * (h == 0 ? j : 2 * kParts - 1 - j);
                    const int live = min(16, x.rows - c0);       // rows of this chunk (none: <= 0)
                    float v[16];
                    __syncwarp();
                    if (live > 0) tmem_ld16(acc + (uint32_t)c0, v);
                    if (P::kOverlap ? j == 2 : j == kParts - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(acc_empty(P::kOverlap ? 0 : tj & 1));
                    }
                    if (live <= 0) continue;
                    const int m = x.m0 + c0;
                    if (p.a_scale) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] *= __ldg(p.a_scale + m + min(i, live - 1));
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = fmaf(v[i], ws, bias);
                    if (p.c_dtype == DT_BF16) store_chunk<DT_BF16>(p, v, n, m, live, odd);
                    else if (p.c_dtype == DT_F16) store_chunk<DT_F16>(p, v, n, m, live, odd);
                    else store_chunk<DT_F32>(p, v, n, m, live, odd);
                }
                __syncwarp();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (SPLIT) cluster_sync();   // no block leaves while a peer may still read its partial sums
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
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

// The launch for a tile height and cluster size; tiles: at least as many as the call has.
template <int F, int BN, bool SPLIT>
cudaError_t launch(const GroupGemmArgs& a, int fmt, int split, long long tiles, cudaStream_t s) {
    using P = Plan<F, BN, SPLIT>;
    const int bf16 = fmt == GF_BF16, block = F == MX ? 32 : 16;
    Maps maps;
    cudaError_t e = make_map(&maps.a, a.A, F, bf16, a.K, a.M, 0, P::kBoxRows);
    if (e == cudaSuccess) e = make_map(&maps.b, a.B, F, bf16, a.K, a.N, a.E, kCh);
    if (e != cudaSuccess) return e;
    Params p{};
    p.M = a.M; p.E = a.E; p.K = a.K; p.N = a.N;
    p.cols = a.act == ACT_SWIGLU ? a.N / 2 : a.N;
    p.n_tiles = (a.N + kCh - 1) / kCh;
    p.stages = F == HALF ? a.K / 64 : (a.K + 255) / 256;
    p.bf16 = bf16;
    p.split = split;
    p.offsets = a.offsets;
    p.As = static_cast<const uint8_t*>(a.As);
    p.Bs = static_cast<const uint8_t*>(a.Bs);
    if (F != HALF) {
        p.pitch = fp4::scale_pitch(a.K, block);
        p.ktiles = fp4::scale_ktiles(a.K, block);
    }
    p.a_scale = a.a_scale; p.b_scale = a.b_scale; p.bias = a.bias;
    p.residual = a.residual;
    p.C = a.C;
    p.act = a.act; p.c_dtype = a.c_dtype;
    p.status = status_word_address();
    if (!p.status) return cudaErrorUnknown;
    p.wait_ns = option_wait_ns();
    p.stall = option_stall();
    auto kern = group_gemm_kernel<F, BN, SPLIT>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)P::kSmem);
    if (e != cudaSuccess) return e;
    const long long most = kTargetSms / split;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((tiles < most ? tiles : most) * split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = P::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = SPLIT ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

// Rows of a group, for the choice of the tile's height: the dense product's, or the mean over the
// experts that can have any.
inline int group_rows(const GroupGemmArgs& a) {
    if (!a.offsets) return a.M;
    const int used = a.M < a.E ? a.M : a.E;
    return (a.M + used - 1) / used;
}
inline long long most_tiles(const GroupGemmArgs& a, int bn) {
    const long long groups = a.offsets ? (a.M < a.E ? a.M : a.E) : 1;
    return (a.M / bn + groups) * ((a.N + kCh - 1) / kCh);
}

template <int F>
cudaError_t launch_form(const GroupGemmArgs& a, int fmt, cudaStream_t s) {
    const int rows = group_rows(a), stages = F == HALF ? a.K / 64 : (a.K + 255) / 256;
    const int bn = rows <= 32 ? 32 : (rows <= 128 ? 128 : 256);
    const long long tiles = a.offsets ? most_tiles(a, bn) : (long long)((a.M + bn - 1) / bn) * ((a.N + kCh - 1) / kCh);
    if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
    int split = 1;
    while (bn < 256 && split < kMaxSplit && tiles * split * 2 <= kTargetSms && stages / (split * 2) >= 2) split *= 2;
    if (bn == 32) return split > 1 ? launch<F, 32, true>(a, fmt, split, tiles, s) : launch<F, 32, false>(a, fmt, 1, tiles, s);
    if (bn == 128) return split > 1 ? launch<F, 128, true>(a, fmt, split, tiles, s) : launch<F, 128, false>(a, fmt, 1, tiles, s);
    return launch<F, 256, false>(a, fmt, 1, tiles, s);
}

}  // namespace gg
}  // namespace qg
