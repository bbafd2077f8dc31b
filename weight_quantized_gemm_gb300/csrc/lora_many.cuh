// The adapters' products for batches of many rows, on the tensor cores' asynchronous path (lora.cuh has the few rows, and
// the mathematics): Y[m] += scale_l B_l (A_l X[m]), a cluster of blocks to a tile of 128 rows of one adapter (64 at ranks
// above 128).
//
//   first product   D1 = X A^T (128 x RP) in tensor memory, a ring of stages of 64 of K (rows of 128 bytes in the
//                   128-byte swizzle) filled by asynchronous copies of all threads, since the rows of a tile lie
//                   anywhere in X. The cluster's blocks share K;
//   join            each block adds 128 / C rows of the blocks' parts, in rank order, splits them into 16-bit terms and
//                   writes these, as the second product's operand, into every block's shared memory;
//   second product  D2 = H B^T, 64 columns a turn (32 for float32 Y) in two buffers of tensor memory: while the tensor cores work on a turn,
//                   all warps add the one before to Y. Y passes through shared memory, copied in and stored by whole
//                   128-byte runs. The blocks share N.
// RP: the ranks rounded up to a power of two; what lies past an adapter's rank is filled with zeros.
//
// There are few operations to a byte, so HBM's bytes are the floor: X, Y and Y again. 8192 x 4096 x 14336 at rank 16 in
// bf16 takes 97 us (5.5 TB/s; a kernel that does nothing but add 1 to that Y in 128-byte runs takes 80 for its 470 MB,
// and 67 MB of X come on top), at rank 64 120; 4099 x 2560 x 2560 at rank 128 28 us, with one block an SM, in which the first
// product takes 6.6 (1260 cycles a stage of 32 KB), the join 4 and a turn 1.1. With 16x8x16 steps from registers, as in
// lora.cuh, these took 109, 189 and 61 us: 12 instructions a value of Y, and the loads that feed
// such steps. Waiting for all memory before each turn's products, and not for shared memory alone, made 102 us 151.
// One block an SM whose warps add to Y without block barriers (a warp its own rows, groups of warps in turns) took the
// same time at rank 16, and 159 and 40 us at ranks 64 and 128, where the one warp that fed the products fell behind. A and B by
// tiled copies of one thread, with the ranks past the adapter's masked, changed nothing (28.1 -> 29.2 us at rank 128).
//
// Every wait is bounded (see ptx.cuh). After a wait that ran out the blocks still meet at the cluster's barriers, wait
// for the MMAs in flight and release their tensor memory.
#pragma once

#include "group_gemm.cuh"
#include "lora.cuh"

namespace qg {
namespace lora {

constexpr int kManyRows = 128;          // of a tile, and of the tensor cores' products

template <int YDT, int RP, int TERMS>
struct Many {
    static constexpr int kYSize = YDT == DT_F32 ? 4 : 2;
    // Rows of a tile: with 256 ranks H of 128 would not fit. The products are formed of 128 all the same; what they read
    // behind a tile's rows is other operands' memory, and what comes of it is not used.
    static constexpr int kRows = RP > 128 ? 64 : kManyRows;
    // The warp that issues the products: one of the eight, or where a turn has 16 of them or more one of its own (4099 x 2560 x
    // 2560 at rank 128: 31 -> 29 us; at ranks up to 64 two blocks an SM lose more by it than they gain).
    static constexpr int kIssuer = RP > 64 ? kWarps : 0, kAll = RP > 64 ? kThreads + 32 : kThreads;
    static constexpr int kCols = 128 / kYSize;                                         // of a turn: 128 bytes of a row of Y
    static constexpr int kX = kRows * 128, kStage = kX + RP * 128;                  // a stage: X's rows, A's ranks
    static constexpr int kBPitch = RP < 64 ? RP * 2 : 128, kBAtoms = (RP + 63) / 64;    // bytes of a column of B, 64 ranks at a time
    static constexpr int kY = kRows * 128, kB = kBAtoms * kCols * kBPitch, kTurn = kY + kB;
    static constexpr int kHAtoms = (TERMS * RP + 63) / 64, kHAtom = kRows * 128, kH = kHAtoms * kHAtom + (kManyRows - kRows) * 128;
    static constexpr int kRoom = (RP <= 64 ? 112 << 10 : 225 << 10) - kH - 2048;        // two blocks an SM where they fit
    static constexpr int kTurns = kRoom / kTurn < 5 ? kRoom / kTurn : 5;                // ring of turns
    static constexpr int kStages = kTurns * kTurn / kStage < 5 ? kTurns * kTurn / kStage : 5;
    // The first product's stages go to kSums accumulators in turn, each of which is emptied after kChain stages if there are
    // more: the tensor cores cut sums off instead of rounding them, and shorter chains lose less (f16 to float32, 6000 rows,
    // K = 8192: off by 5.0e-7 at rank 128 and 6.4e-7 at 256, a float32 product by 6.0e-7 and 1.6e-6; never emptied, with half as
    // many accumulators, by 2.8e-6 and 1.0e-5). They are emptied into registers, in which this costs no time, and at ranks above
    // 128, for which there are too few of those, into H's place (4099 x 2560 x 2560 48 -> 52 us, with registers on the stack 53).
    // The second product's two accumulators take the place of these.
    static constexpr int kTmem = RP <= 64 ? 256 : 512, kSums = kTmem / RP, kChain = 4;
    static constexpr bool kHeld = RP <= 128;        // in registers
    static_assert(kHeld || kRows * RP * 4 <= kH, "H's place");
    static_assert(kSums >= 2 && 2 * kCols <= kTmem, "accumulators");
    static constexpr int kPartPitch = RP + 4;                                          // floats: 16-byte writes of 8 rows meet no bank twice
    static constexpr int kRing = kTurns * kTurn;
    static constexpr size_t kSmem = 1024 + kRing + kH;
    static_assert(kTurns >= 3 && kStages >= 2 && kTurn % 1024 == 0 && kStage % 1024 == 0, "rings");
    static_assert(kRows * kPartPitch * 4 <= (kTurns - 1) * kTurn, "the parts of H take the ring's place but for one turn's");
    static_assert(3 * kSmem > (228 << 10), "at most two blocks an SM, whose tensor memory is there");
};

struct ManyParams {
    LoraArgs a;
    unsigned int* status;
    long long wait_ns;
    int stall;
};

// 16 bytes, zeros where there is nothing to copy. L2 fetches 256 bytes from HBM at a time, the next stage's or turn's 128 with
// this one's (8192 x 4096 x 14336 at rank 16 100.9 -> 98.3 us, at rank 64 131.9 -> 125.2).
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool any) {
    const int bytes = any ? 16 : 0;
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 read16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void write16(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Shared memory written by threads, of this block or another of the cluster, before the tensor cores read it.
__device__ __forceinline__ void to_tensor_cores() { asm volatile("fence.proxy.async;" ::: "memory"); }
// Where 16-byte piece c of row r is, rows of PITCH bytes in the swizzle of that width: the piece's number is combined
// with the bits of the address three places above it.
template <int PITCH>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    constexpr int kShift = PITCH == 128 ? 0 : (PITCH == 64 ? 1 : 2);
    return r * PITCH + ((c ^ ((r >> kShift) & (PITCH / 16 - 1))) << 4);
}
// The high word of such rows' matrix descriptor (K-major, eight rows 8 PITCH bytes apart; swizzles of 128, 64 and 32
// bytes are numbers 2, 4 and 6).
template <int PITCH>
constexpr uint32_t kDescHi = (8u * PITCH >> 4) | (1u << 14) | ((PITCH == 128 ? 2u : (PITCH == 64 ? 4u : 6u)) << 29);
// D (+)= A B^T over 16 of K, issued by one lane of the (whole) warp: A's rows of 128 bytes, B's of PITCH. a, b: the
// descriptors' low words.
template <int PITCH>
__device__ __forceinline__ void mma_async(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %6};\n\t"
        "setp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "n"(kDescHi<128>), "n"(kDescHi<PITCH>)
        : "memory");
}

template <bool BF, int YDT, int RP, bool WIDE>
__global__ void __launch_bounds__(RP > 64 ? kThreads + 32 : kThreads, RP <= 64 ? 2 : 1) lora_many_kernel(const ManyParams p) {
    constexpr int kTerms = terms_of(BF, YDT);
    using S = Many<YDT, RP, kTerms>;
    constexpr int kYSize = S::kYSize, kTurnCols = S::kCols, kHalf = kTurnCols / 2;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) unsigned long long s_bar[S::kStages + 3];      // stages, the two buffers of D2, one that never completes
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ TileSearch s_tile;
    __shared__ int s_row[kManyRows];
    __shared__ float s_unit[kManyRows];         // f16: the power of two that a row of H was divided by
    const LoraArgs& a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int blocks = (int)cluster_size(), shift = __ffs(blocks) - 1, rank_in = blocks > 1 ? (int)cluster_rank() : 0;      // (a power of two, of 8 at most)
    const uint32_t ring = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;       // (the same offset in every block)
    const uint32_t H = ring + S::kRing;
    const uint32_t bar = ptx::smem_u32(s_bar);
    volatile int* abort_flag = &s_abort;
    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < S::kStages + 3; ++i) ptx::mbar_init(bar + 8 * i, 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        // (before the next kernel may come up, and at most two blocks an SM: the columns are free, or will be)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_u32(&s_tmem)), "r"(S::kTmem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    gg::tc_fence_before();
    __syncthreads();
    gg::tc_fence_after();
    const uint32_t tmem = s_tmem;
    grid_wait();
    grid_release();
    int l = 0, from = 0, count = 0;
    const bool any = find_tile(a, blockIdx.x >> shift, S::kRows, s_tile, l, from, count);
    // (the rows, the rank and the scale are asked for together)
    const int m_here = any && tid < count ? load(a.row + from + tid) : -1;
    const float scale = any && a.scale ? load(a.scale + l) : 1.f;
    const int rank = !any ? 0 : (a.rank ? min(max(load(a.rank + l), 0), a.R) : a.R);
    if (rank > 0) {             // (the same for the whole cluster)
        if (tid < S::kRows) {
            s_row[tid] = m_here < a.M ? m_here : -1;
            s_unit[tid] = 1.f;
        }
        __syncthreads();
        bool fail = false;
        auto wait = [&](int i, uint32_t parity) { return ptx::mbar_wait(bar + 8 * i, parity, abort_flag, p.status, p.wait_ns); };
        // The diagnostic wait that runs out is the one for the products of a first stage (whose barrier is number 0), or in every
        // other block for those of a first turn (number kStages), on the barrier that never completes (number kStages + 2).
        const bool odd = blockIdx.x & 1u;
        const int stuck1 = p.stall && !odd ? S::kStages + 2 : 0, stuck2 = p.stall && odd ? 2 : 0;
        const int c8 = tid & 7, r8 = tid >> 3;      // 8 threads copy a row's 128 bytes, 32 rows at a time
        const bool copier = RP <= 64 || warp != S::kIssuer;

        // a warp reads its quarter's lanes of tensor memory, and half of the columns (the issuer of its own none)
        const int quarter = warp & 3, half = warp >> 2, row = quarter * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)quarter * 32 << 16);
        const bool reads = copier && row < S::kRows;
        float held[S::kHeld ? (RP + 31) / 32 : 1][16] = {};
        float* spare = reinterpret_cast<float*>(smem_raw + (H - ptx::smem_u32(smem_raw))) + row;        // [RP][kRows], this thread's row

        // ---- D1 = X A^T over this block's part of K
        const int steps = a.K / 64;
        const int s0 = steps * rank_in >> shift, n1 = (steps * (rank_in + 1) >> shift) - s0;        // (K <= 2^30)
        {
            constexpr int kXC = S::kRows / 32, kAC = (RP + 31) / 32;
            const uint8_t* x[kXC];
            uint32_t live = 0;
#pragma unroll
            for (int i = 0; i < kXC; ++i) {
                const int m = copier ? s_row[r8 + 32 * i] : -1;
                live |= (m >= 0 ? 1u : 0u) << i;
                x[i] = static_cast<const uint8_t*>(a.X) + ((long long)max(m, 0) * a.ldx + (size_t)s0 * 64 + c8 * 8) * 2;
            }
            const uint8_t* A = static_cast<const uint8_t*>(a.A) + (((size_t)l * a.R + r8) * a.K + (size_t)s0 * 64 + c8 * 8) * 2;
            const uint32_t to = ring + swizzled<128>(r8, c8);        // (rows 32 apart have the same swizzle)
            auto fetch = [&](int i, int slot) {
                if (copier && i < n1) {
                    const uint32_t at = to + slot * S::kStage;
#pragma unroll
                    for (int j = 0; j < kXC; ++j) copy16(at + j * 32 * 128, x[j] + (size_t)i * 128, live >> j & 1u);
#pragma unroll
                    for (int j = 0; j < kAC; ++j)
                        if (RP >= 32 || r8 < RP) {
                            const bool in = r8 + 32 * j < rank;
                            copy16(at + S::kX + j * 32 * 128, in ? A + ((size_t)j * 32 * a.K + (size_t)i * 64) * 2 : a.A, in);
                        }
                }
                copies_end();
            };
            const uint32_t idesc = gg::inst_desc<gg::HALF>(kManyRows, RP, BF);
            // Empties the accumulator of stage j (whose products have ended) if it is full and used again. The stage after j, whose
            // products are in flight, has another; the next one that has the same is issued behind a barrier.
            auto empty = [&](int j) {
                if (j / S::kSums % S::kChain != S::kChain - 1 || j + S::kSums >= n1 || !reads) return;
                __syncwarp();       // (the lanes may leave a wait one by one)
                gg::tc_fence_after();
#pragma unroll
                for (int c = 0; c < RP; c += 32)
                    if (c + half * 16 < RP) {
                        float w[16];
                        gg::tmem_ld(lanes + j % S::kSums * RP + c + half * 16, w);
                        if constexpr (S::kHeld) {
#pragma unroll
                            for (int k = 0; k < 16; ++k) held[c / 32][k] += w[k];
                        } else {
                            float* to = spare + (c + half * 16) * S::kRows;
                            const bool first = j == S::kSums * (S::kChain - 1);
#pragma unroll
                            for (int k = 0; k < 16; ++k) to[k * S::kRows] = first ? w[k] : to[k * S::kRows] + w[k];
                        }
                    }
                gg::tc_fence_before();
            };
#pragma unroll
            for (int d = 0; d < S::kStages - 1; ++d) fetch(d, d);
            int slot = 0, before = S::kStages - 1;
            uint32_t parity = 1;        // of the slot before this one
            for (int i = 0; i < n1; ++i) {
                copies_wait<S::kStages - 2>();
                ptx::fence_proxy_async_smem();
                if (__syncthreads_or(fail)) {
                    fail = true;
                    break;
                }
                if (warp == S::kIssuer) {
                    gg::tc_fence_after();
                    const uint32_t at = ring + slot * S::kStage;
                    uint32_t xa = gg::rows_lo(at), wa = gg::rows_lo(at + S::kX);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_async<128>(tmem + i % S::kSums * RP, xa + 2 * k, wa + 2 * k, idesc, i / S::kSums % S::kChain != 0 || k > 0);
                    gg::mma_commit<gg::SOLO>(bar + 8 * slot);
                }
                if (i > 0) {
                    fail = fail || !wait(before + stuck1, parity);       // the stage before has been read
                    empty(i - 1);
                }
                fetch(i + S::kStages - 1, before);
                before = slot;
                if (++slot == S::kStages) slot = 0;
                parity = (uint32_t)(i / S::kStages) & 1u;
            }
            // MMAs in flight end before anything else happens to what they read and write
            copies_wait<0>();
            if (n1 > 0 && !fail) fail = !wait(before + stuck1, parity);
            fail = __syncthreads_or(fail);
        }

        // ---- the second product's first turn comes while the blocks join their parts of H (behind which it has room)
        const int turns = (a.N + kTurnCols - 1) / kTurnCols;
        const int t0 = turns * rank_in >> shift, n2 = (turns * (rank_in + 1) >> shift) - t0;        // (N <= 2^30)
        constexpr int kPer = 16 / kYSize, kYC = S::kRows / 32;        // values of a 16-byte piece; pieces of a thread
        const uint32_t y_to = swizzled<128>(r8, c8);
        // A turn is whole where all of its columns are there and rows of Y start 16-byte aligned. This thread's pieces of the
        // turn that is stored; those of the turn that is fetched lie kAhead turns further on. Rows that are not there
        // have nothing to copy (`full`: none is missing).
        constexpr int kAhead = S::kTurns - 1, kTurnBytes = kTurnCols * kYSize;
        uint8_t* y_at[kYC];
        uint32_t there = 0;
#pragma unroll
        for (int i = 0; i < kYC; ++i) {
            const int m = copier ? s_row[r8 + 32 * i] : -1;
            there |= (m >= 0 ? 1u : 0u) << i;
            y_at[i] = static_cast<uint8_t*>(a.Y) + ((long long)max(m, 0) * a.ldy + (size_t)t0 * kTurnCols + c8 * kPer) * kYSize;
        }
        if (!WIDE) there = 0;
        const bool full = there == (1u << kYC) - 1;
        auto whole = [&](int u) { return (t0 + u + 1) * kTurnCols <= a.N; };
        // (8 columns belong together: they are copied, or at the row's end added one by one)
        auto copied = [&](int u) { return whole(u) || (t0 + u) * kTurnCols + (c8 * kPer / 8 + 1) * 8 <= a.N; };
        constexpr int kBPieces = (RP < 64 ? RP : 64) / 8 * S::kBAtoms;      // 16-byte pieces of a column of B
        constexpr int kBC = (kTurnCols * kBPieces + kThreads - 1) / kThreads, kBApart = kThreads / kBPieces;
        const int bn = tid / kBPieces, bc = tid % kBPieces;
        const uint8_t* b_at = static_cast<const uint8_t*>(a.B) + (((size_t)l * a.N + (size_t)t0 * kTurnCols + bn) * a.R + bc * 8) * 2;
        const uint32_t b_to = S::kY + (bc >> 3) * (kTurnCols * S::kBPitch) + swizzled<S::kBPitch>(bn, bc & 7);     // (kBApart is a multiple of 8)
        static_assert(kBApart % 8 == 0, "columns a thread copies have one order of pieces");
        const int b_bytes = min(max(rank - bc * 8, 0), 8) * 2;              // a piece's values past the adapter's rank become zeros
        // Rows of Y that start anywhere: a warp copies a row at a time, a lane a 4-byte word of it. Of 16-bit rows that start
        // between two words a lane reads and writes its two values one by one. 8192 rows at rank 16 beside 4096 x 5760, bf16:
        // 55 us aligned, 99 in rows of 5762 and 258 of 5761 values, in float32 81, 142 and 144 (with a lane a row's 8 values
        // one after the other 2500 to 2800).
        constexpr int kLoose = S::kRows / kWarps, kWordValues = 4 / kYSize;
        auto loose = [&](int u, auto each) {        // each(word's place in a tile, its address, its values that are there, whether it is a word in memory)
            const int n = (t0 + u) * kTurnCols + lane * kWordValues, left = a.N - n;
#pragma unroll 8
            for (int i = 0; i < kLoose; ++i) {
                const int r = warp + i * kWarps, m = s_row[r];
                uint8_t* p = static_cast<uint8_t*>(a.Y) + ((long long)max(m, 0) * a.ldy + n) * kYSize;
                if (m >= 0 && left > 0)
                    each(swizzled<128>(r, lane >> 2) + (lane & 3) * 4, p, min(left, kWordValues), kYSize == 4 || (reinterpret_cast<uintptr_t>(p) & 2u) == 0);
            }
        };
        // fetches turn u; y_at is kAhead - `back` turns before it
        auto fetch = [&](int u, int slot, int back) {
            if (copier && u < n2) {
                const uint32_t at = ring + slot * S::kTurn;
                if constexpr (!WIDE) {
                    loose(u, [&](uint32_t to, const uint8_t* p, int values, bool word) {
                        if (word) {
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(at + to), "l"(p), "r"(values * kYSize) : "memory");
                        } else {
                            uint32_t v = load(reinterpret_cast<const uint16_t*>(p));
                            if (values > 1) v |= (uint32_t)load(reinterpret_cast<const uint16_t*>(p) + 1) << 16;
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + to), "r"(v) : "memory");
                        }
                    });
                } else if (copied(u)) {
#pragma unroll
                    for (int i = 0; i < kYC; ++i)
                        if (full || (there >> i & 1u)) copy16(at + y_to + i * 32 * 128, y_at[i] + (kAhead - back) * kTurnBytes, true);
                }
#pragma unroll
                for (int i = 0; i < kBC; ++i) {
                    const int n = bn + i * kBApart;
                    if (kTurnCols * kBPieces % kThreads != 0 && n >= kTurnCols) break;
                    const int bytes = whole(u) || (t0 + u) * kTurnCols + n < a.N ? b_bytes : 0;
                    const uint8_t* src = bytes ? b_at + ((size_t)u * kTurnCols + i * kBApart) * a.R * 2 : static_cast<const uint8_t*>(a.B);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at + b_to + i * kBApart * S::kBPitch), "l"(src), "r"(bytes) : "memory");
                }
            }
            copies_end();
        };
        const uint32_t idesc = gg::inst_desc<gg::HALF>(kManyRows, kTurnCols, BF);
        if (!fail) fetch(0, S::kTurns - 1, kAhead);

        // ---- the block's part of H, where the stages were
        float* part = reinterpret_cast<float*>(smem_raw + (ring - ptx::smem_u32(smem_raw)));      // [128][kPartPitch]
        gg::tc_fence_after();
#pragma unroll
        for (int c = 0; c < RP; c += 32) {
            float (&v)[16] = held[S::kHeld ? c / 32 : 0];
            if (reads && c + half * 16 < RP) {
                if (!S::kHeld)
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = n1 > S::kSums * S::kChain ? spare[(c + half * 16 + j) * S::kRows] : 0.f;
                for (int d = 0; d < min(n1, S::kSums); ++d) {
                    float w[16];
                    gg::tmem_ld(lanes + d * RP + c + half * 16, w);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] += w[j];
                }
                float4* to = reinterpret_cast<float4*>(part + row * S::kPartPitch + c + half * 16);
#pragma unroll
                for (int j = 0; j < 4; ++j) to[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            }
        }
        gg::tc_fence_before();
        if (blocks > 1) cluster_sync();
        else __syncthreads();

        // ---- this block's share of the rows: summed, and their terms to every block
        {
            constexpr int kLanes = RP < 128 ? RP / 4 : 32, kSets = RP / 4 / kLanes;      // of a row, sets of 4 values each
            const int rows = S::kRows >> shift;
            for (int i = tid; i < rows * kLanes; i += S::kAll) {
                const int r = rank_in * rows + i / kLanes;
                float x[kSets][4], most = 0.f;
#pragma unroll
                for (int e = 0; e < kSets; ++e) {
                    const int c = (i % kLanes + e * kLanes) * 4;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int b0 = 0; b0 < blocks; b0 += 4) {
                        float4 o[4];
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (b0 + b < blocks) o[b] = ld_cluster_f32x4(in_block(part + r * S::kPartPitch + c, b0 + b));
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (b0 + b < blocks) {
                                v.x += o[b].x; v.y += o[b].y; v.z += o[b].z; v.w += o[b].w;
                            }
                    }
                    x[e][0] = v.x; x[e][1] = v.y; x[e][2] = v.z; x[e][3] = v.w;
                    // columns past the rank become zeros: A's zeros there times an infinite X were NaN
                    if (rank < RP)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (c + k >= rank) x[e][k] = 0.f;
                    if constexpr (!BF)
#pragma unroll
                        for (int k = 0; k < 4; ++k) most = fmaxf(most, finite_size(x[e][k]));
                }
                if constexpr (!BF) {
#pragma unroll
                    for (int o = 1; o < kLanes; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));      // (whole warps are in the loop)
                    const uint32_t bits = __float_as_uint(most);
                    const float by = row_unit_inverse(bits);
#pragma unroll
                    for (int e = 0; e < kSets; ++e)
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[e][k] *= by;
                    if (i % kLanes == 0)
                        for (int b = 0; b < blocks; ++b)
                            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(in_block(&s_unit[r], b)), "f"(row_unit(bits)) : "memory");
                }
#pragma unroll
                for (int e = 0; e < kSets; ++e)
#pragma unroll
                    for (int t = 0; t < kTerms; ++t) {
                        uint32_t w[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t lo = take_term<BF>(x[e][2 * k]), hi = take_term<BF>(x[e][2 * k + 1]);
                            w[k] = lo | hi << 16;
                        }
                        const int col = t * RP + (i % kLanes + e * kLanes) * 4;
                        const uint32_t at = H + (col >> 6) * S::kHAtom + swizzled<128>(r, (col & 63) >> 3) + (col & 7) * 2;
                        for (int b = 0; b < blocks; ++b) {
                            uint32_t to;
                            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(b));
                            asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(to), "r"(w[0]), "r"(w[1]) : "memory");
                        }
                    }
            }
        }
        to_tensor_cores();
        if (blocks > 1) cluster_sync_all();     // (from here on no block reads another's shared memory)
        else __syncthreads();
        to_tensor_cores();

        // ---- Y += scale H B^T, a turn's columns at a time
        const int chunks = (rank + 15) / 16;
        const float by = scale * s_unit[row];       // exact: a power of two
        const int my_row = row < S::kRows ? s_row[row] : -1;
        const uint32_t y_cell = swizzled<128>(row, 0);      // (a row's pieces differ in the same three bits)
#pragma unroll
        for (int d = 1; d < S::kTurns - 2; ++d) fetch(d, d - 1, kAhead - d);
        int slot = S::kTurns - 1, before = S::kTurns - 2, next = S::kTurns - 3;        // this turn's, the last turn's, and the one to fill
        // one turn more than there are: each adds the turn before to Y
        for (int u = 0; u <= n2 && n2 > 0; ++u) {
            copies_wait<S::kTurns - 3>();
            ptx::fence_proxy_async_smem();
            gg::tc_fence_before();
            if (__syncthreads_or(fail)) {       // this turn is in; the one before the last is stored, and its accumulator read
                fail = true;
                break;
            }
            if (warp == S::kIssuer && u < n2) {
                gg::tc_fence_after();
                const uint32_t d = tmem + (u & 1) * kTurnCols, bt = ring + slot * S::kTurn + S::kY;
                // (the small terms first: a sum is cut off by what its size is)
                for (int t = kTerms - 1; t >= 0; --t)
                    for (int k = 0; k < chunks; ++k) {
                        const int col = t * RP + k * 16;
                        const uint32_t ha = gg::rows_lo(H + (col >> 6) * S::kHAtom) + ((col & 63) >> 3);
                        const uint32_t ba = gg::rows_lo(bt + (k >> 2) * (kTurnCols * 128)) + 2 * (k & 3);
                        mma_async<S::kBPitch>(d, ha, ba, idesc, t < kTerms - 1 || k > 0);
                    }
                gg::mma_commit<gg::SOLO>(bar + 8 * (S::kStages + (u & 1)));
            }
            fetch(u + S::kTurns - 2, next, u > 0 ? 0 : 1);
            if (u > 0 && !copier) {
                if (__syncthreads_or(fail)) {
                    fail = true;
                    break;
                }
            } else if (u > 0) {
                const int v = u - 1, n = (t0 + v) * kTurnCols + half * kHalf;
                const uint32_t tile = ring + before * S::kTurn;
                fail = fail || !wait(S::kStages + stuck2 + (v & 1), (uint32_t)(v >> 1) & 1u);
                __syncwarp();       // (the lanes may leave a wait one by one, and read tensor memory together)
                gg::tc_fence_after();
                const bool mine = row < S::kRows;        // (the same for the whole warp)
                float acc[kHalf];
                if (mine) gg::tmem_ld(lanes + (v & 1) * kTurnCols + half * kHalf, acc);
                constexpr int kV = Eight<YDT>::kVecs;
                // (what rows that are not there hold in shared memory goes nowhere; all is read before the first is written,
                // as the compiler keeps the order of these accesses)
                Eight<YDT> y[kHalf / 8];
                const bool fast = mine && (!WIDE || whole(v));       // (values past N go nowhere either)
#pragma unroll
                for (int j = 0; j < kHalf / 8; ++j)
                    if (fast || (mine && n + 8 * j + 8 <= a.N))
#pragma unroll
                        for (int k = 0; k < kV; ++k) y[j].v[k] = read16(tile + (y_cell ^ ((half * 4 + j * kV + k) << 4)));
#pragma unroll
                for (int j = 0; j < kHalf / 8; ++j) {
                    if (fast || (mine && n + 8 * j + 8 <= a.N)) {
                        float x[8];
                        y[j].values(x);
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[k] = fmaf(by, acc[8 * j + k], x[k]);
                        y[j].round_from(x);
#pragma unroll
                        for (int k = 0; k < kV; ++k) write16(tile + (y_cell ^ ((half * 4 + j * kV + k) << 4)), y[j].v[k]);
                    } else if (n + 8 * j < a.N && my_row >= 0 && !fail) {
                        float d[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) d[k] = acc[8 * j + k];
                        add_edge<YDT>(static_cast<uint8_t*>(a.Y) + ((long long)my_row * a.ldy + n + 8 * j) * kYSize, d, by, a.N - n - 8 * j);
                    }
                }
                if (__syncthreads_or(fail)) {       // the tile is summed
                    fail = true;
                    break;
                }
                if constexpr (!WIDE) {
                    loose(v, [&](uint32_t from, uint8_t* p, int values, bool word) {
                        uint32_t w;
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(tile + from) : "memory");
                        if (word && values == kWordValues) {
                            *reinterpret_cast<uint32_t*>(p) = w;
                        } else {
                            *reinterpret_cast<uint16_t*>(p) = (uint16_t)w;
                            if (values > 1) *(reinterpret_cast<uint16_t*>(p) + 1) = (uint16_t)(w >> 16);
                        }
                    });
                } else if (copied(v)) {
                    uint4 out[kYC];
#pragma unroll
                    for (int i = 0; i < kYC; ++i) out[i] = read16(tile + y_to + i * 32 * 128);
#pragma unroll
                    for (int i = 0; i < kYC; ++i)
                        if (full || (there >> i & 1u)) *reinterpret_cast<uint4*>(y_at[i]) = out[i];
                }
#pragma unroll
                for (int i = 0; i < kYC; ++i) y_at[i] += kTurnBytes;
            }
            before = slot;
            if (++slot == S::kTurns) slot = 0;
            if (++next == S::kTurns) next = 0;
        }
        copies_wait<0>();
        if (fail) {
            // The MMAs issued end before the tensor memory is released: a commit of the warp that issued them, as one
            // tracks its own thread's alone.
            volatile int never = 0;
            __syncthreads();
            if (warp == S::kIssuer) {
                gg::mma_commit<gg::SOLO>(bar + 8 * (S::kStages + 2));
                ptx::mbar_wait(bar + 8 * (S::kStages + 2), 0, &never, p.status);
            }
        }
    }
    gg::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        gg::tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kTmem) : "memory");
    }
}

template <bool BF, int YDT, int RP, bool WIDE>
cudaError_t launch_many(const LoraArgs& a, int blocks, cudaStream_t s) {
    using S = Many<YDT, RP, terms_of(BF, YDT)>;
    const ManyParams p{a, status_word_address(), option_wait_ns(), option_stall()};
    if (!p.status) return cudaErrorUnknown;
    auto kern = lora_many_kernel<BF, YDT, RP, WIDE>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
    if (e != cudaSuccess) return e;
    // at most one tile that is not full for each adapter that has rows
    const long long tiles = (long long)a.M / S::kRows + (a.L < a.M ? a.L : a.M);
    return launch_behind(kern, dim3((unsigned)(tiles * blocks)), dim3(S::kAll), S::kSmem, (unsigned)blocks, s, p);
}

// Largest power of two up to 8 of which `tiles` clusters make at most `most` blocks (1 at least).
inline int blocks_of(long long tiles, int most) {
    int blocks = 1;
    while (blocks < 8 && tiles * blocks * 2 <= most) blocks *= 2;
    return blocks;
}

template <bool BF, int YDT, bool WIDE>
cudaError_t launch_y(const LoraArgs& a, cudaStream_t s) {
    // Tiles of 128 rows where there are many rows; from how many on depends on the rank, as the few rows' kernel reads each
    // adapter once for every 16 rows, and from where on it needs a second round of blocks (4096 x 14336, us, few / many:
    // rank 16 2048 rows 42 / 51, 2900 rows 74 / 53; rank 32 1500 rows 46 / 45; rank 64 1024 rows 37 / 48, 1300 rows 65 / 49;
    // rank 128 512 rows 45 / 47, 900 rows 60 / 49, and 2560 x 2560 768 rows 20 / 19, 1024 rows 21 / 19). These two widths are all
    // that was measured, and just above the border the other kernel may be the quicker one (rank 16, 2400 rows 44 / 49: its
    // second round of blocks begins between 2400 and 2900). The cluster's size
    // fills the SMs once (two blocks an SM, one at rank 128), with the number of tiles guessed from M and L, since the host
    // does not see the offsets: of 8192 rows, 4 blocks take 102 us, 8 117 and 2 142 (before L2 fetched 256 bytes).
    const int rank = a.R <= 16 ? 16 : (a.R <= 32 ? 32 : (a.R <= 64 ? 64 : (a.R <= 128 ? 128 : 256)));
    const int from = rank == 16 ? 2304 : (rank == 32 ? 1536 : (rank == 64 ? 1280 : (rank == 128 ? 768 : 256)));
    // Ranks above 128 (tiles of 64 rows, as H of more would not fit): from 256 rows on, where two terms stand for H
    // (2560 x 2560 at rank 256, bf16: 256 rows 28 / 18, 512 rows 37 / 20, 4099 rows 101 / 57; f16 to float32 4099 rows 109 / 79).
    // With three (bf16 to float32) what H leaves of shared memory is too little (6000 x 8192 x 8192 440 / 572).
    // An adapter's rows must fill tiles: 64 of them on average (4096 x 14336, rank 16, rows drawn at random, us: 2400 rows of 100
    // adapters 75 / 129, of 1000 228 / 1073; 2560 x 2560, rank 128, 1000 rows of 30 23 / 35), 16 at ranks above 128 (300 rows
    // of 30 33 / 39).
    constexpr bool kWide = terms_of(BF, YDT) == 2;
    if ((a.R <= 128 || kWide) && a.M >= from && a.M / (rank > 128 ? 16 : 64) >= a.L) {
        const int tiles = a.M / (rank > 128 ? 64 : kManyRows);
        const int blocks = blocks_of(tiles + (a.L < tiles ? a.L : tiles), rank >= 128 ? kTargetSms : 2 * kTargetSms);
        switch (rank) {
            case 16: return launch_many<BF, YDT, 16, WIDE>(a, blocks, s);
            case 32: return launch_many<BF, YDT, 32, WIDE>(a, blocks, s);
            case 64: return launch_many<BF, YDT, 64, WIDE>(a, blocks, s);
            case 128: return launch_many<BF, YDT, 128, WIDE>(a, blocks, s);
            default:
                if constexpr (kWide) return launch_many<BF, YDT, 256, WIDE>(a, blocks, s);
        }
    }
    // 8 blocks for a few rows (16 rows of 16 adapters 4.6 us; 4 blocks 5.4), fewer where the tiles alone fill the GPU
    // (1024 rows 23 us with 4, 28 with 8). As many rows as adapters, each row's drawn at random, leave 5/8 of the
    // adapters with rows, a tile each (4096 x 4096, rank 16, us with 2 / 4 / 8 blocks: 48 of each 11.7 / 8.2 / 6.5, 64
    // of each 12.8 / 9.2 / 11.7, 512 rows of 8 adapters 13.9 / 9.0 / 9.3).
    const int blocks = blocks_of(a.M / 16 + (long long)(a.L < a.M ? a.L : a.M) * 5 / 8, kTargetSms * 9 / 4);
    switch (rank) {
        case 16: return launch<BF, YDT, 1, WIDE>(a, blocks, s);
        case 32: return launch<BF, YDT, 2, WIDE>(a, blocks, s);
        default: return launch<BF, YDT, 4, WIDE>(a, blocks, s);
    }
}

template <bool BF, bool WIDE>
cudaError_t launch_form(const LoraArgs& a, int y_dtype, cudaStream_t s) {
    switch (y_dtype) {
        case DT_F32: return launch_y<BF, DT_F32, WIDE>(a, s);
        case DT_F16: return launch_y<BF, DT_F16, WIDE>(a, s);
        default: return launch_y<BF, DT_BF16, WIDE>(a, s);
    }
}

}  // namespace lora
}  // namespace qg
