// Log probabilities of given tokens, entropy and the likeliest tokens of rows of logits, in one pass over them.
//
// With z = scale * logit, M the row's largest z and S = sum exp(z - M):
//   logprob[j] = z_j - M - ln S,   entropy = ln S - sum (z - M) exp(z - M) / S   (both terms are not negative)
// A thread sums 2^t and t 2^t, t = x c - ref with c = scale log2(e), against a reference of its own, which moves only
// when a value is more than kSlack doublings above it (each move rescales both sums; following the largest value itself
// would take that branch in most steps, as some lane of a warp nearly always finds a larger one). The reference is
// a float32 in units of t, and the fused product and difference round once, so its own rounding costs nothing. t is
// held to -200 from below, which makes both terms 0 and takes in -inf and NaN, too: the larger of NaN and -200 is -200.
// Rows whose largest value times c is 2^22 or more are summed a second time, from differences of values.
// Where one logit has more than 2/3 of the probability (the usual row of a model that is sure), ln S is ln(1 + rest) with the rest
// summed without it, so that a token's small -ln p keeps its digits (at 4e-4 it is off by 6e-7 of itself, and not by 1e-3):
// 4 x 128000, k = 8 then takes 7.5 us; for the sums that are kept for it a row without such a logit takes 6.5, before 6.2.
//
// The k likeliest: each thread keeps its largest value and the pieces in which it found it first. The k best of those
// (by value, then place) belong to k threads that must hold the row's k best values: any other thread has k
// values before its own best one. Of these, what is not below the k-th best is read again and put in order; the largest
// value of each thread's every kUnroll pieces is kept beside, so that few pieces are read (with all of these threads'
// pieces, from HBM where the rows in flight exceed L2, 4096 rows of 131072 in bf16 took 185 us with k = 5, and 253 with
// 32). A key is the value's order-preserving bits above the complement of its index, so of
// equal values the lowest index comes first. The usual row is quick: few runs of pieces reach the k-th best value, ties
// and all, and few of their values; these are collected and sorted once. Where equal values make them many (a row of
// zeros), exactly k threads are chosen, and all their values go through the warps' lists 32 at a time.
//
// A row is cut into equal runs of 16-byte pieces for the blocks of a cluster where the batch has few rows; their
// sums and lists meet in the first block through distributed shared memory.
#include <float.h>

#include <type_traits>

#include "serve.cuh"

namespace qg {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kUnroll = 8;                 // 16-byte loads that a thread has in flight
constexpr int kTogether = 4;               // pieces that are summed between two looks at the largest value
constexpr int kRuns = 16;                  // largest values that a thread keeps
constexpr int kQuickRuns = kThreads, kQuickKeys = kThreads;
constexpr int kMaxCluster = 8;
static_assert(kMaxCluster <= kWarps, "a warp reads each block's list");
constexpr float kSlack = 3.f;
constexpr float kFar = 4194304.f;          // of a reference, whose own rounding is then a quarter or more
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
using Key = unsigned long long;

struct Args {
    int V;
    const uint8_t* logits;
    long long ld_bytes;
    float scale, c;             // c = scale * log2(e)
    const int32_t* token;
    float* logprob;
    float* entropy;
    int k;
    int32_t* top;
    float* top_logprob;
};

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xFF800000u); }
__device__ __forceinline__ float pos_inf() { return __uint_as_float(0x7F800000u); }
__device__ __forceinline__ float exp2_fast(float t) {      // 2^t, a few units in the last place; 0 below 2^-126
    float p;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(t));
    return p;
}

// Grows with the value; 0 for -inf and NaN.
__device__ __forceinline__ uint32_t to_key(float x) {
    if (!(x > neg_inf())) return 0u;
    const uint32_t b = __float_as_uint(x + 0.f);   // -0 and 0 are one value
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_key(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// ---------------------------------------------------------------- a warp's 32 keys in falling order
template <class T>
__device__ __forceinline__ T exchange(T x, int o, bool larger) {
    const T y = __shfl_xor_sync(0xffffffffu, x, o);
    return (x > y) == larger ? x : y;
}
template <class T>
__device__ __forceinline__ T sorted(T x, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int o = size >> 1; o; o >>= 1) x = exchange(x, o, ((lane & o) == 0) == ((lane & size) == 0));
    return x;
}
// The 32 largest of two lists in falling order.
template <class T>
__device__ __forceinline__ T merged(T a, T b, int lane) {
    const T y = __shfl_sync(0xffffffffu, b, 31 - lane);
    T x = a > y ? a : y;
#pragma unroll
    for (int o = 16; o; o >>= 1) x = exchange(x, o, (lane & o) == 0);
    return x;
}
// The 32 largest of `count` (a power of two) warps' lists, in warp 0. Every thread of the block calls it.
template <class T>
__device__ __forceinline__ T merge_warps(T key, int count, T (*lists)[32], int warp, int lane) {
    __syncthreads();
    lists[warp][lane] = key;
    for (int h = count >> 1; h; h >>= 1) {
        __syncthreads();
        if (warp < h) {
            key = merged(key, lists[warp + h][lane], lane);
            lists[warp][lane] = key;
        }
    }
    return key;
}

// ---------------------------------------------------------------- a row
template <int DT>
struct Row {
    static constexpr int kSize = DT == DT_F32 ? 4 : 2, kPer = 16 / kSize;
    static constexpr uint32_t kNone = DT == DT_F32 ? 0xFF800000u : (DT == DT_F16 ? 0xFC00FC00u : 0xFF80FF80u);    // -inf
    const uint8_t* from;        // 16-byte aligned, at or before the row's first value
    int skip, end;              // the row is values skip .. end - 1 from there
    __device__ __forceinline__ Row(const uint8_t* row, int V) {
        const int over = (int)(reinterpret_cast<uintptr_t>(row) & 15u);
        from = row - over;
        skip = over / kSize;
        end = skip + V;         // (V <= 2^30)
    }
    __device__ __forceinline__ int pieces() const { return (end + kPer - 1) / kPer; }
    // A piece at an end of the row: the values outside are neither read nor counted.
    __device__ __noinline__ uint4 edge(int v) const {
        uint32_t w[4] = {kNone, kNone, kNone, kNone};
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int i = v * kPer + j;
            if (i < skip || i >= end) continue;
            if constexpr (DT == DT_F32) w[j] = load(reinterpret_cast<const uint32_t*>(from) + i);
            else {
                const uint32_t h = load(reinterpret_cast<const uint16_t*>(from) + i);
                w[j >> 1] = (j & 1) ? (w[j >> 1] & 0xFFFFu) | h << 16 : (w[j >> 1] & 0xFFFF0000u) | h;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ uint4 piece(int v) const {
        if (v * kPer >= skip && (v + 1) * kPer <= end) return load(reinterpret_cast<const uint4*>(from) + v);
        return edge(v);
    }
    // The largest of N pieces' values, NaN left out.
    template <int N>
    __device__ __forceinline__ static float largest(const uint4* raw) {
        if constexpr (DT == DT_F32) {
            float m = __uint_as_float(raw[0].x);
#pragma unroll
            for (int u = 0; u < N; ++u)
                m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(raw[u].x)), __uint_as_float(raw[u].y)), fmaxf(__uint_as_float(raw[u].z), __uint_as_float(raw[u].w)));
            return m;
        } else {        // two at a time
            using T = std::conditional_t<DT == DT_F16, __half2, __nv_bfloat162>;
            const T* p = reinterpret_cast<const T*>(raw);
            T m[4] = {p[0], p[1], p[2], p[3]};
#pragma unroll
            for (int i = 4; i < 4 * N; ++i) m[i & 3] = __hmax2(m[i & 3], p[i]);
            const T all = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
            return fmaxf(__low2float(all), __high2float(all));
        }
    }
    __device__ __forceinline__ static void values(const uint4& raw, float (&x)[kPer]) {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if constexpr (DT == DT_F32) x[j] = __uint_as_float(w[j]);
            else if constexpr (DT == DT_BF16) x[j] = __uint_as_float(j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
            else x[j] = __half2float(__ushort_as_half((unsigned short)(w[j >> 1] >> (16 * (j & 1)))));
        }
    }
};

// Two float32 at once.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// sum of 2^t and of t 2^t against `ref`
struct Sums {
    float ref, s, e;
    // the same against another reference, at or above this one
    __device__ __forceinline__ void against(float to) {
        const float d = ref - to, f = exp2_fast(d);
        e = f > 0.f ? f * fmaf(s, d, e) : 0.f;      // (a reference of -inf has no sums, or none that can be told)
        s = f > 0.f ? s * f : 0.f;
        ref = to;
    }
};
// Sums over the block, in thread 0; part: [kWarps] shared memory.
__device__ __forceinline__ void block_sums(Sums& sums, float2* part, int warp, int lane) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sums.s += __shfl_xor_sync(0xffffffffu, sums.s, o);
        sums.e += __shfl_xor_sync(0xffffffffu, sums.e, o);
    }
    if (lane == 0) part[warp] = make_float2(sums.s, sums.e);
    __syncthreads();
    if (warp == 0 && lane == 0) {
        sums.s = sums.e = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            sums.s += part[w].x;
            sums.e += part[w].y;
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const Args a) {
    using R = Row<DT>;
    constexpr int P = R::kPer;
    __shared__ __align__(16) Key lists[kWarps][32];
    __shared__ Key best[32];            // the block's threads with the largest values, then its largest values
    __shared__ Key found[kQuickKeys];
    __shared__ float runs[kRuns][kThreads];        // each thread's, the largest values of its runs of pieces
    __shared__ int which[kQuickRuns], s_which, s_found;
    __shared__ uint32_t s_least;
    __shared__ float s_top[kWarps];
    __shared__ float2 s_sums[kWarps];
    __shared__ float4 s_again;          // the sums a second time
    __shared__ float2 s_mine[kThreads]; // each thread's sums
    __shared__ int s_owner;             // a thread that holds the block's largest logit
    __shared__ float4 s_block;          // the block's largest logit, and its sums against that
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t blocks = cluster_size(), rank = blocks > 1 ? cluster_rank() : 0u;
    const size_t t = blockIdx.x / blocks;
    grid_wait();
    grid_release();
    const R row(a.logits + (long long)t * a.ld_bytes, a.V);
    const int pieces = row.pieces(), share = (pieces + (int)blocks - 1) / (int)blocks;
    const int v0 = min((int)rank * share, pieces), v1 = min(v0 + share, pieces);

    // the given token's logit, which the end would else wait for
    int token = -1;
    float given = 0.f;
    if (a.logprob && rank == 0 && tid == 0) {
        token = load(a.token + t);
        if (token >= 0 && token < a.V) given = load_as_float<DT>(row.from, (size_t)row.skip + token);
    }

    // ---- the pass
    float most = neg_inf(), limit = neg_inf(), ref = neg_inf();
    int place = 0;
    uint64_t s2 = 0, e2 = 0, minus2 = 0;
    const uint64_t c2 = pack2(a.c, a.c);
    const float slack = kSlack / a.c;
    // A logit in units of t, rounded: not to be fused with what follows, which would then see another reference.
    auto in_units = [&](float x) { return __fmul_rn(x, a.c); };
    auto sums_now = [&]() {
        float s0, s1, e0, e1;
        unpack2(s2, s0, s1);
        unpack2(e2, e0, e1);
        return Sums{ref, s0 + s1, e0 + e1};
    };
    // a run is `per` turns of kUnroll pieces of a thread
    const int turns = (v1 - v0 + kUnroll * kThreads - 1) / (kUnroll * kThreads), per = (turns + kRuns - 1) / kRuns;
    float run_most = neg_inf();
    // N pieces, the first of which is piece v: one look at their largest value, then sums without branches.
    auto take = [&](auto count, const uint4* raw, int v) {
        constexpr int N = decltype(count)::value;
        const float here = R::template largest<N>(raw);
        run_most = fmaxf(run_most, here);
        if (here > most) {
            most = here;
            place = v;
        }
        if (here > limit) {
            Sums sums = sums_now();
            sums.against(in_units(here));
            ref = sums.ref;
            s2 = pack2(sums.s, 0.f);
            e2 = pack2(sums.e, 0.f);
            minus2 = pack2(-ref, -ref);
            limit = here + slack;
        }
#pragma unroll
        for (int u = 0; u < N; ++u) {
            float x[P];
            R::values(raw[u], x);
#pragma unroll
            for (int j = 0; j < P; j += 2) {
                float t0, t1;
                unpack2(fma2(pack2(x[j], x[j + 1]), c2, minus2), t0, t1);
                t0 = fmaxf(t0, -200.f);
                t1 = fmaxf(t1, -200.f);
                const uint64_t p2 = pack2(exp2_fast(t0), exp2_fast(t1));
                s2 = add2(s2, p2);
                e2 = fma2(p2, pack2(t0, t1), e2);
            }
        }
    };
    using One = std::integral_constant<int, 1>;
    using Some = std::integral_constant<int, kTogether>;
    // The row's first and last piece may be cut: by themselves, in their place in the order of each thread's pieces.
    const int whole0 = max(v0, row.skip ? 1 : 0), whole1 = min(v1, row.end / P);
    if (tid == 0 && v0 < min(whole0, v1)) {
        const uint4 raw = row.edge(v0);
        take(One(), &raw, v0);
    }
    int turn = 0, run = 0;          // turns of the run at hand
    for (int v = v0; v < whole1; v += kUnroll * kThreads) {
        const uint4* from = reinterpret_cast<const uint4*>(row.from) + v + tid;
        uint4 raw[kUnroll];
        if (v >= whole0 && v + kUnroll * kThreads <= whole1) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) raw[u] = load(from + u * kThreads);
#pragma unroll
            for (int u = 0; u < kUnroll; u += kTogether) take(Some(), raw + u, v + tid + u * kThreads);
        } else {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int w = v + tid + u * kThreads;
                raw[u] = make_uint4(R::kNone, R::kNone, R::kNone, R::kNone);
                if (w >= whole0 && w < whole1) raw[u] = load(from + u * kThreads);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; u += kTogether)
                if (v + u * kThreads < whole1) take(Some(), raw + u, v + tid + u * kThreads);
        }
        if (++turn == per) {
            runs[run++][tid] = run_most;
            run_most = neg_inf();
            turn = 0;
        }
    }
    // the cut last piece belongs to the last run, which may be written already
    if (const int last = max(whole1, v0); last < v1 && last >= whole0 && tid == (last - v0) % kThreads) {
        const bool again = turn == 0 && run > 0 && (last - v0) / (kUnroll * kThreads * per) < run;
        if (again) run_most = runs[run - 1][tid];
        const uint4 raw = row.edge(last);
        take(One(), &raw, last);
        if (again) runs[run - 1][tid] = run_most;
    }
    for (; run * per < turns; ++run) {
        runs[run][tid] = run_most;
        run_most = neg_inf();
    }

    // ---- the block's sums
    float top = most;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
    top = s_top[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_top[w]);
    Sums sums = sums_now();
    sums.against(in_units(top));
    s_mine[tid] = make_float2(sums.s, sums.e);
    if (most == top) s_owner = tid;         // (used where there is one only)
    block_sums(sums, s_sums, warp, lane);
    if (tid == 0) s_block = make_float4(top, sums.s, sums.e, 0.f);

    // ---- the block's k largest values
    if (a.k > 0) {
        const uint32_t high = to_key(most);
        // piece v's values that are not below `least`, one bit each
        auto reach = [&](int v, uint32_t least, float (&x)[P]) {
            uint32_t left = 0;
            R::values(row.piece(v), x);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const uint32_t h = to_key(x[i]);
                if (h != 0 && h >= least) left |= 1u << i;
            }
            return left;
        };
        auto key_of = [&](float x, int v, int i) { return (Key)to_key(x) << 32 | (uint32_t)~(v * P + i - row.skip); };
        if (tid == 0) s_which = s_found = 0;
        if (warp == 0) best[lane] = 0;
        auto rows = reinterpret_cast<uint32_t(*)[32]>(lists);
        const uint32_t kth = merge_warps(sorted(high, lane), kWarps, rows, warp, lane);
        if (tid == a.k - 1) s_least = kth;
        __syncthreads();
        uint32_t least = s_least;       // 0: fewer than k threads hold any value
        if (high != 0 && high >= least)
            for (int r = 0; r * per < turns; ++r) {
                const uint32_t h = to_key(runs[r][tid]);
                if (h != 0 && h >= least) {
                    const int at = atomicAdd(&s_which, 1);      // (the order does not matter)
                    if (at < kQuickRuns) which[at] = r * kThreads + tid;
                }
            }
        __syncthreads();
        const int reached = s_which;
        bool quick = reached <= kQuickRuns;
        if (quick) {
            const int each = per * kUnroll;     // pieces of a run
            for (uint32_t i = tid; i < (uint32_t)(reached * each); i += kThreads) {       // (V <= 2^30: below 2^24)
                const int j = (int)(i / (uint32_t)each), at = which[j];
                const int v = v0 + at % kThreads + (at / kThreads * each + (int)i - j * each) * kThreads;
                if (v >= v1) continue;
                float x[P];
                const uint32_t left = reach(v, least, x);
                if (left)
#pragma unroll
                    for (int q = 0; q < P; ++q)
                        if (left >> q & 1u) {
                            const int to = atomicAdd(&s_found, 1);      // (nor here: keys differ)
                            if (to < kQuickKeys) found[to] = key_of(x[q], v, q);
                        }
            }
            __syncthreads();
            const int n = s_found;
            quick = n <= kQuickKeys;
            if (quick) {
                if (tid < n) {          // keys differ: a key's place is the number of those above it
                    const Key key = found[tid];
                    int place = 0;
#pragma unroll 4
                    for (int j = 0; j < n; ++j) place += found[j] > key;
                    if (place < 32) best[place] = key;
                }
            }
        }
        if (!quick) {
            // the first piece that holds the largest value is among those taken together
            if (high != 0)
                for (int u = 0; u < kTogether && place < v1; ++u, place += kThreads) {
                    const uint4 raw = row.piece(place);
                    if (R::template largest<1>(&raw) == most) break;
                }
            Key key = high ? (Key)high << 32 | (uint32_t)~place : 0;
            key = merge_warps(sorted(key, lane), kWarps, lists, warp, lane);
            if (warp == 0) best[lane] = key;
            __syncthreads();
            least = (uint32_t)(best[a.k - 1] >> 32);
            Key list = 0;
            for (int j = warp; j < a.k; j += kWarps) {
                if (best[j] == 0) break;
                const int mine = ((int)~(uint32_t)best[j] - v0) % kThreads + v0;      // that thread's first piece
                for (int v = mine + lane * kThreads; __any_sync(0xffffffffu, v < v1); v += 32 * kThreads) {
                    float x[P];
                    uint32_t left = v < v1 ? reach(v, least, x) : 0u;
                    while (__any_sync(0xffffffffu, left != 0)) {
                        Key cand = 0;
                        if (left) {
                            const int i = __ffs(left) - 1;
                            left &= left - 1;
                            float y = x[0];
#pragma unroll
                            for (int q = 1; q < P; ++q) y = i == q ? x[q] : y;
                            cand = key_of(y, v, i);
                        }
                        list = merged(list, sorted(cand, lane), lane);
                    }
                }
            }
            int count = 1;
            while (count < min(a.k, kWarps)) count <<= 1;
            list = merge_warps(list, count, lists, warp, lane);
            if (warp == 0) best[lane] = list;       // (merge_warps has synchronized since best was read)
        }
    }

    // ---- the row's, by the cluster's first block
    float4 all;
    Key theirs = 0;         // of the warp's block
    if (blocks > 1) {
        cluster_sync();
        if (rank == 0 && a.k > 0 && warp < (int)blocks) theirs = ld_cluster_u64(in_block(&best[lane], warp));
        float4 part[kMaxCluster];
        top = neg_inf();
#pragma unroll
        for (int b = 0; b < kMaxCluster; ++b)
            if (b < (int)blocks) {
                part[b] = ld_cluster_f32x4(in_block(&s_block, b));
                top = fmaxf(top, part[b].x);
            }
        all = make_float4(top, 0.f, 0.f, 0.f);
#pragma unroll
        for (int b = 0; b < kMaxCluster; ++b)
            if (b < (int)blocks) {
                Sums p{in_units(part[b].x), part[b].y, part[b].z};
                p.against(in_units(top));
                all.y += p.s;
                all.z += p.e;
            }
    } else {
        __syncthreads();
        all = s_block;
    }
    // Sums a second time (the same for all threads of the cluster). A reference too far away: with logits of +inf their
    // number is the sum; else both from differences. A row that one logit dominates: without that one, whose rounding
    // would cover the others (ln S = ln(1 + rest)); the thread that met it reads its pieces again, of the others' sums
    // nothing was lost.
    const bool infinite = all.x == pos_inf();
    const bool far = infinite || (all.x > neg_inf() && fabsf(in_units(all.x)) >= kFar);
    all.w = all.x > neg_inf() && !far ? fmaf(all.x, a.c, -in_units(all.x)) : 0.f;      // of the largest value, against the reference
    const bool sharp = !far && all.x > neg_inf() && all.y < 1.5f;
    if (far || sharp) {
        Sums again{0.f, 0.f, 0.f};
        int v = v0 + tid, step = kThreads;
        if (sharp) {
            const bool here = s_block.x == all.x;
            const float2 m = s_mine[tid];
            if (!here || tid != s_owner) {
                again = Sums{in_units(s_block.x), m.x, m.y};
                again.against(in_units(all.x));
                const float f = exp2_fast(-all.w);          // from the rounded reference to the largest value itself
                again.e = f * fmaf(-all.w, again.s, again.e);
                again.s *= f;
            }
            v = here ? v0 + s_owner + tid * kThreads : v1;
            step = kThreads * kThreads;
        }
        for (; v < v1; v += step) {
            float x[P];
            R::values(row.piece(v), x);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                float t = infinite ? (x[j] == pos_inf() ? 0.f : -200.f) : fmaxf((x[j] - all.x) * a.c, -200.f);
                if (sharp && x[j] == all.x) t = -200.f;
                const float p = exp2_fast(t);
                again.s += p;
                again.e = fmaf(p, t, again.e);
            }
        }
        block_sums(again, s_sums, warp, lane);
        if (tid == 0) s_again = make_float4(all.x, again.s, again.e, 0.f);
        if (blocks > 1) cluster_sync();
        else __syncthreads();
        all.y = all.z = 0.f;
        for (int b = 0; b < (int)blocks; ++b) {
            const float4 p = blocks > 1 ? ld_cluster_f32x4(in_block(&s_again, b)) : s_again;
            all.y += p.y;
            all.z += p.z;
        }
    }
    if (rank == 0) {
        const float over = sharp ? log1pf(all.y) : logf(all.y) - kLn2 * all.w;      // ln S
        auto log_p = [&](float x) {
            if (infinite) return x == pos_inf() ? -over : neg_inf();
            return x > neg_inf() ? fminf((x - all.x) * a.scale - over, 0.f) : neg_inf();
        };
        if (tid == 0) {
            if (a.logprob) a.logprob[t] = token >= 0 && token < a.V ? log_p(given) : 0.f;
            if (a.entropy) a.entropy[t] = sharp ? over - kLn2 * all.z / (1.f + all.y) : (all.y > 0.f ? fmaxf(logf(all.y) - kLn2 * all.z / all.y, 0.f) : 0.f);
        }
        if (a.k > 0) {
            if (blocks > 1) {
                const Key key = merge_warps(theirs, (int)blocks, lists, warp, lane);
                if (warp == 0) best[lane] = key;
            }
            if (tid < a.k) {
                const Key key = best[tid];
                const float x = from_key((uint32_t)(key >> 32));
                const bool any = key != 0 && (!infinite || x == pos_inf());
                a.top[t * a.k + tid] = any ? (int)~(uint32_t)key : -1;
                a.top_logprob[t * a.k + tid] = any ? log_p(x) : neg_inf();
            }
        }
    }
    if (blocks > 1) {       // no block leaves while the first reads its shared memory
        cluster_arrive();
        cluster_wait();
    }
}

template <int DT>
cudaError_t launch_dt(const Args& a, int T, cudaStream_t s) {
    const int pieces = (int)(((long long)a.V * (DT == DT_F32 ? 4 : 2) + 15) / 16);
    int blocks = 1;
    while (blocks < kMaxCluster && (long long)T * blocks < kTargetSms && pieces > 2 * blocks * kThreads) blocks *= 2;
    return launch_behind(logprobs_kernel<DT>, dim3((unsigned)T * blocks), dim3(kThreads), 0, (unsigned)blocks, s, a);
}

}  // namespace

cudaError_t launch_logprobs(int T, int V, const void* logits, int dtype, long long ld, float scale, const int32_t* token,
                            float* logprob, float* entropy, int k, int32_t* top, float* top_logprob, cudaStream_t s) {
    const float c = scale * kLog2e;
    const Args a{V, static_cast<const uint8_t*>(logits), ld * (long long)dt_size(dtype), scale, c < FLT_MAX ? c : FLT_MAX,
                 token, logprob, entropy, k, top, top_logprob};
    switch (dtype) {
        case DT_F32: return launch_dt<DT_F32>(a, T, s);
        case DT_F16: return launch_dt<DT_F16>(a, T, s);
        default: return launch_dt<DT_BF16>(a, T, s);
    }
}

}  // namespace qg
