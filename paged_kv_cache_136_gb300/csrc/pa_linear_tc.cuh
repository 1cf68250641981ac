// pa_linear_tc.cuh -- linear attention with a decay for each head over packed
// prompts, on the 5th-generation tensor cores (tcgen05, accumulators in tensor
// memory).
//
// Mathematics.  Tokens are taken in chunks of 128.  With b_i the sum of a chunk's
// log decays up to its token i, and S the state before the chunk,
//   o_i = e^(b_i) q_i S + sum_(j<=i) e^(b_i - b_j) (q_i . k_j) v_j
//   S'  = e^(b_last) S + sum_j k_j (e^(b_last - b_j) v_j)^T
// which is four products of 128 rows: Q K^T, P V, Q S and V'^T K.  An exponent is
// always a sum of the log decays between two tokens (between blocks of 32: rest of the
// column's block, blocks between, the row's block up to it), each factor at most 1 if
// decays are.  A difference of two sums from a common start would be off by 2^-24 of
// the larger one: weights by 2e-4 where half of a block's tokens forget.
//
// Precision.  P, S and V' are fp32 values that enter a product as a 16-bit part and
// the rounded remainder (two MMAs that share the other operand).  One part alone
// would add the error of a second output rounding, and 2^-9 to the states.  fp16
// operands are scaled by powers of two (P by row, V' by chunk, S as a whole), so that
// large scores or states do not leave fp16's range and small ones keep their bits:
// those down to 2^-17 of the largest all 22, smaller ones what lies above 2^-39 of it.
// The state itself stays in fp32 registers and is only added to by fp32 additions that
// round to nearest.
//
// Bounds.  A chunk of 128 x 128 takes 3.9 us (8000 cycles) with one query head a kv head
// and about 2.4 for each of more (5000), about twice its MMAs' time (64 and 40 of 64
// cycles each).  With one head the chain V' -> delta -> state -> operand -> Q S sets the
// pace, each step a wait for the one before, with more of them the rows' chain scores ->
// P -> P V -> output.  16 prompts of 256 to 2048 tokens, 32 heads, take 178 us in fp16;
// one of 131072, 64 heads and 8 kv heads, in bf16 1.37 ms, in which the MMAs run at 1.1
// PFLOP/s.  A chain's start (an SM's turnover, its first tiles and state, a first look at
// V) and its state's store take 8 us besides.
//
// A CTA walks one segment of one sequence for one kv head with all of its query
// heads.  Roles in a CTA of 640 threads:
//   warps 0-7    a row of the chunk and half of its columns per thread: P from the
//                scores, O scaled by e^(b_i) between its two products, the output
//                tile over the query tile that made it
//   warps 8-15   a value channel and half of the key channels (and tokens) per thread:
//                V' from the V tile, and the state (in registers), which goes to
//                shared memory as the operand of the next chunk's Q S
//   warp 16      a chunk's decay sums, and its tiles by TMA: K (2 slots) and Q and V (2
//                slots and 1, or with one query head 1 and 2)
//   warp 17      the MMAs: per query head O = Q S, O += P V, the next head's scores;
//                per chunk delta = V'^T K, behind the second head's Q S (the only one's)
//   warp 18      output tiles to global memory by TMA
//   warp 19      looks through V tiles: rows behind the sequence and values that are not
//                finite become zeros; with fp16 the largest magnitude
// Two threads share a row or a channel because one warp a scheduler is not enough to
// hide the latency of tensor memory and of fetching a role's instructions; the loops
// over blocks are rolled for the latter's sake.
// Tensor memory: the scores in columns 0-127, in each block of 32 columns P over them
// (16 columns of high parts, 16 of remainders); O at 128; delta at 256; V' behind.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "pa_internal.h"
#include "pa_linear.cuh"
#include "pa_ptx.cuh"

namespace pa {
namespace lin {

constexpr int kChunk = 128;        // tokens
constexpr int kTcThreads = 640;
constexpr int kProducerWarp = 16, kMmaWarp = 17, kStoreWarp = 18, kLookWarp = 19;
// Five warpgroups are launched with 96 registers a thread; the last one, whose warps
// issue copies and MMAs, hands some to the two that hold states: 2 * 128 + 2 * 96 + 32.
constexpr int kRegsLaunched = 96, kRegsFew = 32, kRegsMany = 128;
constexpr uint32_t kTmemCols = 512;
constexpr int kSms = 152;
// Named barriers: of all rows, of all channels, of the two warps that share 32 rows (4).
constexpr int kRowsBarrier = 1, kChannelsBarrier = 2, kPairBarrier = 3;
constexpr uint32_t kTmemO = 128, kTmemDelta = 256, kTmemV = 384;
constexpr int kRegion = kChunk * 128; // 128 token rows of 64 elements

template <typename T, int D>
struct Geo {
    // V' enters V'^T K in three parts with bf16, 2^-24 of its size: with two the states
    // would be off by 2.6e-6 (measured), with fp16's longer parts two reach 2^-22.
    static constexpr int kSplit = std::is_same<T, __half>::value ? 2 : 3;
    // Tensor memory has 128 columns for V': a ring of blocks of 32 tokens, which are made
    // while the MMAs take the ones before.
    static constexpr int kRing = 128 / (kSplit * 16);
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = kHalves * kRegion;      // a Q, K or V tile
    static constexpr int kStateRegion = D * 128;         // 64 key channels of all value channels
    static constexpr int kState = kHalves * kStateRegion;
    // Five tiles: K twice, then with one query head a kv head Q once and V twice, with
    // more of them Q twice and V once.
    static constexpr int kOffK = 0, kOffQ = 2 * kTile, kOffV = 4 * kTile, kOffS = 5 * kTile;
    static constexpr int kOffMisc = kOffS + 2 * kState;
};

// A chunk's decays, in log2 units where they are sums.
struct alignas(16) Decays { // read four floats at a time
    float each[kChunk];   // the token's own
    float rest[kChunk];   // 2^(sum behind this one to the block's end)
    float block[4];       // the blocks' sums
};

// What a CTA works on: a sequence (-1: nothing), one of its segments, its tokens, its
// states.  Then the first token (-1: nothing), state and head of what will follow on some
// SM when this is done.
struct Unit {
    int seq, segment, segments, first, tokens, src, dst;
    int next_first, next_src, next_head;
};

struct Misc {
    uint64_t k_full[2], k_empty[2], q_full[2], q_empty[2], v_full[2], v_empty[2];
    uint64_t dec_full[2], dec_empty[2];
    uint64_t s_full, p_full, o1_full, o_full, o_free, o_staged;
    uint64_t vok_full[2], st_full[2], ring_full[4], ring_empty[4], d_full, qs_done, drain;
    uint32_t hurt[2];        // whether a chunk had values that are not finite
    int value_exponent[2];   // fp16: V' is divided by 2^this
    Decays dec[2];
    float state_scale[2];    // what the state's operand was divided by
    uint32_t tmem_base;
    Unit unit;
    uint8_t first[2][128];   // by value channel: the chunk's first token whose value is not
                             // finite, or 128
    float warp_max[2][8];
};

template <typename T, int D> constexpr int tc_smem_bytes()
{
    // at least half of an SM's: two CTAs would wait for each other's tensor memory
    constexpr int n = Geo<T, D>::kOffMisc + (int)sizeof(Misc);
    return n > 120 * 1024 ? n : 120 * 1024;
}
static_assert(tc_smem_bytes<__half, 128>() <= 232448, "shared memory of an SM");

template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w);
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <typename T> __device__ __forceinline__ float value_of(uint16_t u);
template <> __device__ __forceinline__ float value_of<__half>(uint16_t u)
{
    return __half2float(__ushort_as_half(u));
}
template <> __device__ __forceinline__ float value_of<__nv_bfloat16>(uint16_t u)
{
    return __uint_as_float((uint32_t)u << 16);
}

template <typename T> struct Pair;
template <> struct Pair<__half> { using type = __half2; };
template <> struct Pair<__nv_bfloat16> { using type = __nv_bfloat162; };
__device__ __forceinline__ uint32_t bits_of(__half2 x) { return *reinterpret_cast<uint32_t *>(&x); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t *>(&x); }

// The larger magnitudes of two pairs; a NaN stays.
template <typename T>
__device__ __forceinline__ typename Pair<T>::type most_of_pairs(typename Pair<T>::type m, uint32_t x)
{
    return __hmax2_nan(m, __habs2(*reinterpret_cast<const typename Pair<T>::type *>(&x)));
}

// x less the two 16-bit values of `part`, by multiply-adds that take 16-bit factors: the
// parts are not unpacked first, which would be twice the work on a narrower pipe.
template <typename T> __device__ __forceinline__ float2 less(float2 x, uint32_t part);
template <> __device__ __forceinline__ float2 less<__half>(float2 x, uint32_t part)
{
    asm("{\n"
        "  .reg .b16 l, h, m;\n"
        "  mov.b32 {l, h}, %2;\n"
        "  mov.b16 m, 0xBC00;\n"
        "  fma.rn.f32.f16 %0, l, m, %0;\n"
        "  fma.rn.f32.f16 %1, h, m, %1;\n"
        "}\n"
        : "+f"(x.x), "+f"(x.y)
        : "r"(part));
    return x;
}
template <> __device__ __forceinline__ float2 less<__nv_bfloat16>(float2 x, uint32_t part)
{
    asm("{\n"
        "  .reg .b16 l, h, m;\n"
        "  mov.b32 {l, h}, %2;\n"
        "  mov.b16 m, 0xBF80;\n"
        "  fma.rn.f32.bf16 %0, l, m, %0;\n"
        "  fma.rn.f32.bf16 %1, h, m, %1;\n"
        "}\n"
        : "+f"(x.x), "+f"(x.y)
        : "r"(part));
    return x;
}

// Two values as N 16-bit parts, each the rounded remainder of those before it.
template <typename T, int N>
__device__ __forceinline__ void split(float2 x, uint32_t (&part)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        part[i] = pack2<T>(x.x, x.y);
        if (i + 1 < N)
            x = less<T>(x, part[i]);
    }
}
__device__ __forceinline__ float2 pair_of(const uint32_t *x)
{
    return make_float2(__uint_as_float(x[0]), __uint_as_float(x[1]));
}

// max(m, |x.x|, |x.y|); a NaN is passed over.
__device__ __forceinline__ float most_of(float m, float2 x)
{
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(x.x), "f"(x.y));
    return r;
}

// Exponent E that brings magnitudes up to m below 2^14 (or up to there): m 2^-E.
__device__ __forceinline__ int range_exponent(float m)
{
    return max((int)(__float_as_uint(m) >> 23 & 255) - 127 - 13, -40);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// A phase of a barrier, awaited by a whole converged warp, with a limit of tries (16 M of
// 20 cycles or more: a wait of these kernels takes microseconds).  One short loop that
// all lanes run: it stands at twenty places of a kernel whose roles have to fit the
// instruction cache together, and a loop of lane 0 alone leaves code behind it that is
// compiled for diverged lanes, MMA issue above all (16 prompts of 32 heads: 453 us with
// mbar_wait's unrolled tries in lane 0, 520 with a short loop there, 300 with this).
constexpr int kTries = 1 << 24;
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity)
{
    int left = kTries;
#pragma unroll 1
    while (!mbar_try_wait(bar, parity) && --left) {
    }
    return __all_sync(~0u, left > 0);
}

// A group of N threads goes on, or gives up, together: one of its warps waits on an
// mbarrier (a waiting warp asks again and again, and takes issue slots and fetches from
// those that work), another one on the next if there is one, all of them at named
// barrier `id`.
template <int N> __device__ __forceinline__ bool together(int id, bool ok)
{
    return !bar_sync_or(id, N, !ok);
}

// Where sequence s lies, and in how many segments; 0 if it is skipped.
__device__ __forceinline__ int segments_of(const LinearParams &p, int s, int &q0, int &len, bool tell)
{
    q0 = p.query_start_loc[s];
    const int q1 = p.query_start_loc[s + 1];
    len = q1 - q0;
    if (q0 < 0 || q1 > p.num_tokens || q1 < q0 || len > p.max_query_len) {
        if (tell)
            atomicOr(p.err, PA_DEVERR_SEQ_LEN_);
        return 0;
    }
    if (p.dst_states[s] < 0)
        return 0;
    return p.segment >= len ? 1 : (len - 1) / p.segment + 1;
}

// The sequence and segment of line y of the grid, by one warp: s < 0 past the end.
__device__ __forceinline__ void find_unit(const LinearParams &p, int y, int lane, bool tell, int &s,
                                          int &j, int &n)
{
    int before = 0;
    s = -1;
    for (int base = 0; base < p.num_seqs; base += 32) {
        int q0, len, mine = 0;
        if (base + lane < p.num_seqs)
            mine = segments_of(p, base + lane, q0, len, tell);
        int x = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(~0u, x, o);
            if (lane >= o)
                x += v;
        }
        const unsigned here = __ballot_sync(~0u, before + x > y);
        if (here) {
            const int l = __ffs(here) - 1;
            s = base + l;
            n = __shfl_sync(~0u, mine, l);
            j = y - before - (__shfl_sync(~0u, x, l) - n);
            // Sequences that overlap can be more than the lines there are: one that does
            // not fit is skipped as a whole, here and in the join.
            if (y - j + n > p.lines)
                s = -1;
            return;
        }
        before += __shfl_sync(~0u, x, 31);
    }
}

// kParts: the first pass over sequences of several segments.  It forms the state
// that each segment but the last one leaves, the first from the sequence's own
// state, the others from zero, and the segments' decays.  The last segment's line,
// which has no such state, takes a copy of the sequence's own: the second pass starts
// the first segment from there.  So that pass reads no state of a cut sequence, and
// its last segment can write the state at any time, src_states[s] = dst_states[s] or
// not.
template <typename T, int D, bool kParts>
__global__ void __launch_bounds__(kTcThreads, 1)
    linear_chunk_kernel(const __grid_constant__ CUtensorMap q_map,
                        const __grid_constant__ CUtensorMap k_map,
                        const __grid_constant__ CUtensorMap v_map,
                        const __grid_constant__ CUtensorMap out_map, const LinearParams p)
{
    using Gm = Geo<T, D>;
    constexpr int TB = Gm::kTile;
    constexpr int kSplit = Gm::kSplit;
    constexpr bool kHalf = std::is_same<T, __half>::value;
    constexpr int H = D / 2; // channels of a thread that has half of them
    constexpr uint32_t kFmt = kHalf ? 0u : 1u;
    constexpr uint32_t kIdescScores = idesc_f16_f32(kFmt, 0, 0, kChunk, kChunk);
    constexpr uint32_t kIdescState = idesc_f16_f32(kFmt, 0, 0, kChunk, D);             // Q S
    constexpr uint32_t kIdescValue = idesc_f16_f32(kFmt, 0, 1, kChunk, D);             // P V
    constexpr uint32_t kIdescDelta = idesc_f16_f32(kFmt, 0, 1, 128, D);    // V'^T K

    extern __shared__ __align__(1024) uint8_t smem[];
    Misc *m = reinterpret_cast<Misc *>(smem + Gm::kOffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int head = blockIdx.x, y = blockIdx.y;

    griddep_wait();
    if (warp == kMmaWarp) {
        tmem_alloc(&m->tmem_base, kTmemCols);
        tmem_relinquish();
    } else if (warp == 0) {
        // the last line is past every unit, so its search sees every sequence
        const bool tell = head == 0 && y == (int)gridDim.y - 1 && !kParts;
        int s = y, j = 0, n = 0, q0 = 0, len = -1, src = -1, dst = -1;
        const int64_t next = (int64_t)y * gridDim.x + head + kSms;
        const int next_y = (int)(next / gridDim.x);
        int next_first = -1, next_src = -1;
        if (p.segment != INT32_MAX) {
            find_unit(p, y, lane, tell, s, j, n);
            if (s >= 0) {
                q0 = p.query_start_loc[s], len = p.query_start_loc[s + 1] - q0;
                src = p.src_states[s], dst = p.dst_states[s];
            }
        } else if (p.num_seqs > 32) {
            // one segment each
            src = p.src_states[y], dst = p.dst_states[y];
            n = segments_of(p, y, q0, len, head == 0 && lane == 0);
            if (next_y < p.num_seqs)
                next_first = p.query_start_loc[next_y], next_src = p.src_states[next_y];
        } else {
            // Of up to 32 sequences line y is the y-th longest, so that the long ones start
            // first (8 of 32 to 4000 tokens, 32 heads: 133 us, in their own order 188; 16
            // ascending ones 272 and 315; 24 in any order with 8 kv heads 373 and 371).  More
            // keep their own order: 33 to 60 with 2 or 4 kv heads take the same in any, within
            // 1 %; 40 with 8 heads and 8 kv heads 180 descending, 235 ascending, 250 mixed.
            if (lane < p.num_seqs) {
                src = p.src_states[lane], dst = p.dst_states[lane];
                n = segments_of(p, lane, q0, len, head == 0 && lane == y);
            }
            int rank = 0;
            for (int i = 0; i < p.num_seqs; ++i) {
                const int other = __shfl_sync(~0u, len, i);
                rank += other > len || (other == len && i < lane);
            }
            const int behind = __ffs(__ballot_sync(~0u, lane < p.num_seqs && rank == next_y)) - 1;
            if (behind >= 0) {
                const int live = __shfl_sync(~0u, n, behind), at = __shfl_sync(~0u, q0, behind);
                next_first = live ? at : -1, next_src = __shfl_sync(~0u, src, behind);
            }
            s = __ffs(__ballot_sync(~0u, lane < p.num_seqs && rank == y)) - 1;
            n = __shfl_sync(~0u, n, s), q0 = __shfl_sync(~0u, q0, s), len = __shfl_sync(~0u, len, s);
            src = __shfl_sync(~0u, src, s), dst = __shfl_sync(~0u, dst, s);
        }
        if (lane == 0)
            m->unit = {n ? s : -1, j, n, q0, len, src, dst, next_first, next_src, (int)(next % gridDim.x)};
    }
    if (tid == 32) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m->k_full[i], 1);
            mbar_init(&m->k_empty[i], 1);
            mbar_init(&m->q_full[i], 1);
            mbar_init(&m->q_empty[i], 1);
            mbar_init(&m->vok_full[i], 1);
            mbar_init(&m->st_full[i], 8);
            mbar_init(&m->v_full[i], 1);
            mbar_init(&m->v_empty[i], 1);
            mbar_init(&m->dec_full[i], 1);
            mbar_init(&m->dec_empty[i], kParts ? 8 : 16);
        }
        mbar_init(&m->s_full, 1);
        mbar_init(&m->p_full, 8);
        mbar_init(&m->o1_full, 1);
        mbar_init(&m->o_full, 1);
        mbar_init(&m->o_free, 8);
        mbar_init(&m->o_staged, 8);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&m->ring_full[i], 8);
            mbar_init(&m->ring_empty[i], 1);
        }
        mbar_init(&m->d_full, 1);
        mbar_init(&m->qs_done, 1);
        mbar_init(&m->drain, 1);
        fence_barrier_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = m->tmem_base;
    const Unit unit = m->unit;
    const int j = unit.segment, nseg = unit.segments, src = unit.src, dst = unit.dst;
    if (unit.seq < 0 || (kParts && j == nseg - 1)) {
        if (kParts && unit.seq >= 0 && nseg > 1) {
            const int64_t one = (int64_t)D * D;
            float4 *const to = reinterpret_cast<float4 *>(p.parts + ((int64_t)y * p.num_kv_heads + head) * one);
            const float4 *const from =
                src >= 0 && src < p.num_states
                    ? reinterpret_cast<const float4 *>(p.states + ((int64_t)src * p.num_kv_heads + head) * one)
                    : nullptr;
            for (int i = tid; i < D * D / 4; i += kTcThreads)
                to[i] = from ? from[i] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (warp == kMmaWarp)
            tmem_dealloc(tmem, kTmemCols);
        return;
    }
    const int t0 = unit.first + (j ? j * p.segment : 0);
    const int len = min(unit.first + unit.tokens - t0, p.segment), n = (len + kChunk - 1) / kChunk;
    const int per = p.num_heads / p.num_kv_heads;
    const int total = kParts ? n : n * per; // (chunk, query head) pairs
    // With one query head a kv head (and without any, in the first pass) a chunk is short,
    // and its chain -- V', delta, state -- sets the pace: V is loaded a chunk ahead, into
    // what is the second Q slot otherwise, Q's slot is free after Q S, and the output
    // goes over the K tile.  With more of them two Q slots let a head's scores be formed
    // during the one before, and V has a chunk's time to arrive.
    const bool solo = kParts || per == 1;
    auto v_slot = [&](int c) { return solo ? c & 1 : 0; };
    auto v_phase = [&](int c) { return (uint32_t)(solo ? c >> 1 : c) & 1; };
    auto v_offset = [&](int c) { return Gm::kOffV - v_slot(c) * TB; };
    auto q_slot = [&](int it) { return solo ? 0 : it & 1; };
    auto q_phase = [&](int it) { return (uint32_t)(solo ? it : it >> 1) & 1; };
    const bool output_first = !kParts && solo && n == 1;
    // where a pair's output is staged
    auto out_offset = [&](int it) {
        return (solo && !output_first ? Gm::kOffK : Gm::kOffQ) + (it & 1) * TB;
    };
    if (tid == 0 && head == 0 && !kParts && (src >= p.num_states || dst >= p.num_states))
        atomicOr(p.err, PA_DEVERR_STATE_);

    if (warp >= kProducerWarp) {
        registers_down<kRegsFew>();
        if (warp == kProducerWarp) {
            // ============================================================ producer
            if (lane == 0) {
                prefetch_tensormap(&k_map);
                prefetch_tensormap(&v_map);
                if (!kParts)
                    prefetch_tensormap(&q_map);
            }
            auto load = [&](int off, const CUtensorMap *map, uint64_t *bar, int h, int t) {
                mbar_arrive_expect_tx(bar, (uint32_t)TB);
#pragma unroll
                for (int hf = 0; hf < Gm::kHalves; ++hf)
                    tma_load_3d(smem + off + hf * kRegion, map, bar, hf * 64, h, t);
            };
            const float *const log_decay = p.log_decay + head;
            // this lane's four tokens of chunk c
            auto read_decays = [&](int c, float (&g)[4]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = c * kChunk + lane * 4 + i;
                    g[i] = t < len ? log_decay[(int64_t)(t0 + t) * p.decay_stride] : 0.f;
                }
            };
            float g[4];
            bool ok = true;
            int loaded_k = 0, loaded_q = 0, loaded_v = 0;
            auto put_decays = [&](int c) {
                const int b = c & 1;
                if (c >= 2 && !warp_wait(&m->dec_empty[b], (uint32_t)((c >> 1) - 1) & 1))
                    return false;
                Decays &d = m->dec[b];
                float rest[4], sum = 0.f;
                // in log2 units; below 2^-149 is 0, and so many of them add up to a number
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    g[i] *= 1.4426950408889634f;
                    g[i] = g[i] < -150.f ? -150.f : g[i];
                    sum += g[i];
                }
                rest[3] = 0.f;
#pragma unroll
                for (int i = 2; i >= 0; --i)
                    rest[i] = rest[i + 1] + g[i + 1];
                float down = sum; // over the 8 lanes of a block
#pragma unroll
                for (int o = 1; o < 8; o *= 2) {
                    const float z = __shfl_down_sync(~0u, down, o, 8);
                    if ((lane & 7) + o < 8)
                        down += z;
                }
                float behind = __shfl_down_sync(~0u, down, 1, 8);
                behind = (lane & 7) < 7 ? behind : 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    d.each[lane * 4 + i] = g[i];
                    d.rest[lane * 4 + i] = exp2f(behind + rest[i]);
                }
                if ((lane & 7) == 0)
                    d.block[lane >> 3] = down;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&m->dec_full[b]);
                if (c + 1 < n)
                    read_decays(c + 1, g);
                return true;
            };
            auto load_k = [&](int c) {
                if (c >= 2 && !warp_wait(&m->k_empty[c & 1], (uint32_t)((c >> 1) - 1) & 1))
                    return false;
                if (lane == 0)
                    load(Gm::kOffK + (c & 1) * TB, &k_map, &m->k_full[c & 1], head, t0 + c * kChunk);
                ++loaded_k;
                return true;
            };
            auto load_q = [&](int c, int h) { // the pairs in turn
                const int it = loaded_q, b = q_slot(it), slots = solo ? 1 : 2;
                if (kParts)
                    return true;
                if (it >= slots && !warp_wait(&m->q_empty[b], q_phase(it - slots)))
                    return false;
                if (lane == 0)
                    load(Gm::kOffQ + b * TB, &q_map, &m->q_full[b], head * per + h, t0 + c * kChunk);
                ++loaded_q;
                return true;
            };
            auto load_v = [&](int c) {
                const int b = v_slot(c), slots = solo ? 2 : 1;
                if (c >= slots && !warp_wait(&m->v_empty[b], v_phase(c - slots)))
                    return false;
                if (lane == 0)
                    load(v_offset(c), &v_map, &m->v_full[b], head, t0 + c * kChunk);
                ++loaded_v;
                return true;
            };
            if (n > 0) {
                read_decays(0, g);
                ok = load_k(0) && load_q(0, 0) && load_v(0) && put_decays(0);
            }
            // in the order in which their places come free
#pragma unroll 1
            for (int c = 0; ok && c < n; ++c) {
                const bool more = c + 1 < n;
                if (solo && more)
                    ok = load_v(c + 1);
                if (more)
                    ok = ok && put_decays(c + 1);
#pragma unroll 1
                for (int h = 1; ok && h < per; ++h)
                    ok = load_q(c, h);
                if (ok && more)
                    ok = load_k(c + 1) && load_q(c + 1, 0) && (solo || load_v(c + 1));
            }
            // This chain's loads are under way: what will follow it starts with tiles and a
            // state that are in L2.  (All SMs' first loads at once take HBM 4 us: 32 prompts
            // of 100 tokens, 32 heads, 90 us without, 82 with.)
            if (!kParts && ok && lane == 0 && unit.next_first >= 0 && unit.next_first < p.num_tokens) {
                if (unit.next_src >= 0 && unit.next_src < p.num_states)
                    l2_prefetch(p.states + ((int64_t)unit.next_src * p.num_kv_heads + unit.next_head) * D * D,
                                D * D * 4);
#pragma unroll
                for (int hf = 0; hf < Gm::kHalves; ++hf) {
                    tma_prefetch_3d(&k_map, hf * 64, unit.next_head, unit.next_first);
                    tma_prefetch_3d(&v_map, hf * 64, unit.next_head, unit.next_first);
                    tma_prefetch_3d(&q_map, hf * 64, unit.next_head * per, unit.next_first);
                }
            }
            if (!ok) {
                // Given up: no tile may land in a later CTA's memory, so the last load on
                // each barrier is awaited, within the waits' own limit.
                if (lane == 0)
                    atomicOr(p.err, PA_DEVERR_TIMEOUT_);
                auto settle = [](uint64_t *bar, int loads) {
                    if (loads > 0)
                        warp_wait(bar, (uint32_t)(loads - 1) & 1);
                };
#pragma unroll 1
                for (int b = 0; b < 2; ++b) {
                    settle(&m->k_full[b], (loaded_k + 1 - b) >> 1);
                    settle(&m->q_full[b], solo ? (b ? 0 : loaded_q) : (loaded_q + 1 - b) >> 1);
                    settle(&m->v_full[b], solo ? (loaded_v + 1 - b) >> 1 : (b ? 0 : loaded_v));
                }
            }
        } else if (warp == kMmaWarp) {
            // ========================================================== MMA issuer
            const uint64_t k_desc = smem_desc_sw128(smem_addr(smem + Gm::kOffK), 16, 1024);
            const uint64_t kt_desc = smem_desc_sw128(smem_addr(smem + Gm::kOffK), kRegion, 1024);
            const uint64_t q_desc = smem_desc_sw128(smem_addr(smem + Gm::kOffQ), 16, 1024);
            const uint64_t s_desc = smem_desc_sw128(smem_addr(smem + Gm::kOffS), 16, 1024);
            auto slot = [](int b) { return (uint64_t)((uint32_t)(b * TB) >> 4); };
            // the scores of pair `it`, over the P that the last product has read
            auto scores = [&](int it, int c, bool first) {
                if (first && !warp_wait(&m->k_full[c & 1], (uint32_t)(c >> 1) & 1))
                    return false;
                if (!warp_wait(&m->q_full[q_slot(it)], q_phase(it)))
                    return false;
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint64_t qd = q_desc + slot(q_slot(it)), kd = k_desc + slot(c & 1);
#pragma unroll 1
                    for (uint32_t kk = 0; kk < D / 16; ++kk) {
                        const uint64_t o = ((kk >> 2) * kRegion + (kk & 3) * 32) >> 4;
                        umma_f16(tmem, qd + o, kd + o, kIdescScores, kk);
                    }
                    umma_commit(&m->s_full);
                }
                __syncwarp();
                return true;
            };
            // delta = V'^T K, block after block of V', the last tokens' first
            auto delta = [&](int c) {
#pragma unroll 1
                for (uint32_t k = 0; k < 4; ++k) {
                    const uint32_t block = (uint32_t)c * 4 + k, at = block % Gm::kRing;
                    if (!warp_wait(&m->ring_full[at], (block / Gm::kRing) & 1))
                        return false;
                    tc_fence_after_sync();
                    if (elect_one()) {
                        const uint64_t kd = kt_desc + slot(c & 1) + (3 - k) * (2 * 2048 >> 4);
                        const uint32_t a = tmem + kTmemV + at * (kSplit * 16);
#pragma unroll 1
                        for (uint32_t kk = 0; kk < 2; ++kk)
#pragma unroll
                            for (uint32_t part = 0; part < kSplit; ++part)
                                umma_f16_tmem_a(tmem + kTmemDelta, a + part * 16 + kk * 8,
                                                kd + kk * (2048 >> 4), kIdescDelta, k + kk + part);
                        umma_commit(&m->ring_empty[at]);
                        if (k == 3)
                            umma_commit(&m->d_full);
                    }
                    __syncwarp();
                }
                return true;
            };
            // With several query heads V arrives late in the first one's time.  Nothing but
            // its store waits for the state of an only chunk: its output goes first.
            const int delta_head = solo ? 0 : 1;
            bool ok = n == 0 || kParts || scores(0, 0, true);
            for (int it = 0, c = 0, h = 0; ok && it < total; ++it) {
                const bool last = kParts || h == per - 1;
                const int next = last ? c + 1 : c;
                if (kParts)
                    ok = warp_wait(&m->k_full[c & 1], (uint32_t)(c >> 1) & 1);
                if (!kParts) {
                    // O = Q S, both parts
                    if (ok && h == 0)
                        ok = warp_wait(&m->st_full[c & 1], (uint32_t)(c >> 1) & 1);
                    if (ok && it > 0)
                        ok = warp_wait(&m->o_free, (uint32_t)(it - 1) & 1);
                    if (!ok)
                        break;
                    tc_fence_after_sync();
                    if (elect_one()) {
                        const uint64_t qd = q_desc + slot(q_slot(it));
#pragma unroll 1
                        for (uint32_t kk = 0; kk < D / 16; ++kk) {
                            const uint64_t o = ((kk >> 2) * kRegion + (kk & 3) * 32) >> 4;
                            const uint64_t so = ((kk >> 2) * Gm::kStateRegion + (kk & 3) * 32) >> 4;
                            umma_f16(tmem + kTmemO, qd + o, s_desc + so, kIdescState, kk);
                            umma_f16(tmem + kTmemO, qd + o, s_desc + (Gm::kState >> 4) + so,
                                     kIdescState, 1u);
                        }
                        umma_commit(&m->o1_full);
                        if (last)
                            umma_commit(&m->qs_done);
                        if (solo)
                            umma_commit(&m->q_empty[0]);
                    }
                    __syncwarp();
                }
                if (kParts || (h == delta_head && !output_first))
                    ok = ok && delta(c);
                if (!kParts) {
                    ok = ok && warp_wait(&m->p_full, (uint32_t)it & 1);
                    if (ok && h == 0)
                        ok = warp_wait(&m->vok_full[c & 1], (uint32_t)(c >> 1) & 1);
                    if (!ok)
                        break;
                    tc_fence_after_sync();
                    if (elect_one()) { // O += P V, both parts
                        const uint64_t vd0 =
                            smem_desc_sw128(smem_addr(smem + v_offset(c)), kRegion, 1024);
#pragma unroll 1
                        for (uint32_t kk = 0; kk < kChunk / 16; ++kk) {
                            const uint64_t vd = vd0 + kk * (2048 >> 4);
                            const uint32_t pa = tmem + (kk >> 1) * 32 + (kk & 1) * 8;
                            umma_f16_tmem_a(tmem + kTmemO, pa, vd, kIdescValue, 1u);
                            umma_f16_tmem_a(tmem + kTmemO, pa + 16, vd, kIdescValue, 1u);
                        }
                        umma_commit(&m->o_full);
                        if (last) // V' was made before delta (no V follows an only one)
                            umma_commit(&m->v_empty[v_slot(c)]);
                    }
                    __syncwarp();
                    if (output_first)
                        ok = delta(c);
                    if (it + 1 < total)
                        ok = scores(it + 1, next, last);
                }
                if (last && elect_one()) {
                    if (kParts)
                        umma_commit(&m->v_empty[v_slot(c)]);
                    if (kParts || !solo) // else free with the output's store
                        umma_commit(&m->k_empty[c & 1]);
                }
                __syncwarp();
                c = next;
                h = last ? 0 : h + 1;
            }
            if (!ok && lane == 0)
                atomicOr(p.err, PA_DEVERR_TIMEOUT_);
            if (elect_one())
                umma_commit(&m->drain);
            __syncwarp();
            warp_wait(&m->drain, 0);
        } else if (warp == kStoreWarp && !kParts) {
            // ============================================================== outputs
            bool ok = true;
            for (int it = 0, c = 0, h = 0; ok && it < total; ++it) {
                if (!(ok = warp_wait(&m->o_staged, (uint32_t)it & 1)))
                    break;
                if (lane == 0) {
                    if (len - c * kChunk >= kChunk) { // a tail's rows were written one by one
#pragma unroll
                        for (int hf = 0; hf < Gm::kHalves; ++hf)
                            tma_store_3d(&out_map, smem + out_offset(it) + hf * kRegion, hf * 64,
                                         head * per + h, t0 + c * kChunk);
                        bulk_commit();
                        bulk_wait_read();
                    }
                    mbar_arrive(solo ? &m->k_empty[it & 1] : &m->q_empty[it & 1]);
                }
                __syncwarp();
                if (++h == per)
                    h = 0, ++c;
            }
            if (lane == 0) {
                bulk_wait();
                if (!ok)
                    atomicOr(p.err, PA_DEVERR_TIMEOUT_);
            }
        } else if (warp == kLookWarp) {
            // ======================================================== a look at V
            bool ok = true;
#pragma unroll 1
            for (int c = 0; c < n; ++c) {
                const int b = c & 1, live = min(kChunk, len - c * kChunk);
                uint8_t *const v = smem + v_offset(c);
                ok = warp_wait(&m->v_full[v_slot(c)], v_phase(c)) &&
                     // everyone is through with chunk c - 2, whose `first` is written over
                     warp_wait(&m->dec_full[b], (uint32_t)(c >> 1) & 1) &&
                     (live == kChunk || warp_wait(&m->k_full[b], (uint32_t)(c >> 1) & 1));
                if (!ok)
                    break;
                // the tiles' rows behind the sequence are a neighbour's: zeros
#pragma unroll 1
                for (int i = live * 8 + lane; i < kChunk * 8; i += 32)
#pragma unroll
                    for (int hf = 0; hf < Gm::kHalves; ++hf) {
                        *reinterpret_cast<uint4 *>(v + hf * kRegion + i * 16) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(smem + Gm::kOffK + b * TB + hf * kRegion + i * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                __syncwarp();
                // The largest magnitude, of both halves of four words; NaN stays.
                typename Pair<T>::type most2[4] = {};
#pragma unroll 4
                for (int i = 0; i < TB / 512; ++i) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(v + lane * 16 + i * 512);
                    most2[0] = most_of_pairs<T>(most2[0], x.x);
                    most2[1] = most_of_pairs<T>(most2[1], x.y);
                    most2[2] = most_of_pairs<T>(most2[2], x.z);
                    most2[3] = most_of_pairs<T>(most2[3], x.w);
                }
                const float2 top = unpack2<T>(bits_of(__hmax2_nan(__hmax2_nan(most2[0], most2[1]),
                                                                  __hmax2_nan(most2[2], most2[3]))));
                const bool hurt = __any_sync(~0u, !(top.x < INFINITY && top.y < INFINITY));
                float most = fmaxf(top.x, top.y);
                if (hurt) {
                    // What is not finite is taken out of the tile: in P V it would reach the
                    // rows before it as 0 * NaN.  `first` is where a channel is lost from.
                    most = 0.f;
#pragma unroll 1
                    for (int ch = lane; ch < D; ch += 32) {
                        int first = 128;
#pragma unroll 1
                        for (int t = kChunk - 1; t >= 0; --t) {
                            uint16_t *const at = reinterpret_cast<uint16_t *>(
                                v + (ch / 64) * kRegion + t * 128 + (((ch % 64) / 8 ^ (t & 7)) * 16) +
                                (ch % 8) * 2);
                            const float x = fabsf(value_of<T>(*at));
                            if (!(x < INFINITY)) {
                                first = t;
                                *at = 0;
                            } else {
                                most = fmaxf(most, x);
                            }
                        }
                        m->first[b][ch] = (uint8_t)first;
                    }
                }
                const unsigned largest = __reduce_max_sync(~0u, __float_as_uint(most));
                if (lane == 0) {
                    m->hurt[b] = hurt;
                    m->value_exponent[b] = range_exponent(__uint_as_float(largest));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&m->vok_full[b]);
            }
            if (!ok && lane == 0)
                atomicOr(p.err, PA_DEVERR_TIMEOUT_);
        }
    } else if (warp < 8) {
        // ===================================================== rows: P and outputs
        const int row = tid & 127, blk = warp & 3, half = warp >> 2;
        const uint32_t lane_base = (uint32_t)(blk * 32) << 16;
        const uint32_t s_addr = tmem + lane_base;
        const uint32_t o_addr = tmem + lane_base + kTmemO + (uint32_t)(half * H);
        // this thread's column blocks: 0 and 3, or 1 and 2, which is as even as the
        // triangle allows
        const int block[2] = {half, 3 - half};
        bool ok = true;
        float inter = 0.f, f[2] = {0.f, 0.f};
        float after[4] = {}; // sums behind each 8 tokens of the row's block, up to the row
        for (int it = 0; !kParts && it < total; ++it) {
            const int c = it / per, h = it - c * per;
            const Decays &d = m->dec[c & 1];
            const int live = min(kChunk, len - c * kChunk);
            if (h == 0) { // there before the scores
                ok = warp_wait(&m->dec_full[c & 1], (uint32_t)(c >> 1) & 1);
                // decays from the end of a column block to this row, and from the
                // chunk's beginning
                float sum = d.each[row]; // of the row's 8 tokens, up to it
#pragma unroll
                for (int o = 1; o < 8; o *= 2) {
                    const float x = __shfl_up_sync(~0u, sum, o, 8);
                    sum += (lane & 7) >= o ? x : 0.f;
                }
                const float own = sum;
#pragma unroll
                for (int k = 2; k >= 0; --k) { // and of those before, in its block
                    const float of8 = __shfl_sync(~0u, own, k * 8 + 7);
                    after[k] = k < lane / 8 ? sum : 0.f;
                    sum += k < lane / 8 ? of8 : 0.f;
                }
                f[0] = f[1] = 0.f;
#pragma unroll
                for (int k = 3; k >= 0; --k)
                    if (k < blk) {
                        if (k == block[0])
                            f[0] = exp2f(sum) * p.scale;
                        if (k == block[1])
                            f[1] = exp2f(sum) * p.scale;
                        sum += d.block[k];
                    }
                inter = exp2f(sum) * p.scale;
            }
            if (warp == 0)
                ok = ok && warp_wait(&m->s_full, (uint32_t)it & 1);
            if (!(ok = together<256>(kRowsBarrier, ok)))
                break;
            tc_fence_after_sync();
            float down = 1.f, up = 1.f; // 2^-E, 2^E
            if constexpr (kHalf) {
                float most = 0.f; // of the whole row, by both of its threads
#pragma unroll 1
                for (int b = 0; b <= blk; ++b) {
                    uint32_t sv[32];
                    tmem_ld32_nowait(s_addr + (uint32_t)(b * 32), sv);
                    tmem_wait_ld();
                    if (b == blk)
#pragma unroll
                        for (int i = 1; i < 32; ++i)
                            sv[i] = i <= lane ? sv[i] : 0;
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        most = most_of(most, pair_of(sv + i));
                }
                const int e = range_exponent(most * fabsf(p.scale));
                down = power_of_two(-e);
                up = power_of_two(e);
                // P goes over the scores: both threads have seen all of them
                bar_sync(kPairBarrier + blk, 64);
            }
#pragma unroll 1
            for (int z = 0; z < 2; ++z) {
                const int b = z ? 3 - half : half;
                const uint32_t at = s_addr + (uint32_t)(b * 32);
                uint32_t hi[16], lo[16];
                auto put = [&](int i, float2 x) {
                    uint32_t part[2];
                    split<T, 2>(x, part);
                    hi[i] = part[0], lo[i] = part[1];
                };
                if (b > blk) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        hi[i] = lo[i] = 0;
                } else {
                    uint32_t sv[32];
                    tmem_ld32_nowait(at, sv);
                    tmem_wait_ld();
                    if (b < blk) {
                        const float fb = (z ? f[1] : f[0]) * down;
                        const float2 fb2 = make_float2(fb, fb);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 r = *reinterpret_cast<const float4 *>(&d.rest[b * 32 + i * 4]);
                            put(2 * i, __fmul2_rn(pair_of(sv + i * 4), __fmul2_rn(make_float2(r.x, r.y), fb2)));
                            put(2 * i + 1, __fmul2_rn(pair_of(sv + i * 4 + 2),
                                                      __fmul2_rn(make_float2(r.z, r.w), fb2)));
                        }
                    } else {
                        const float2 fb2 = make_float2(p.scale * down, p.scale * down);
                        // from this row back, 8 columns at a time: the sum of what lies
                        // behind each (16 prompts of 32 heads in fp16 178 us; one chain of
                        // 32 182; differences of sums from the block's start 179)
                        float sum = 0.f;
#pragma unroll
                        for (int i = 15; i >= 0; --i) {
                            if (i % 4 == 3)
                                sum = after[i / 4];
                            const float2 g = *reinterpret_cast<const float2 *>(&d.each[b * 32 + i * 2]);
                            float2 w;
                            w.y = ex2(sum);
                            sum += 2 * i < lane ? g.y : 0.f;
                            w.x = ex2(sum);
                            sum += 2 * i <= lane ? g.x : 0.f;
                            const float2 x = __fmul2_rn(pair_of(sv + i * 2), __fmul2_rn(w, fb2));
                            put(i, make_float2(2 * i <= lane ? x.x : 0.f, 2 * i < lane ? x.y : 0.f));
                        }
                    }
                }
                tmem_st16(at, hi);
                tmem_st16(at + 16, lo);
            }
            if (warp == 0)
                ok = warp_wait(&m->o1_full, (uint32_t)it & 1);
            else if (h == 0 && warp == 1)
                ok = warp_wait(&m->st_full[c & 1], (uint32_t)(c >> 1) & 1);
            else if (h == 0 && warp == 2)
                ok = warp_wait(&m->vok_full[c & 1], (uint32_t)(c >> 1) & 1);
            if (!(ok = together<256>(kRowsBarrier, ok)))
                break;
            if (kHalf && h == 0)
                inter *= m->state_scale[c & 1];
            tc_fence_after_sync();
            const float2 of = make_float2(inter * down, inter * down);
#pragma unroll 1
            for (int b = 0; b < H / 32; ++b) {
                uint32_t o[32];
                tmem_ld32_nowait(o_addr + (uint32_t)(b * 32), o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float2 x = __fmul2_rn(pair_of(o + i), of);
                    o[i] = __float_as_uint(x.x), o[i + 1] = __float_as_uint(x.y);
                }
                tmem_st32(o_addr + (uint32_t)(b * 32), o);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&m->p_full);
            if (warp == 0)
                ok = warp_wait(&m->o_full, (uint32_t)it & 1);
            if (!(ok = together<256>(kRowsBarrier, ok)))
                break;
            tc_fence_after_sync();
            const bool hurt = m->hurt[c & 1] != 0;
            uint8_t *const tile = smem + out_offset(it) + (half * H / 64) * kRegion + row * 128;
            T *const out = static_cast<T *>(p.out) + half * H +
                           ((int64_t)(t0 + c * kChunk + row) * p.num_heads + head * per + h) * D;
#pragma unroll 1
            for (int b = 0; b < H / 32; ++b) {
                uint32_t o[32];
                tmem_ld32_nowait(o_addr + (uint32_t)(b * 32), o);
                tmem_wait_ld();
                if (hurt) {
                    // A value that is not finite was taken out of the product, where it
                    // would have reached the rows before it as 0 * NaN.
                    const uint8_t *const first = &m->first[c & 1][half * H + b * 32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (first[i] <= row)
                            o[i] = 0x7FFFFFFFu;
                }
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float2 x = pair_of(o + 2 * i);
                    if constexpr (kHalf)
                        x = __fmul2_rn(x, make_float2(up, up));
                    w[i] = pack2<T>(x.x, x.y);
                }
                if (live == kChunk) {
                    const int piece = (half * H % 64) / 8 + b * 4;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4 *>(tile + ((piece + i) ^ (row & 7)) * 16) =
                            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                } else if (row < live) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        reinterpret_cast<uint4 *>(out)[b * 4 + i] =
                            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                }
            }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&m->o_free);
                mbar_arrive(&m->o_staged);
                if (h == per - 1)
                    mbar_arrive(&m->dec_empty[c & 1]);
            }
        }
        if (!ok && lane == 0)
            atomicOr(p.err, PA_DEVERR_TIMEOUT_);
    } else {
        // ================================================= value channels: the state
        registers_up<kRegsMany>();
        const int wg = warp & 3, ch = tid & 127, half = (warp - 8) >> 2;
        const uint32_t lane_base = (uint32_t)(wg * 32) << 16;
        const bool mine = ch < D;
        const int64_t one = (int64_t)D * D, at0 = (int64_t)half * H * D + ch;
        float S[H]; // key channels from half * H on
        {
            const float *from = nullptr;
            if (!kParts && nseg > 1) // behind the segment before, or the sequence's own
                from = p.parts + ((int64_t)(j ? y - 1 : y + nseg - 1) * p.num_kv_heads + head) * one + at0;
            else if (j == 0 && src >= 0 && src < p.num_states)
                from = p.states + ((int64_t)src * p.num_kv_heads + head) * one + at0;
#pragma unroll
            for (int k = 0; k < H; ++k)
                S[k] = mine && from ? from[(int64_t)k * D] : 0.f;
        }
        // The state as the operand of Q S: row = value channel, 64 key channels a
        // region, 16-byte pieces in the 128-byte swizzle.  False where a thread of the
        // group has given up.
        auto put_state = [&](int c, bool ok) {
            float down = 1.f;
            if constexpr (kHalf) {
                float most = 0.f;
#pragma unroll
                for (int k = 0; k < H; k += 2)
                    most = most_of(most, make_float2(S[k], S[k + 1]));
                if (most == INFINITY) { // the largest that is finite, then
                    most = 0.f;
#pragma unroll
                    for (int k = 0; k < H; ++k)
                        most = fmaxf(most, fabsf(S[k]) < INFINITY ? fabsf(S[k]) : 0.f);
                }
                const unsigned top = __reduce_max_sync(~0u, __float_as_uint(most));
                if (lane == 0)
                    m->warp_max[c & 1][warp - 8] = __uint_as_float(top);
                if (!together<256>(kChannelsBarrier, ok))
                    return false;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    most = fmaxf(most, m->warp_max[c & 1][i]);
                const int e = range_exponent(most);
                down = power_of_two(-e);
                if (tid == 256)
                    m->state_scale[c & 1] = power_of_two(e);
            } else if (!ok) {
                return false;
            }
            if (mine) {
                uint8_t *const at = smem + Gm::kOffS + ch * 128 + (half * H / 64) * Gm::kStateRegion;
#pragma unroll
                for (int k = 0; k < H; k += 8) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2 x = make_float2(S[k + 2 * i], S[k + 2 * i + 1]);
                        if constexpr (kHalf)
                            x = __fmul2_rn(x, make_float2(down, down));
                        uint32_t part[2];
                        split<T, 2>(x, part);
                        hi[i] = part[0], lo[i] = part[1];
                    }
                    const int off = (((half * H % 64) / 8 + k / 8) ^ (ch & 7)) * 16;
                    *reinterpret_cast<uint4 *>(at + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(at + Gm::kState + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&m->st_full[c & 1]);
            return true;
        };
        float decay_log2 = 0.f; // of the whole segment
        bool ok = true;         // of this warp, until the next barrier
#pragma unroll 1
        for (int c = 0; c < n; ++c) {
            const int b = c & 1;
            const Decays &d = m->dec[b];
            // Without other heads' products between, one wait serves a whole round (below).
            if (!kParts) {
                if (!solo && c > 0) {
                    if (warp == 8)
                        ok = ok && warp_wait(&m->qs_done, (uint32_t)(c - 1) & 1);
                    ok = together<256>(kChannelsBarrier, ok);
                }
                ok = put_state(c, ok);
            }
            if (!solo || c == 0) {
                if (warp == 8)
                    ok = ok && warp_wait(&m->vok_full[b], (uint32_t)(c >> 1) & 1);
                else if (warp == 9)
                    ok = ok && warp_wait(&m->dec_full[b], (uint32_t)(c >> 1) & 1);
                ok = together<256>(kChannelsBarrier, ok);
            }
            if (!ok)
                break;
            const bool hurt = mine && m->hurt[b] && m->first[b][ch] < 128;
            float scale = 1.f, back = 1.f;
            if constexpr (kHalf) {
                scale = power_of_two(-m->value_exponent[b]);
                back = power_of_two(m->value_exponent[b]);
            }
            // V', decayed to the chunk's end, from the last block on: of each block of 32
            // tokens this warp has 16 channels.  Transposed 8x8 matrices give a lane two
            // tokens of a channel, as the operand in tensor memory wants them.
            const uint32_t tile = smem_addr(smem + v_offset(c) + (wg / 2) * kRegion) +
                                  (uint32_t)(((lane >> 4) * 8 + (lane & 7)) * 128 +
                                             ((((wg & 1) * 4 + half * 2 + (lane >> 3 & 1)) ^ (lane & 7)) * 16));
            const float4 sums = *reinterpret_cast<const float4 *>(d.block);
            const float behind[3] = {sums.w, sums.w + sums.z, sums.w + sums.z + sums.y};
            const float factor[3] = {exp2f(behind[0]), exp2f(behind[1]), exp2f(behind[2])};
            // a block is handed on while the next one is worked out
            auto hand_on = [&](int i) {
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&m->ring_full[((uint32_t)c * 4 + i) % Gm::kRing]);
            };
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const uint32_t block = (uint32_t)c * 4 + i, at = block % Gm::kRing;
                const int k = 3 - i;
                uint32_t part[kSplit][8];
                if (mine) {
                    const float f = i == 0 ? 1.f : i == 1 ? factor[0] : i == 2 ? factor[1] : factor[2];
                    const float2 f2 = make_float2(f, f);
                    uint32_t x[2][4];
                    ldmatrix_x4_trans(x[0], tile + (uint32_t)(k * 4096));
                    ldmatrix_x4_trans(x[1], tile + (uint32_t)(k * 4096 + 2048));
#pragma unroll
                    for (int z = 0; z < 8; ++z) {
                        const float2 w = __fmul2_rn(
                            *reinterpret_cast<const float2 *>(&d.rest[k * 32 + (z >> 1) * 8 + (lane & 3) * 2]), f2);
                        float2 v = __fmul2_rn(unpack2<T>(x[z >> 2][z & 3]), w);
                        if constexpr (kHalf)
                            v = __fmul2_rn(v, make_float2(scale, scale));
                        uint32_t y[kSplit];
                        split<T, kSplit>(v, y);
#pragma unroll
                        for (int q = 0; q < kSplit; ++q)
                            part[q][z] = y[q];
                    }
                }
                if (i > 0)
                    hand_on(i - 1);
                // the chunk before is through: its delta has been read
                if (ok && i >= Gm::kRing)
                    ok = warp_wait(&m->ring_empty[at], (block / Gm::kRing - 1) & 1);
                if (mine) {
#pragma unroll
                    for (int q = 0; q < kSplit; ++q)
                        tmem_st_16x128b_x4(tmem + lane_base + ((uint32_t)(half * 16) << 16) + kTmemV +
                                               at * (kSplit * 16) + (uint32_t)(q * 16), part[q]);
                }
            }
            hand_on(3);
            if (lane == 0)
                mbar_arrive(&m->dec_empty[b]);
            const float sum = behind[2] + sums.x;
            const float decay = exp2f(sum);
            decay_log2 += sum;
            if (warp == 8) {
                ok = ok && warp_wait(&m->d_full, (uint32_t)c & 1);
            } else if (solo && c + 1 < n) { // and what the next round wants
                if (warp == 9)
                    ok = ok && warp_wait(&m->vok_full[b ^ 1], (uint32_t)((c + 1) >> 1) & 1);
                else if (warp == 10)
                    ok = ok && warp_wait(&m->dec_full[b ^ 1], (uint32_t)((c + 1) >> 1) & 1);
                else if (warp == 11 && !kParts)
                    ok = ok && warp_wait(&m->qs_done, (uint32_t)c & 1);
            }
            ok = together<256>(kChannelsBarrier, ok);
            tc_fence_after_sync();
            if (ok && mine) {
                const uint32_t from = tmem + lane_base + kTmemDelta + (uint32_t)(half * H);
#pragma unroll
                for (int k = 0; k < H / 32; ++k) {
                    uint32_t x[32];
                    tmem_ld32_nowait(from + (uint32_t)(k * 32), x);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float2 add = pair_of(x + i);
                        if constexpr (kHalf)
                            add = __fmul2_rn(add, make_float2(back, back));
                        const float2 to = __ffma2_rn(make_float2(S[k * 32 + i], S[k * 32 + i + 1]),
                                                     make_float2(decay, decay), add);
                        S[k * 32 + i] = to.x, S[k * 32 + i + 1] = to.y;
                    }
                }
                if (hurt)
#pragma unroll
                    for (int k = 0; k < H; ++k)
                        S[k] = __uint_as_float(0x7FFFFFFFu);
            }
            tc_fence_before_sync();
        }
        if (!ok && lane == 0)
            atomicOr(p.err, PA_DEVERR_TIMEOUT_);
        if (ok && mine) {
            float *to = nullptr;
            if (kParts)
                to = p.parts + ((int64_t)y * p.num_kv_heads + head) * one + at0;
            else if (j == nseg - 1 && dst < p.num_states)
                to = p.states + ((int64_t)dst * p.num_kv_heads + head) * one + at0;
            if (to)
#pragma unroll
                for (int k = 0; k < H; ++k)
                    to[(int64_t)k * D] = S[k];
            if (kParts && tid == 256)
                p.part_decay[(int64_t)y * p.num_kv_heads + head] = exp2f(decay_log2);
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Between the passes: the state behind segment j is the one behind segment j - 1,
// decayed, plus what segment j adds.  A thread has one float4 of a state.
template <int D>
__global__ void __launch_bounds__(256) linear_join_kernel(const LinearParams p)
{
    __shared__ long long first;
    __shared__ int count;
    griddep_wait();
    const int tid = threadIdx.x, head = blockIdx.y, s = blockIdx.z;
    if (tid < 32) {
        int q0, len, n = segments_of(p, s, q0, len, false);
        long long before = 0;
        for (int i = tid; n > 2 && i < s; i += 32) {
            int a, l;
            before += segments_of(p, i, a, l, false);
        }
#pragma unroll
        for (int o = 16; o; o /= 2)
            before += __shfl_xor_sync(~0u, before, o);
        if (tid == 0) // skipped as in find_unit
            first = before, count = before + n <= p.lines ? n : 0;
    }
    __syncthreads();
    if (count < 3)
        return;
    const int64_t step = (int64_t)p.num_kv_heads * D * D;
    float4 *at = reinterpret_cast<float4 *>(p.parts + first * step + (int64_t)head * D * D) +
                 blockIdx.x * 256 + tid;
    const float *decay = p.part_decay + (int64_t)first * p.num_kv_heads + head;
    float4 S = *at;
    // the last segment's line has the sequence's own state
    constexpr int kAhead = 8;
    for (int j = 1; j < count - 1; j += kAhead) {
        float4 x[kAhead];
        float f[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (j + k < count - 1) {
                x[k] = at[(int64_t)(j + k) * (step / 4)];
                f[k] = decay[(int64_t)(j + k) * p.num_kv_heads];
            }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (j + k < count - 1) {
                S.x = fmaf(f[k], S.x, x[k].x);
                S.y = fmaf(f[k], S.y, x[k].y);
                S.z = fmaf(f[k], S.z, x[k].z);
                S.w = fmaf(f[k], S.w, x[k].w);
                at[(int64_t)(j + k) * (step / 4)] = S;
            }
    }
}

} // namespace lin
} // namespace pa
