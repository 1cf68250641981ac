// pa_linear_tc.cuh -- linear attention with a decay for each head over packed
// prompts, on the 5th-generation tensor cores (tcgen05, accumulators in tensor
// memory).
//
// Mathematics.  Tokens are taken in chunks of 128.  With b_i the sum of a chunk's
// log decays up to its token i, and S the state before the chunk,
//   o_i = e^(b_i) q_i S + sum_(j<=i) e^(b_i - b_j) (q_i . k_j) v_j
//   S'  = e^(b_last) S + sum_j k_j (e^(b_last - b_j) v_j)^T
// which is four products of 128 rows: Q K^T, P V, Q S and V'^T K.  Every exponent
// is formed as a sum of the log decays between two tokens, never as a difference of
// large sums: between blocks of 32 tokens as (rest of the column's block) + (blocks
// between) + (the row's block up to it), each factor at most 1.
//
// Precision.  P, S and V' are fp32 values that enter a product as a 16-bit part and
// the rounded remainder (two MMAs that share the other operand).  One part alone
// would add the error of a second output rounding, and 2^-9 to the states.  fp16
// operands are scaled by powers of two (P by row, V' by channel, S as a whole), so
// that large scores or states do not leave fp16's range and small ones keep their
// bits.  The state itself stays in fp32 registers and is only added to by fp32
// additions that round to nearest.
//
// A CTA walks one segment of one sequence for one kv head with all of its query
// heads.  Roles in a CTA of 320 threads:
//   warp 8 (producer)  a chunk's decay sums, and its tiles by TMA: K (2 slots), the
//                      query heads' Q (2 slots), V (1 slot)
//   warp 9 (MMA)       per query head: scores = Q K^T, O = Q S, O += P V; per chunk,
//                      after the first head: delta = V'^T K
//   warps 0-3          one row of the chunk per thread: P from the scores, O scaled
//                      by e^(b_i) between its two products, the output
//   warps 4-7          one value channel per thread: V' from the V tile, and the
//                      state's column (head_size floats in registers), which goes to
//                      shared memory as the operand of the next chunk's Q S
// Tensor memory: scores, then P over them, in columns 0-127; O at 128; delta at 256;
// V' at 384 (high parts, then remainders at 448).
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
constexpr int kBlock = 32;         // tokens whose decays are summed as one
constexpr int kTcThreads = 320;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 128, kTmemDelta = 256, kTmemV = 384;
constexpr int kRegion = kChunk * 128; // 128 token rows of 64 elements

template <int D>
struct Geo {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = kHalves * kRegion;      // a Q, K or V tile
    static constexpr int kStateRegion = D * 128;         // 64 key channels of all value channels
    static constexpr int kState = kHalves * kStateRegion;
    static constexpr int kOffK = 0, kOffQ = 2 * kTile, kOffV = 4 * kTile, kOffS = 5 * kTile;
    static constexpr int kOffMisc = kOffS + 2 * kState;
};

// A chunk's decays, in log2 units where they are sums.
struct Decays {
    float upto[kChunk];   // sum from the block's first token up to this one
    float rest[kChunk];   // 2^(sum behind this one to the block's end)
    float block[4];       // the blocks' sums
};

struct Misc {
    uint64_t k_full[2], k_empty[2], q_full[2], q_empty[2], v_full, v_empty;
    uint64_t dec_full[2], dec_empty[2];
    uint64_t s_full, p_full, o1_full, o_full, o_free;
    uint64_t v1_full, d_full, st_full, qs_done, drain;
    Decays dec[2];
    float state_scale[2];    // what the state's operand was divided by
    float warp_max[4];
    uint32_t tmem_base;
    int unit[4];
    uint8_t poison[2][128];  // by value channel: the chunk's first token that is not finite, or 128
};

template <int D> constexpr int tc_smem_bytes()
{
    // at least half of an SM's: two CTAs would wait for each other's tensor memory
    return Geo<D>::kOffMisc + (int)sizeof(Misc) > 120 * 1024 ? Geo<D>::kOffMisc + (int)sizeof(Misc)
                                                             : 120 * 1024;
}
static_assert(tc_smem_bytes<128>() <= 232448, "shared memory of an SM");

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

// Two values as a 16-bit part and the rounded remainder.
template <typename T>
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo)
{
    hi = pack2<T>(a, b);
    const float2 h = unpack2<T>(hi);
    lo = pack2<T>(a - h.x, b - h.y);
}

// Exponent E that brings magnitudes up to m below 2^14 (or up to there): m 2^-E.
__device__ __forceinline__ int range_exponent(float m)
{
    return max((int)(__float_as_uint(m) >> 23 & 255) - 127 - 13, -40);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int lane)
{
    bool ok = true;
    if (lane == 0)
        ok = mbar_wait(bar, parity);
    return __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
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
            return;
        }
        before += __shfl_sync(~0u, x, 31);
    }
}

// kParts: the first pass over sequences of several segments.  It forms the state
// that each segment but the last one leaves, the first from the sequence's own
// state, the others from zero, and the segments' decays.
template <typename T, int D, bool kParts>
__global__ void __launch_bounds__(kTcThreads, 1)
    linear_chunk_kernel(const __grid_constant__ CUtensorMap q_map,
                        const __grid_constant__ CUtensorMap k_map,
                        const __grid_constant__ CUtensorMap v_map, const LinearParams p)
{
    using Gm = Geo<D>;
    constexpr int TB = Gm::kTile;
    constexpr bool kHalf = std::is_same<T, __half>::value;
    constexpr uint32_t kFmt = kHalf ? 0u : 1u;
    constexpr uint32_t kIdescScores = idesc_f16_f32(kFmt, 0, 0, kChunk, kChunk);
    constexpr uint32_t kIdescState = idesc_f16_f32(kFmt, 0, 0, kChunk, D); // Q S
    constexpr uint32_t kIdescValue = idesc_f16_f32(kFmt, 0, 1, 128, D);    // P V, V'^T K

    extern __shared__ __align__(1024) uint8_t smem[];
    Misc *m = reinterpret_cast<Misc *>(smem + Gm::kOffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int head = blockIdx.x, y = blockIdx.y;

    griddep_wait();
    // the last line is past every unit, so its search sees every sequence
    const bool tell = head == 0 && y == (int)gridDim.y - 1 && !kParts;
    if (p.segment == INT32_MAX) { // one segment each: line y is sequence y
        if (tid == 0) {
            int q0, len;
            m->unit[2] = segments_of(p, y, q0, len, head == 0);
            m->unit[0] = m->unit[2] ? y : -1;
            m->unit[1] = 0;
        }
    } else if (warp == 0) {
        int s, j = 0, n = 0;
        find_unit(p, y, lane, tell, s, j, n);
        if (lane == 0)
            m->unit[0] = s, m->unit[1] = j, m->unit[2] = n;
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m->k_full[i], 1);
            mbar_init(&m->k_empty[i], 1);
            mbar_init(&m->q_full[i], 1);
            mbar_init(&m->q_empty[i], 1);
            mbar_init(&m->dec_full[i], 1);
            mbar_init(&m->dec_empty[i], kParts ? 4 : 8);
        }
        mbar_init(&m->v_full, 1);
        mbar_init(&m->v_empty, 1);
        mbar_init(&m->s_full, 1);
        mbar_init(&m->p_full, 4);
        mbar_init(&m->o1_full, 1);
        mbar_init(&m->o_full, 1);
        mbar_init(&m->o_free, 4);
        mbar_init(&m->v1_full, 4);
        mbar_init(&m->d_full, 1);
        mbar_init(&m->st_full, 4);
        mbar_init(&m->qs_done, 1);
        mbar_init(&m->drain, 1);
        fence_barrier_init();
    }
    __syncthreads();
    const int s = m->unit[0], j = m->unit[1], nseg = m->unit[2];
    if (s < 0 || (kParts && j == nseg - 1))
        return;
    const int q0 = p.query_start_loc[s], q1 = p.query_start_loc[s + 1];
    const int t0 = q0 + (j ? j * p.segment : 0);
    const int len = min(q1 - t0, p.segment), n = (len + kChunk - 1) / kChunk;
    const int src = p.src_states[s], dst = p.dst_states[s];
    const int per = p.num_heads / p.num_kv_heads;
    if (tid == 0 && head == 0 && !kParts && (src >= p.num_states || dst >= p.num_states))
        atomicOr(p.err, PA_DEVERR_STATE_);
    if (warp == kMmaWarp) {
        tmem_alloc(&m->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = m->tmem_base;

    if (warp == kProducerWarp) {
        // ================================================================ producer
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
        // this lane's four tokens of chunk c, in log2 units; below 2^-128 is 0, and
        // a difference of two such sums stays a number
        auto read_decays = [&](int c, float (&g)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = c * kChunk + lane * 4 + i;
                float x = 0.f;
                if (t < len)
                    x = log_decay[(int64_t)(t0 + t) * p.decay_stride] * 1.4426950408889634f;
                g[i] = x < -128.f ? -128.f : x;
            }
        };
        float g[4];
        bool ok = true;
        int loaded_k = 0, loaded_q = 0, loaded_v = 0;
        if (n > 0)
            read_decays(0, g);
        for (int c = 0, it = 0; ok && c < n; ++c) {
            const int b = c & 1, t = t0 + c * kChunk;
            const uint32_t again = (uint32_t)((c >> 1) - 1) & 1;
            if (c >= 2 && !warp_wait(&m->k_empty[b], again, lane)) {
                ok = false;
                break;
            }
            if (lane == 0)
                load(Gm::kOffK + b * TB, &k_map, &m->k_full[b], head, t);
            ++loaded_k;
            if (c >= 2 && !warp_wait(&m->dec_empty[b], again, lane)) {
                ok = false;
                break;
            }
            Decays &d = m->dec[b];
            float upto[4], rest[4], total;
            upto[0] = g[0];
#pragma unroll
            for (int i = 1; i < 4; ++i)
                upto[i] = upto[i - 1] + g[i];
            rest[3] = 0.f;
#pragma unroll
            for (int i = 2; i >= 0; --i)
                rest[i] = rest[i + 1] + g[i + 1];
            total = upto[3];
            float up = total, down = total; // over the 8 lanes of a block
#pragma unroll
            for (int o = 1; o < 8; o *= 2) {
                const float a = __shfl_up_sync(~0u, up, o, 8), z = __shfl_down_sync(~0u, down, o, 8);
                if ((lane & 7) >= o)
                    up += a;
                if ((lane & 7) + o < 8)
                    down += z;
            }
            float before = __shfl_up_sync(~0u, up, 1, 8), behind = __shfl_down_sync(~0u, down, 1, 8);
            before = lane & 7 ? before : 0.f;
            behind = (lane & 7) < 7 ? behind : 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                d.upto[lane * 4 + i] = before + upto[i];
                d.rest[lane * 4 + i] = exp2f(behind + rest[i]);
            }
            if ((lane & 7) == 7)
                d.block[lane >> 3] = up;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&m->dec_full[b]);
            if (c + 1 < n)
                read_decays(c + 1, g);
            for (int h = 0; h < (kParts ? 1 : per); ++h, ++it) {
                if (!kParts) {
                    if (it >= 2 && !warp_wait(&m->q_empty[it & 1], (uint32_t)((it >> 1) - 1) & 1, lane)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0)
                        load(Gm::kOffQ + (it & 1) * TB, &q_map, &m->q_full[it & 1], head * per + h, t);
                    ++loaded_q;
                }
                if (h == 0) {
                    if (c >= 1 && !warp_wait(&m->v_empty, (uint32_t)(c - 1) & 1, lane)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0)
                        load(Gm::kOffV, &v_map, &m->v_full, head, t);
                    ++loaded_v;
                }
            }
        }
        if (!ok && lane == 0) {
            // Given up: no tile may land in a later CTA's memory, so the last load on
            // each barrier is awaited, within the waits' own limit.
            atomicOr(p.err, PA_DEVERR_TIMEOUT_);
            auto settle = [](uint64_t *bar, int loads) {
                if (loads > 0)
                    mbar_wait(bar, (uint32_t)(loads - 1) & 1);
            };
            for (int b = 0; b < 2; ++b) {
                settle(&m->k_full[b], (loaded_k + 1 - b) >> 1);
                settle(&m->q_full[b], (loaded_q + 1 - b) >> 1);
            }
            settle(&m->v_full, loaded_v);
        }
    } else if (warp == kMmaWarp) {
        // ============================================================== MMA issuer
        const uint64_t k_desc = smem_desc_sw128(smem_addr(smem + Gm::kOffK), 16, 1024);
        const uint64_t kt_desc = smem_desc_sw128(smem_addr(smem + Gm::kOffK), kRegion, 1024);
        const uint64_t q_desc = smem_desc_sw128(smem_addr(smem + Gm::kOffQ), 16, 1024);
        const uint64_t v_desc = smem_desc_sw128(smem_addr(smem + Gm::kOffV), kRegion, 1024);
        const uint64_t s_desc = smem_desc_sw128(smem_addr(smem + Gm::kOffS), 16, 1024);
        auto slot = [](int b) { return (uint64_t)((uint32_t)(b * TB) >> 4); };
        bool ok = true;
        int it = 0;
        for (int c = 0; ok && c < n; ++c) {
            const int kb = c & 1;
            if (!(ok = warp_wait(&m->k_full[kb], (uint32_t)(c >> 1) & 1, lane)))
                break;
            for (int h = 0; h < (kParts ? 1 : per); ++h, ++it) {
                const int qb = it & 1;
                const uint64_t qd = q_desc + slot(qb);
                if (!kParts) {
                    // scores, over the P that the last product has read
                    if (!(ok = warp_wait(&m->q_full[qb], (uint32_t)(it >> 1) & 1, lane)))
                        break;
                    tc_fence_after_sync();
                    if (lane == 0) {
                        const uint64_t kd = k_desc + slot(kb);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t o = (uint64_t)(((kk >> 2) * kRegion + (kk & 3) * 32) >> 4);
                            umma_f16(tmem, qd + o, kd + o, kIdescScores, kk > 0 ? 1u : 0u);
                        }
                        umma_commit(&m->s_full);
                    }
                    __syncwarp();
                    // O = Q S, both parts
                    if (h == 0)
                        ok = warp_wait(&m->st_full, (uint32_t)c & 1, lane);
                    if (ok && it > 0)
                        ok = warp_wait(&m->o_free, (uint32_t)(it - 1) & 1, lane);
                    if (!ok)
                        break;
                    tc_fence_after_sync();
                    if (lane == 0) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t o = (uint64_t)(((kk >> 2) * kRegion + (kk & 3) * 32) >> 4);
                            const uint64_t so =
                                (uint64_t)(((kk >> 2) * Gm::kStateRegion + (kk & 3) * 32) >> 4);
                            umma_f16(tmem + kTmemO, qd + o, s_desc + so, kIdescState, kk > 0 ? 1u : 0u);
                            umma_f16(tmem + kTmemO, qd + o, s_desc + (Gm::kState >> 4) + so,
                                     kIdescState, 1u);
                        }
                        umma_commit(&m->o1_full);
                        umma_commit(&m->q_empty[qb]);
                        if (h == per - 1)
                            umma_commit(&m->qs_done);
                    }
                    __syncwarp();
                    // O += P V
                    ok = warp_wait(&m->p_full, (uint32_t)it & 1, lane);
                }
                if (ok && h == 0)
                    ok = warp_wait(&m->v1_full, (uint32_t)c & 1, lane);
                if (!ok)
                    break;
                tc_fence_after_sync();
                if (lane == 0) {
                    if (!kParts) {
#pragma unroll
                        for (int kk = 0; kk < kChunk / 16; ++kk) {
                            const uint64_t vd = v_desc + (uint64_t)((kk * 2048) >> 4);
                            umma_f16_tmem_a(tmem + kTmemO, tmem + (uint32_t)(kk * 8), vd, kIdescValue, 1u);
                            umma_f16_tmem_a(tmem + kTmemO, tmem + (uint32_t)(64 + kk * 8), vd,
                                            kIdescValue, 1u);
                        }
                        umma_commit(&m->o_full);
                    }
                    if (h == 0) { // delta = V'^T K
                        const uint64_t kd = kt_desc + slot(kb);
#pragma unroll
                        for (int kk = 0; kk < kChunk / 16; ++kk) {
                            const uint64_t o = (uint64_t)((kk * 2048) >> 4);
                            umma_f16_tmem_a(tmem + kTmemDelta, tmem + kTmemV + (uint32_t)(kk * 8), kd + o,
                                            kIdescValue, kk > 0 ? 1u : 0u);
                            umma_f16_tmem_a(tmem + kTmemDelta, tmem + kTmemV + (uint32_t)(64 + kk * 8),
                                            kd + o, kIdescValue, 1u);
                        }
                        umma_commit(&m->d_full);
                    }
                    if (kParts || h == per - 1) {
                        umma_commit(&m->v_empty);
                        umma_commit(&m->k_empty[kb]);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0)
            atomicOr(p.err, PA_DEVERR_TIMEOUT_);
        if (lane == 0)
            umma_commit(&m->drain);
        warp_wait(&m->drain, 0, lane);
    } else if (warp < 4) {
        // ===================================================== rows: P and outputs
        const int row = tid, blk = warp;
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const uint32_t s_addr = tmem + lane_base, o_addr = tmem + lane_base + kTmemO;
        bool ok = true;
        int it = 0;
        for (int c = 0; ok && !kParts && c < n; ++c) {
            const Decays &d = m->dec[c & 1];
            const int live = min(kChunk, len - c * kChunk);
            float upto = 0.f, inter = 0.f, f[3] = {0.f, 0.f, 0.f};
            for (int h = 0; h < per; ++h, ++it) {
                if (h == 0) {
                    if (!(ok = warp_wait(&m->dec_full[c & 1], (uint32_t)(c >> 1) & 1, lane)))
                        break;
                    // 2^(decays from the end of column block J to this row), J = blk - 1 - k
                    upto = d.upto[row];
                    float sum = upto;
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        if (k < blk) {
                            f[k] = exp2f(sum) * p.scale;
                            sum += d.block[blk - 1 - k];
                        }
                    inter = exp2f(sum) * p.scale; // from the chunk's beginning
                }
                if (!(ok = warp_wait(&m->s_full, (uint32_t)it & 1, lane)))
                    break;
                tc_fence_after_sync();
                uint32_t sv[kChunk];
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (b <= blk)
                        tmem_ld32_nowait(s_addr + (uint32_t)(b * 32),
                                         *reinterpret_cast<uint32_t(*)[32]>(sv + b * 32));
                tmem_wait_ld();
                float down = 1.f, up = 1.f; // 2^-E, 2^E
                if constexpr (kHalf) {
                    float most = 0.f;
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        if (b <= blk)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (b < blk || i <= lane)
                                    most = fmaxf(most, fabsf(__uint_as_float(sv[b * 32 + i])));
                    const int e = range_exponent(most * fabsf(p.scale));
                    down = power_of_two(-e);
                    up = power_of_two(e);
                }
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    uint32_t hi[16], lo[16];
                    if (b < blk) {
                        const float fb = (b == blk - 1 ? f[0] : b == blk - 2 ? f[1] : f[2]) * down;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 r = *reinterpret_cast<const float4 *>(&d.rest[b * 32 + i * 4]);
                            const uint32_t *const x = sv + b * 32 + i * 4;
                            split2<T>(__uint_as_float(x[0]) * (r.x * fb), __uint_as_float(x[1]) * (r.y * fb),
                                      hi[2 * i], lo[2 * i]);
                            split2<T>(__uint_as_float(x[2]) * (r.z * fb), __uint_as_float(x[3]) * (r.w * fb),
                                      hi[2 * i + 1], lo[2 * i + 1]);
                        }
                    } else if (b == blk) {
                        const float fb = p.scale * down;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 u = *reinterpret_cast<const float4 *>(&d.upto[b * 32 + i * 4]);
                            const float l[4] = {u.x, u.y, u.z, u.w};
                            float x[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                x[k] = i * 4 + k <= lane ? __uint_as_float(sv[b * 32 + i * 4 + k]) *
                                                               (ex2(upto - l[k]) * fb)
                                                         : 0.f;
                            split2<T>(x[0], x[1], hi[2 * i], lo[2 * i]);
                            split2<T>(x[2], x[3], hi[2 * i + 1], lo[2 * i + 1]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            hi[i] = lo[i] = 0;
                    }
                    // over the scores, which are all in registers
                    tmem_st16(s_addr + (uint32_t)(b * 16), hi);
                    tmem_st16(s_addr + (uint32_t)(64 + b * 16), lo);
                }
                if (h == 0) {
                    // both before p_full lets their next phases begin
                    ok = warp_wait(&m->st_full, (uint32_t)c & 1, lane) &&
                         warp_wait(&m->v1_full, (uint32_t)c & 1, lane);
                    if (ok && kHalf)
                        inter *= m->state_scale[c & 1];
                }
                ok = ok && warp_wait(&m->o1_full, (uint32_t)it & 1, lane);
                if (!ok)
                    break;
                tc_fence_after_sync();
                const float of = inter * down;
#pragma unroll
                for (int b = 0; b < D / 32; ++b) {
                    uint32_t o[32];
                    tmem_ld32_nowait(o_addr + (uint32_t)(b * 32), o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        o[i] = __float_as_uint(__uint_as_float(o[i]) * of);
                    tmem_st32(o_addr + (uint32_t)(b * 32), o);
                }
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&m->p_full);
                if (!(ok = warp_wait(&m->o_full, (uint32_t)it & 1, lane)))
                    break;
                tc_fence_after_sync();
                T *const out = static_cast<T *>(p.out) +
                               ((int64_t)(t0 + c * kChunk + row) * p.num_heads + head * per + h) * D;
                uint32_t w[D / 2];
#pragma unroll
                for (int b = 0; b < D / 32; ++b) {
                    uint32_t o[32];
                    tmem_ld32_nowait(o_addr + (uint32_t)(b * 32), o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        w[b * 16 + i] = pack2<T>(__uint_as_float(o[2 * i]) * up,
                                                 __uint_as_float(o[2 * i + 1]) * up);
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&m->o_free);
                if (row < live) {
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
                        reinterpret_cast<uint4 *>(out)[i] =
                            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                    // A value that is not finite was taken out of the product, where it
                    // would have reached the rows before it as 0 * NaN.
                    const uint32_t *const hurt = reinterpret_cast<const uint32_t *>(m->poison[c & 1]);
                    for (int i = 0; i < D / 4; ++i) {
                        const uint32_t x = hurt[i];
                        if (x != 0x80808080u)
                            for (int k = 0; k < 4; ++k)
                                if ((int)(x >> 8 * k & 255) <= row)
                                    out[4 * i + k] = (T)__uint_as_float(0x7FFFFFFFu);
                    }
                }
                if (h == per - 1) {
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&m->dec_empty[c & 1]);
                }
            }
        }
        if (!ok && lane == 0)
            atomicOr(p.err, PA_DEVERR_TIMEOUT_);
    } else {
        // ================================================= value channels: the state
        const int wg = warp & 3, ch = tid & 127; // value channel, and token row in a tail
        const uint32_t lane_base = (uint32_t)(wg * 32) << 16;
        const bool mine = ch < D;
        const int64_t one = (int64_t)D * D;
        float S[D];
        {
            const float *from = nullptr;
            if (j > 0 && !kParts)
                from = p.parts + ((int64_t)(y - 1) * p.num_kv_heads + head) * one;
            else if (j == 0 && src >= 0 && src < p.num_states)
                from = p.states + ((int64_t)src * p.num_kv_heads + head) * one;
#pragma unroll
            for (int k = 0; k < D; ++k)
                S[k] = mine && from ? from[(int64_t)k * D + ch] : 0.f;
        }
        // The state as the operand of Q S: row = value channel, 64 key channels a
        // region, 16-byte pieces in the 128-byte swizzle.
        auto put_state = [&](int c) {
            float down = 1.f;
            if constexpr (kHalf) {
                float most = 0.f;
#pragma unroll
                for (int k = 0; k < D; ++k)
                    most = fmaxf(most, fabsf(S[k]) < INFINITY ? fabsf(S[k]) : 0.f);
                const unsigned top = __reduce_max_sync(~0u, __float_as_uint(most));
                if (lane == 0)
                    m->warp_max[wg] = __uint_as_float(top);
                bar_sync(1, 128);
                most = fmaxf(fmaxf(m->warp_max[0], m->warp_max[1]), fmaxf(m->warp_max[2], m->warp_max[3]));
                bar_sync(1, 128);
                const int e = range_exponent(most);
                down = power_of_two(-e);
                if (ch == 0)
                    m->state_scale[c & 1] = power_of_two(e);
            }
            if (mine) {
                uint8_t *const at = smem + Gm::kOffS + ch * 128;
#pragma unroll
                for (int k = 0; k < D; k += 8) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        split2<T>(S[k + 2 * i] * down, S[k + 2 * i + 1] * down, hi[i], lo[i]);
                    const int off = (k / 64) * Gm::kStateRegion + (((k % 64) / 8) ^ (ch & 7)) * 16;
                    *reinterpret_cast<uint4 *>(at + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(at + Gm::kState + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&m->st_full);
        };
        if (!kParts && n > 0)
            put_state(0);
        float decay_log2 = 0.f; // of the whole segment
        bool ok = true; // of this warp, until the next barrier
        for (int c = 0; c < n; ++c) {
            const int b = c & 1, live = min(kChunk, len - c * kChunk);
            const Decays &d = m->dec[b];
            ok = ok && warp_wait(&m->dec_full[b], (uint32_t)(c >> 1) & 1, lane) &&
                 warp_wait(&m->v_full, (uint32_t)c & 1, lane);
            if (ok && live < kChunk)
                ok = warp_wait(&m->k_full[b], (uint32_t)(c >> 1) & 1, lane);
            // every thread of the group leaves or none does: barriers follow
            ok = !bar_sync_or(1, 128, !ok);
            if (!ok)
                break;
            if (live < kChunk) {
                // the tile's rows behind the sequence are a neighbour's: zeros
                if (ch >= live)
#pragma unroll
                    for (int hf = 0; hf < Gm::kHalves; ++hf)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int off = hf * kRegion + ch * 128 + i * 16;
                            *reinterpret_cast<uint4 *>(smem + Gm::kOffV + off) = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4 *>(smem + Gm::kOffK + b * TB + off) =
                                make_uint4(0, 0, 0, 0);
                        }
                bar_sync(1, 128);
            }
            // 2^(decays behind each block of 32, to the chunk's end)
            float behind[4];
            float sum = 0.f;
#pragma unroll
            for (int k = 3; k >= 0; --k) {
                behind[k] = exp2f(sum);
                sum += d.block[k];
            }
            const float decay = exp2f(sum);
            decay_log2 += sum;
            // V': this channel of all tokens, decayed to the chunk's end
            float back = 1.f;
            bool hurt = false;
            if (mine) {
                const uint8_t *const col = smem + Gm::kOffV + (ch / 64) * kRegion + (ch % 8) * 2;
                const int piece = (ch % 64) / 8;
                auto value = [&](int t) {
                    return value_of<T>(*reinterpret_cast<const uint16_t *>(
                        col + t * 128 + ((piece ^ (t & 7)) * 16)));
                };
                float scale = 1.f;
                if constexpr (kHalf) {
                    float most = 0.f;
#pragma unroll 32
                    for (int t = 0; t < kChunk; ++t)
                        most = fmaxf(most, fabsf(value(t)));
                    const int e = range_exponent(most < INFINITY ? most : 65504.f);
                    scale = power_of_two(-e);
                    back = power_of_two(e);
                }
                auto put = [&]() {
                    float odd = 0.f; // NaN once a value is not finite
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float f = behind[k] * scale;
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 r = *reinterpret_cast<const float4 *>(&d.rest[k * 32 + i * 4]);
                            float x[4];
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                x[z] = value(k * 32 + i * 4 + z);
                                odd = fmaf(x[z], 0.f, odd);
                            }
                            split2<T>(x[0] * (r.x * f), x[1] * (r.y * f), hi[2 * i], lo[2 * i]);
                            split2<T>(x[2] * (r.z * f), x[3] * (r.w * f), hi[2 * i + 1], lo[2 * i + 1]);
                        }
                        tmem_st16(tmem + lane_base + kTmemV + (uint32_t)(k * 16), hi);
                        tmem_st16(tmem + lane_base + kTmemV + (uint32_t)(64 + k * 16), lo);
                    }
                    return odd;
                };
                const float odd = put();
                hurt = odd != 0.f; // NaN compares unequal
                int first = 128;
                if (hurt) {
                    for (int t = kChunk - 1; t >= 0; --t) {
                        uint16_t *const at = reinterpret_cast<uint16_t *>(
                            const_cast<uint8_t *>(col) + t * 128 + ((piece ^ (t & 7)) * 16));
                        if (!(fabsf(value_of<T>(*at)) < INFINITY)) {
                            first = t;
                            *at = 0;
                        }
                    }
                }
                if (__any_sync(~0u, hurt))
                    put();
                m->poison[b][ch] = (uint8_t)first;
                tmem_wait_st();
            }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&m->dec_empty[b]);
                mbar_arrive(&m->v1_full);
            }
            ok = warp_wait(&m->d_full, (uint32_t)c & 1, lane);
            tc_fence_after_sync();
            if (ok && mine) {
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    uint32_t x[32];
                    tmem_ld32_nowait(tmem + lane_base + kTmemDelta + (uint32_t)(k * 32), x);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        S[k * 32 + i] = fmaf(decay, S[k * 32 + i], __uint_as_float(x[i]) * back);
                }
                if (hurt)
#pragma unroll
                    for (int k = 0; k < D; ++k)
                        S[k] = __uint_as_float(0x7FFFFFFFu);
            }
            tc_fence_before_sync();
            if (!kParts && c + 1 < n) {
                ok = ok && warp_wait(&m->qs_done, (uint32_t)c & 1, lane);
                ok = !bar_sync_or(1, 128, !ok);
                if (!ok)
                    break;
                put_state(c + 1);
            }
        }
        if (!ok && lane == 0)
            atomicOr(p.err, PA_DEVERR_TIMEOUT_);
        if (ok && mine) {
            float *to = nullptr;
            if (kParts)
                to = p.parts + ((int64_t)y * p.num_kv_heads + head) * one;
            else if (j == nseg - 1 && dst < p.num_states)
                to = p.states + ((int64_t)dst * p.num_kv_heads + head) * one;
            if (to)
#pragma unroll
                for (int k = 0; k < D; ++k)
                    to[(int64_t)k * D + ch] = S[k];
            if (kParts && ch == 0)
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
        // sequences that overlap can be more than the lines there are
        if (tid == 0)
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
    // the last segment has no part
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
