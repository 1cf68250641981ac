// pa_block_decode.cuh -- decode attention over whole or listed blocks of a
// 16-bit pool, or of an e4m3 pool with one scale for each (plane, block, kv
// head).
//
// For a sequence, a kv head and the (at most 8) query heads of its group:
//   out = sum_t softmax_t(scale * q . k_t) v_t
// over the tokens of the sequence, or of its listed blocks.  One pass: a warp
// takes 16 tokens of one kv head at a time, forms S^T = K Q^T (16 x 8) and
// O^T += V^T P (D x 8) with m16n8k16 products, and keeps the running maximum
// and normaliser of the softmax in fp32.
//
// The operands are loaded straight into the registers of the products.  The
// contraction index of a product is any permutation of the channels (S) or of
// the tokens (O) as long as both operands use the same one, and the rows of
// O^T are any permutation of the channels, so every lane takes 16-byte pieces:
//   K  lane 4g + t: rows g and g + 8, bytes 16t + 64c of the row;
//   V  lane 4g + t: rows 2t, 2t+1, 2t+8, 2t+9, bytes 16g (+ 128 c) of the row.
// e4m3 codes become halves (exactly) in registers.
//
// Work.  The (sequence, group of HG kv heads, 16-token tile) triples are laid
// out in one line and cut into equal runs, one for each CTA, so that any mix
// of lengths balances.  Inside a CTA the 8 warps are HG heads times 8 / HG
// interleaved tiles.  A (sequence, group) that a cut divides leaves partial
// states, which a second kernel merges.
//
// e4m3 scales: the score takes the key scale; the value scale multiplies the
// probability before it is rounded to 16 bits.  The softmax's reference m is
// the maximum of score + log2(value scale), so that the largest product
// p * scale is 1 and halves hold the products of every block to the same
// absolute precision.
#pragma once

#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "pa_block.cuh"
#include "pa_internal.h"

namespace pa {
namespace block {

constexpr int kWarps = 8;      // warps of a CTA
constexpr int kMaxCtas = 304;  // CTAs of a launch, at most (workspace size)
constexpr int kTile = 16;      // tokens a warp takes at a time
constexpr int kMinRun = 8;     // tiles a warp takes at least before work is cut

struct DecodeArgs {
    void *out;                 // [B, H, D]
    float *lse;                // [B, H] or NULL
    const void *q;             // [B, H, D]
    const char *pool;          // [2, NB, bs, Hkv, D]
    const float *scales;       // [2, NB, Hkv] (e4m3 pool)
    const int32_t *tables;     // [B, MB]
    const int32_t *seq_lens;   // [B]
    const int32_t *lists;      // [B, Hkv, K] block positions, or NULL: all blocks
    const int32_t *list_lens;  // [B]
    unsigned int *err;
    int4 *cuts;                // [CTAs] {sequence, head group, CTAs sharing it, -}
    float *ws_o;               // [CTAs, 2, HG * G, D]
    float *ws_ml;              // [CTAs, 2, HG * G, 2]
    int64_t plane;             // bytes of a plane
    int num_seqs, num_heads, num_kv_heads, group, heads_log2, num_groups, num_blocks, max_blocks,
        block_log2, max_listed, len_cap;
    float qscale;              // scale * log2 e
};

// Tiles of sequence s, at least one (an empty sequence writes zeros).
__device__ __forceinline__ int tiles_of(const DecodeArgs &p, int s, bool report)
{
    int n;
    if (p.lists) {
        n = p.list_lens[s];
        if (n < 0 || n > p.max_listed) {
            if (report)
                atomicOr(p.err, PA_DEVERR_SEQ_LEN_);
            n = n < 0 ? 0 : p.max_listed;
        }
        n <<= p.block_log2 - 4;
    } else {
        n = p.seq_lens[s];
        n = (min(max(n, 0), p.len_cap) + kTile - 1) / kTile;
    }
    return max(n, 1);
}

__device__ __forceinline__ int length_of(const DecodeArgs &p, int s, bool report)
{
    const int len = p.seq_lens[s];
    if (len >= 0 && len <= p.len_cap)
        return len;
    if (report)
        atomicOr(p.err, PA_DEVERR_SEQ_LEN_);
    return len < 0 ? 0 : p.len_cap;
}

// Where a tile's 16 tokens are: the first pool row, or -1 for a block outside
// the pool (read as zeros); how many of them count.
struct Tile {
    int64_t row;
    int block, live;
};

// `listed`: entries of the sequence's lists.
__device__ __forceinline__ Tile locate(const DecodeArgs &p, int s, int head, int tile, int len,
                                       int listed)
{
    const int per = p.block_log2 - 4;
    int j = tile >> per;
    const int sub = tile & ((1 << per) - 1);
    Tile r = {-1, -1, 0};
    const int blocks = (len + (1 << p.block_log2) - 1) >> p.block_log2;
    if (p.lists) {
        const int i = j;
        if (i >= listed)
            return r;
        j = p.lists[((int64_t)s * p.num_kv_heads + head) * p.max_listed + i];
        if (j < 0)
            return r; // padding
        if (j >= blocks) {
            atomicOr(p.err, PA_DEVERR_BLOCK_ID_);
            return r;
        }
    }
    r.live = min(kTile, len - (j << p.block_log2) - sub * kTile);
    if (j >= blocks || r.live <= 0) {
        r.live = 0;
        return r;
    }
    const int blk = p.tables[(int64_t)s * p.max_blocks + j];
    if (blk < 0 || blk >= p.num_blocks) {
        atomicOr(p.err, PA_DEVERR_BLOCK_ID_);
        return r;
    }
    r.block = blk;
    r.row = ((int64_t)blk << p.block_log2) + sub * kTile;
    return r;
}

constexpr float kLn2 = 0.6931471805599453f;

// Probabilities and normalisers are carried times 2^lift.  In halves the
// largest probability is then 2^15, and the smallest that is not lost 2^-39 of
// it; bf16 has fp32's range and needs none.
template <typename M> constexpr float lift_of() { return std::is_same<M, __half>::value ? 15.f : 0.f; }

// T: type of q and out (and of a 16-bit pool).  E4M3: pool of e4m3 codes.
template <typename T, bool E4M3, int D>
__global__ void __launch_bounds__(32 * kWarps) block_decode_kernel(const DecodeArgs p)
{
    using M = typename std::conditional<E4M3, __half, T>::type; // type of the products
    // P is split into a 16-bit high part and the rounded remainder where one
    // part would add an error like the output's own rounding: not for a bf16
    // output of products in halves (11 bits against 8).
    constexpr bool kTwoParts = !(E4M3 && std::is_same<T, __nv_bfloat16>::value);
    constexpr float kLift = lift_of<M>();
    constexpr int kRow = D * (E4M3 ? 1 : 2);     // bytes of a head's row
    constexpr int kKPieces = kRow / 64;          // 16-byte pieces of a lane and row of K
    constexpr int kVWords = kRow / 32;           // words of a lane and row of V
    constexpr int kSteps = D / 16;               // products along D
    __shared__ int first_seq, first_base, total_tiles, warp_sums[kWarps];
    __shared__ float merge[kWarps][8][D + 2];

    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int heads = 1 << p.heads_log2;         // kv heads of the CTA
    const int hl = warp & (heads - 1), tw = warp >> p.heads_log2, tws = kWarps >> p.heads_log2;

    // ---- this CTA's run: [begin, end) of the line of tiles ----
    const int slice = (p.num_seqs + 32 * kWarps - 1) / (32 * kWarps);
    const int s_lo = min(tid * slice, p.num_seqs), s_hi = min(s_lo + slice, p.num_seqs);
    int mine = 0;
    for (int s = s_lo; s < s_hi; ++s)
        mine += tiles_of(p, s, blockIdx.x == 0);
    mine *= p.num_groups;
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, x, o);
        if (lane >= o)
            x += y;
    }
    if (lane == 31)
        warp_sums[warp] = x;
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        base += w < warp ? warp_sums[w] : 0;
        total += warp_sums[w];
    }
    base += x - mine;
    const int run = max((total + (int)gridDim.x - 1) / (int)gridDim.x, kMinRun * tws);
    const int begin = blockIdx.x * run, end = min(begin + run, total);
    if (tid == 0)
        p.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (begin >= total)
        return;
    if (begin >= base && begin < base + mine) {
        int s = s_lo;
        while (true) {
            const int n = tiles_of(p, s, false) * p.num_groups;
            if (begin < base + n)
                break;
            base += n;
            ++s;
        }
        first_seq = s;
        first_base = base;
    }
    __syncthreads();
    int s = first_seq, at = begin, seg = first_base;
    int tiles = tiles_of(p, s, false);
    int grp = (at - seg) / tiles;
    seg += grp * tiles;

    while (at < end) { // one (sequence, head group) after another
        const int seg_end = seg + tiles, stop = min(end, seg_end);
        const int head = (grp << p.heads_log2) + hl;
        const int len = length_of(p, s, lane == 0 && warp == 0);
        const int listed = p.lists ? min(p.list_lens[s], p.max_listed) : 0;

        // Query rows of the group, as the products take them; for e4m3 in
        // halves, scaled by a power of two so that the largest is near 2^15
        // (bf16 values keep their 8 bits over 29 binades below it).
        uint32_t qf[kSteps][2];
        float qmul0 = p.qscale, qmul1 = p.qscale;
        {
            const T *q = static_cast<const T *>(p.q) +
                         ((int64_t)s * p.num_heads + head * p.group + min(g, p.group - 1)) * D;
            uint2 raw[kSteps];
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int d = E4M3 ? (i / 4) * 64 + t * 16 + (i % 4) * 4
                                   : (i / 2) * 32 + t * 8 + (i % 2) * 4;
                raw[i] = *reinterpret_cast<const uint2 *>(q + d);
                if (g >= p.group)
                    raw[i] = make_uint2(0, 0);
            }
            if constexpr (E4M3 && std::is_same<T, __nv_bfloat16>::value) {
                float amax = 0.f;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const float2 a = float2_of<T>(raw[i].x), b = float2_of<T>(raw[i].y);
                    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)),
                                             fmaxf(fabsf(b.x), fabsf(b.y))));
                }
                amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
                const int e = max((int)(__float_as_uint(amax) >> 23) - 127 - 14, -120);
                const float down = two_to(-e);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const float2 a = float2_of<T>(raw[i].x), b = float2_of<T>(raw[i].y);
                    qf[i][0] = pair_of<__half>(a.x * down, a.y * down);
                    qf[i][1] = pair_of<__half>(b.x * down, b.y * down);
                }
                const float up = two_to(e);
                qmul0 *= __shfl_sync(~0u, up, 8 * t);
                qmul1 *= __shfl_sync(~0u, up, 8 * t + 4);
            } else {
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
                    qf[i][0] = raw[i].x, qf[i][1] = raw[i].y;
            }
        }

        float o[kSteps][4];
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[i][k] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        for (int tile = at - seg + tw; tile < stop - seg; tile += tws) {
            const Tile where = locate(p, s, head, tile, len, listed);
            if (where.live == 0)
                continue;
            float ks = 1.f, vs = 1.f;
            uint4 kr[2][kKPieces];
            uint32_t vr[4][kVWords];
#pragma unroll
            for (int i = 0; i < kKPieces; ++i)
                kr[0][i] = kr[1][i] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < kVWords; ++k)
                    vr[i][k] = 0;
            if (where.block >= 0) {
                const int64_t stride = (int64_t)p.num_kv_heads * kRow;
                const char *src = p.pool + where.row * stride + head * kRow;
#pragma unroll
                for (int i = 0; i < kKPieces; ++i) {
                    kr[0][i] = load16(src + g * stride + i * 64 + t * 16);
                    kr[1][i] = load16(src + (g + 8) * stride + i * 64 + t * 16);
                }
                src += p.plane;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 2 * t + (i & 1) + (i >> 1) * 8;
                    if constexpr (kRow == 64) {
                        const uint2 v = load8(src + row * stride + g * 8);
                        vr[i][0] = v.x, vr[i][1] = v.y;
                    } else {
#pragma unroll
                        for (int k = 0; k < kVWords; k += 4) {
                            const uint4 v = load16(src + row * stride + k * 32 + g * 16);
                            vr[i][k] = v.x, vr[i][k + 1] = v.y, vr[i][k + 2] = v.z,
                            vr[i][k + 3] = v.w;
                        }
                    }
                    if (row >= where.live) // what lies there may be NaN
#pragma unroll
                        for (int k = 0; k < kVWords; ++k)
                            vr[i][k] = 0;
                }
                if constexpr (E4M3) {
                    const int64_t sc = (int64_t)where.block * p.num_kv_heads + head;
                    ks = p.scales[sc];
                    vs = p.scales[sc + (int64_t)p.num_blocks * p.num_kv_heads];
                }
            }

            // S^T: rows are tokens g and g + 8, columns queries 2t and 2t + 1
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                if constexpr (E4M3) {
                    const uint32_t a = (&kr[0][i / 4].x)[i % 4], b = (&kr[1][i / 4].x)[i % 4];
                    mma_16816<M>(c, half2_of_e4m3x2(a), half2_of_e4m3x2(b), half2_of_e4m3x2_hi(a),
                                 half2_of_e4m3x2_hi(b), qf[i][0], qf[i][1]);
                } else {
                    const uint32_t *a = &kr[0][i / 2].x + i % 2 * 2, *b = &kr[1][i / 2].x + i % 2 * 2;
                    mma_16816<M>(c, a[0], b[0], a[1], b[1], qf[i][0], qf[i][1]);
                }
            }
            const float f0 = E4M3 ? qmul0 * ks : qmul0, f1 = E4M3 ? qmul1 * ks : qmul1;
            const bool live0 = g < where.live, live1 = g + 8 < where.live;
            c[0] = live0 ? c[0] * f0 : -INFINITY;
            c[1] = live0 ? c[1] * f1 : -INFINITY;
            c[2] = live1 ? c[2] * f0 : -INFINITY;
            c[3] = live1 ? c[3] * f1 : -INFINITY;

            // running maximum of score + log2(value scale), over the 16 tokens
            float n0 = fmaxf(c[0], c[2]), n1 = fmaxf(c[1], c[3]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                n0 = fmaxf(n0, __shfl_xor_sync(~0u, n0, off));
                n1 = fmaxf(n1, __shfl_xor_sync(~0u, n1, off));
            }
            if constexpr (E4M3) {
                const float lift = __log2f(vs);
                n0 += lift;
                n1 += lift;
            }
            n0 = fmaxf(m0, n0);
            n1 = fmaxf(m1, n1);
            float r0 = n0 == -INFINITY ? 0.f : n0, r1 = n1 == -INFINITY ? 0.f : n1;
            if (__any_sync(~0u, n0 != m0 || n1 != m1)) {
                const float a0 = ex2(m0 - r0), a1 = ex2(m1 - r1);
                l0 *= a0;
                l1 *= a1;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    o[i][0] *= a0;
                    o[i][1] *= a1;
                    o[i][2] *= a0;
                    o[i][3] *= a1;
                }
                m0 = n0;
                m1 = n1;
            }
            r0 -= kLift;
            r1 -= kLift;
            c[0] = ex2(c[0] - r0);
            c[1] = ex2(c[1] - r1);
            c[2] = ex2(c[2] - r0);
            c[3] = ex2(c[3] - r1);
            l0 += c[0] + c[2];
            l1 += c[1] + c[3];
            if constexpr (E4M3)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    c[k] *= vs;
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t h = pair_of<M>(c[2 * k], c[2 * k + 1]);
                hi[k] = transpose_8x8(h);
                if constexpr (kTwoParts) {
                    const float2 back = float2_of<M>(h);
                    lo[k] = transpose_8x8(pair_of<M>(c[2 * k] - back.x, c[2 * k + 1] - back.y));
                }
            }

            // O^T: rows are channels 2i and 2i + 1 of each lane's list
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                uint32_t a0, a1, a2, a3;
                if constexpr (E4M3) {
                    const uint32_t sel = i % 2 ? 0x7362 : 0x5140;
                    const uint32_t u = __byte_perm(vr[0][i / 2], vr[1][i / 2], sel);
                    const uint32_t v = __byte_perm(vr[2][i / 2], vr[3][i / 2], sel);
                    a0 = half2_of_e4m3x2(u);
                    a1 = half2_of_e4m3x2_hi(u);
                    a2 = half2_of_e4m3x2(v);
                    a3 = half2_of_e4m3x2_hi(v);
                } else {
                    a0 = __byte_perm(vr[0][i], vr[1][i], 0x5410);
                    a1 = __byte_perm(vr[0][i], vr[1][i], 0x7632);
                    a2 = __byte_perm(vr[2][i], vr[3][i], 0x5410);
                    a3 = __byte_perm(vr[2][i], vr[3][i], 0x7632);
                }
                mma_16816<M>(o[i], a0, a1, a2, a3, hi[0], hi[1]);
                if constexpr (kTwoParts)
                    mma_16816<M>(o[i], a0, a1, a2, a3, lo[0], lo[1]);
            }
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l0 += __shfl_xor_sync(~0u, l0, off);
            l1 += __shfl_xor_sync(~0u, l1, off);
        }

        // Join the warps that shared the head's tiles.
        if (tws > 1) {
            __syncthreads();
            float *const dst0 = merge[warp][2 * t], *const dst1 = merge[warp][2 * t + 1];
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                dst0[g * (D / 8) + 2 * i] = o[i][0];
                dst1[g * (D / 8) + 2 * i] = o[i][1];
                dst0[g * (D / 8) + 2 * i + 1] = o[i][2];
                dst1[g * (D / 8) + 2 * i + 1] = o[i][3];
            }
            if (g == 0) {
                dst0[D] = m0, dst0[D + 1] = l0;
                dst1[D] = m1, dst1[D + 1] = l1;
            }
            __syncthreads();
            if (tw == 0) {
                float w0 = m0, w1 = m1;
                for (int k = 1; k < tws; ++k) {
                    w0 = fmaxf(w0, merge[hl + (k << p.heads_log2)][2 * t][D]);
                    w1 = fmaxf(w1, merge[hl + (k << p.heads_log2)][2 * t + 1][D]);
                }
                const float r0 = w0 == -INFINITY ? 0.f : w0, r1 = w1 == -INFINITY ? 0.f : w1;
                float a0 = ex2(m0 - r0), a1 = ex2(m1 - r1);
                l0 *= a0;
                l1 *= a1;
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
                    o[i][0] *= a0, o[i][1] *= a1, o[i][2] *= a0, o[i][3] *= a1;
                for (int k = 1; k < tws; ++k) {
                    const float *src0 = merge[hl + (k << p.heads_log2)][2 * t];
                    const float *src1 = merge[hl + (k << p.heads_log2)][2 * t + 1];
                    a0 = ex2(src0[D] - r0);
                    a1 = ex2(src1[D] - r1);
                    l0 += a0 * src0[D + 1];
                    l1 += a1 * src1[D + 1];
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) {
                        o[i][0] += a0 * src0[g * (D / 8) + 2 * i];
                        o[i][1] += a1 * src1[g * (D / 8) + 2 * i];
                        o[i][2] += a0 * src0[g * (D / 8) + 2 * i + 1];
                        o[i][3] += a1 * src1[g * (D / 8) + 2 * i + 1];
                    }
                }
                m0 = w0;
                m1 = w1;
            }
        }

        // A whole (sequence, group) is finished here; a cut one leaves its
        // state: slot 1 of the CTA that began it, slot 0 of the others.
        const bool whole = at == seg && stop == seg_end;
        const int slot = at == seg ? 1 : 0;
        if (tid == 0 && at == seg && !whole)
            p.cuts[blockIdx.x] = make_int4(s, grp, (seg_end - 1) / run - (int)blockIdx.x + 1, 0);
        if (tw == 0) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int col = 2 * t + k;
                if (col >= p.group)
                    continue;
                const float l = k ? l1 : l0, m = k ? m1 : m0;
                if (whole) {
                    const int64_t row = (int64_t)s * p.num_heads + head * p.group + col;
                    const float inv = l != 0.f ? 1.f / l : 0.f;
                    T *dst = static_cast<T *>(p.out) + row * D;
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) {
                        const int d = E4M3 || D == 64 ? g * (D / 8) + 2 * i
                                                      : (i / 4) * 64 + g * 8 + (i % 4) * 2;
                        *reinterpret_cast<uint32_t *>(dst + d) =
                            pair_of<T>(o[i][k] * inv, o[i][k + 2] * inv);
                    }
                    if (p.lse && g == 0)
                        p.lse[row] = l != 0.f ? (m - kLift + log2f(l)) * kLn2 : -INFINITY;
                } else {
                    const int64_t row = ((int64_t)(2 * blockIdx.x + slot) << p.heads_log2) * p.group +
                                        hl * p.group + col;
                    float *dst = p.ws_o + row * D;
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) {
                        const int d = E4M3 || D == 64 ? g * (D / 8) + 2 * i
                                                      : (i / 4) * 64 + g * 8 + (i % 4) * 2;
                        *reinterpret_cast<float2 *>(dst + d) = make_float2(o[i][k], o[i][k + 2]);
                    }
                    if (g == 0)
                        *reinterpret_cast<float2 *>(p.ws_ml + row * 2) = make_float2(m, l);
                }
            }
        }
        at = stop;
        if (at == seg_end) {
            seg = seg_end;
            if (++grp == p.num_groups) {
                grp = 0;
                if (++s < p.num_seqs)
                    tiles = tiles_of(p, s, false);
            }
        }
    }
}

// Merge of the (sequence, group)s that a cut divides: with M = max m_i,
// out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.  One CTA of D threads a
// (cut, row) pair in turn.
template <typename T, bool E4M3, int D>
__global__ void __launch_bounds__(D) block_merge_kernel(const DecodeArgs p, int ctas)
{
    constexpr float kLift = lift_of<typename std::conditional<E4M3, __half, T>::type>();
    griddep_wait();
    griddep_launch_dependents();
    const int rows = p.group << p.heads_log2;
    for (int c = blockIdx.x; c < ctas; c += gridDim.x) {
        const int4 cut = p.cuts[c];
        if (cut.z < 2)
            continue;
        for (int r = blockIdx.y; r < rows; r += gridDim.y) {
            float top = -INFINITY;
            for (int i = 0; i < cut.z; ++i) {
                const int64_t row = (int64_t)(2 * (c + i) + (i == 0)) * rows + r;
                top = fmaxf(top, p.ws_ml[row * 2]);
            }
            const float ref = top == -INFINITY ? 0.f : top;
            float acc = 0.f, l = 0.f;
            for (int i = 0; i < cut.z; ++i) {
                const int64_t row = (int64_t)(2 * (c + i) + (i == 0)) * rows + r;
                const float w = ex2(p.ws_ml[row * 2] - ref);
                l += w * p.ws_ml[row * 2 + 1];
                acc += w * p.ws_o[row * D + threadIdx.x];
            }
            const int64_t row = (int64_t)cut.x * p.num_heads + (int64_t)cut.y * rows + r;
            static_cast<T *>(p.out)[row * D + threadIdx.x] = static_cast<T>(l != 0.f ? acc / l : 0.f);
            if (p.lse && threadIdx.x == 0)
                p.lse[row] = l != 0.f ? (top - kLift + log2f(l)) * kLn2 : -INFINITY;
        }
    }
}

} // namespace block
} // namespace pa
