// pa_block_decode.cu -- C entries of the decode over an e4m3 pool with block
// scales and over listed blocks; compiled once per type of q
// (PA_INST_DTYPE: 0 fp16 with the entries, 1 bf16).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "pa.h"
#include "pa_block_decode.cuh"

namespace pa {
namespace block {

// `nearest`: for an e4m3 pool (block_decode_kernel); a 16-bit one always is.
cudaError_t launch_block_decode_f16(bool e4m3, bool nearest, int head_size, const CUtensorMap &map,
                                    const DecodeArgs &p, int ctas, cudaStream_t s);
cudaError_t launch_block_decode_bf16(bool e4m3, bool nearest, int head_size, const CUtensorMap &map,
                                     const DecodeArgs &p, int ctas, cudaStream_t s);

int block_decode_resident_f16(bool e4m3, int head_size, int warps, bool hand_over);
int block_decode_resident_bf16(bool e4m3, int head_size, int warps, bool hand_over);

// What is looked up once for each device.  Host threads that come at the same
// time look up, and store, the same; a device past the array looks up each time.
constexpr int kKnownDevices = 64;

// The kernel's shared memory is allowed once a device (it takes most of an SM's).
template <typename T, bool E4M3, int D, bool NEAREST> static cudaError_t prepare()
{
    static std::atomic<bool> ready[kKnownDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const bool known = dev < kKnownDevices;
    if (e == cudaSuccess && !(known && ready[dev])) {
        e = cudaFuncSetAttribute(block_decode_kernel<T, E4M3, D, NEAREST>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 decode_smem<E4M3, D>(kWarps, true));
        if (known)
            ready[dev] = e == cudaSuccess;
    }
    return e;
}

// CTAs of so many warps that an SM of the current device holds at once (both
// kernels of an e4m3 pool take as many registers); 0 on an error.
template <typename T, bool E4M3, int D> static int resident(int warps, bool hand_over)
{
    static std::atomic<int> seen[kKnownDevices][kWarps + 1][2];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return 0;
    const bool known = dev < kKnownDevices;
    int now = known ? seen[dev][warps][hand_over].load() : 0;
    if (!now) {
        if (prepare<T, E4M3, D, !E4M3>() != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                &now, block_decode_kernel<T, E4M3, D, !E4M3>, 32 * warps,
                decode_smem<E4M3, D>(warps, hand_over)) != cudaSuccess)
            return 0;
        if (known)
            seen[dev][warps][hand_over] = now;
    }
    return now;
}

template <typename T, bool E4M3, int D, bool NEAREST>
static cudaError_t launch(const CUtensorMap &map, const DecodeArgs &p, int ctas, cudaStream_t s)
{
    const int warps = p.heads * p.tiles_at_once;
    const int smem = decode_smem<E4M3, D>(warps, p.tiles_at_once > 1);
    cudaError_t e = prepare<T, E4M3, D, NEAREST>();
    if (e != cudaSuccess)
        return e;
    e = launch_after_previous(block_decode_kernel<T, E4M3, D, NEAREST>, dim3(ctas),
                              dim3(32 * warps), smem, s, map, p);
    if (e != cudaSuccess)
        return e;
    if (p.whole)
        return cudaSuccess;
    // A warp for each query row of the most cuts there can be, as far as two CTAs
    // an SM go.
    const int rows = p.group * p.heads;
    const int merge = std::min((ctas * rows + kMergeWarps - 1) / kMergeWarps, 2 * kMaxCtas / 3);
    return launch_after_previous(block_merge_kernel<T, E4M3, D>, dim3(merge),
                                 dim3(32 * kMergeWarps), 0, s, p, ctas);
}

template <typename T, int D>
static cudaError_t launch_of(bool e4m3, bool nearest, const CUtensorMap &map, const DecodeArgs &p,
                             int ctas, cudaStream_t s)
{
    return !e4m3     ? launch<T, false, D, true>(map, p, ctas, s)
           : nearest ? launch<T, true, D, true>(map, p, ctas, s)
                     : launch<T, true, D, false>(map, p, ctas, s);
}

#if PA_INST_DTYPE == 1
cudaError_t launch_block_decode_bf16(bool e4m3, bool nearest, int head_size, const CUtensorMap &map,
                                     const DecodeArgs &p, int ctas, cudaStream_t s)
{
    return head_size == 128 ? launch_of<__nv_bfloat16, 128>(e4m3, nearest, map, p, ctas, s)
                            : launch_of<__nv_bfloat16, 64>(e4m3, nearest, map, p, ctas, s);
}

int block_decode_resident_bf16(bool e4m3, int head_size, int warps, bool hand_over)
{
    if (head_size == 128)
        return e4m3 ? resident<__nv_bfloat16, true, 128>(warps, hand_over)
                    : resident<__nv_bfloat16, false, 128>(warps, hand_over);
    return e4m3 ? resident<__nv_bfloat16, true, 64>(warps, hand_over)
                : resident<__nv_bfloat16, false, 64>(warps, hand_over);
}
#else
cudaError_t launch_block_decode_f16(bool e4m3, bool nearest, int head_size, const CUtensorMap &map,
                                    const DecodeArgs &p, int ctas, cudaStream_t s)
{
    return head_size == 128 ? launch_of<__half, 128>(e4m3, nearest, map, p, ctas, s)
                            : launch_of<__half, 64>(e4m3, nearest, map, p, ctas, s);
}

int block_decode_resident_f16(bool e4m3, int head_size, int warps, bool hand_over)
{
    if (head_size == 128)
        return e4m3 ? resident<__half, true, 128>(warps, hand_over)
                    : resident<__half, false, 128>(warps, hand_over);
    return e4m3 ? resident<__half, true, 64>(warps, hand_over)
                : resident<__half, false, 64>(warps, hand_over);
}

static bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

static size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// The pool as TMA sees it: 128-byte columns (64-byte ones for e4m3 rows of 64),
// token rows, columns of a head's row, heads, planes.  A box is both planes of
// a 16-row tile of one head, swizzled.  Rows past the pool read as zeros.
static bool make_map(CUtensorMap *map, const void *pool, bool e4m3, int dtype, int num_blocks,
                     int block_size, int num_kv_heads, int head_size)
{
    cudaError_t err;
    auto fn = encode_fn(&err);
    if (!fn)
        return false;
    const cuuint64_t es = e4m3 ? 1 : 2, row = head_size * es, rows = (cuuint64_t)num_blocks * block_size;
    const cuuint64_t wide = row > 128 ? 128 : row, all = row * num_kv_heads;
    const CUtensorMapDataType type = e4m3               ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUtensorMapSwizzle swizzle =
        wide == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    CUresult r;
    if (row > 128) {
        const cuuint64_t dims[5] = {wide / es, rows, row / wide, (cuuint64_t)num_kv_heads, 2};
        const cuuint64_t strides[4] = {all, wide, row, rows * all};
        const cuuint32_t box[5] = {(cuuint32_t)(wide / es), kTile, (cuuint32_t)(row / wide), 1, 2};
        r = fn(map, type, 5, const_cast<void *>(pool), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    } else {
        const cuuint64_t dims[4] = {wide / es, rows, (cuuint64_t)num_kv_heads, 2};
        const cuuint64_t strides[3] = {all, row, rows * all};
        const cuuint32_t box[4] = {(cuuint32_t)(wide / es), kTile, 1, 2};
        r = fn(map, type, 4, const_cast<void *>(pool), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    }
    return r == CUDA_SUCCESS;
}

// Tiles that the warps of a CTA of `heads` heads take at a time: 1, 2, 4 or 8.
static int tiles_at_once(int heads)
{
    int t = 1;
    while (2 * t * heads <= kWarps)
        t *= 2;
    return t;
}

// CTAs of a launch that cuts, at most: 456, three for each of GB300's 152 SMs,
// where its warps are few or its tiles small, else two.
static int max_ctas(int heads, int head_size)
{
    return heads <= 5 || head_size == 64 ? kMaxCtas : kMaxCtas / 3 * 2;
}

// Workspace: the cuts, then two partial states of each CTA.
struct Layout {
    size_t ml, o, total;
};

static Layout layout(int num_heads, int num_kv_heads, int head_size)
{
    const int heads = heads_together(num_kv_heads);
    const size_t rows = (size_t)max_ctas(heads, head_size) * 2 * (num_heads / num_kv_heads) * heads;
    Layout w;
    w.ml = round_up(kMaxCtas * sizeof(int4));
    w.o = w.ml + round_up(rows * 2 * sizeof(float));
    w.total = w.o + round_up(rows * head_size * sizeof(float));
    return w;
}

static pa_status decode(void *out, float *lse, const void *q, const void *kv_cache,
                        const float *kv_scales, const int32_t *tables, const int32_t *seq_lens,
                        const int32_t *lists, const int32_t *list_lens, int num_seqs,
                        int num_heads, int num_kv_heads, int head_size, int block_size,
                        int num_blocks, int max_blocks, int max_listed, float scale,
                        pa_dtype dtype, int64_t len_cap, void *workspace, size_t workspace_bytes,
                        void *stream)
{
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_size <= 0 ||
        block_size <= 0 || num_blocks <= 0 || max_blocks <= 0 || !isfinite(scale) ||
        num_heads % num_kv_heads != 0)
        return PA_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!out || !q || !kv_cache || !tables || !seq_lens))
        return PA_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(q, 16) || !aligned(kv_cache, 16) ||
        !aligned(kv_scales, 4) || !aligned(tables, 4) || !aligned(seq_lens, 4) ||
        !aligned(lists, 4) || !aligned(list_lens, 4))
        return PA_ERR_INVALID_ARG;
    const int group = num_heads / num_kv_heads;
    if ((head_size != 64 && head_size != 128) || (block_size != 16 && block_size != 32) ||
        (group != 1 && group != 2 && group != 4 && group != 8) ||
        (dtype != PA_FP16 && dtype != PA_BF16))
        return PA_ERR_UNSUPPORTED;
    if ((int64_t)num_blocks * block_size >= (int64_t)INT32_MAX ||
        (int64_t)max_blocks * block_size >= (int64_t)INT32_MAX || num_kv_heads > 65535 ||
        num_seqs > 65535)
        return PA_ERR_UNSUPPORTED;
    // tiles are counted in 32 bits
    const int64_t cap = std::min<int64_t>(len_cap, (int64_t)max_blocks * block_size);
    const int64_t most = lists ? (int64_t)max_listed * (block_size / kTile) : cap / kTile + 1;
    if (most * num_seqs > INT32_MAX / 2 / num_kv_heads)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0)
        return PA_OK;
    const Layout w = layout(num_heads, num_kv_heads, head_size);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < w.total)
        return PA_ERR_WORKSPACE;
    cudaError_t e;
    const int sms = sm_count(&e);
    if (!sms)
        return PA_ERR_CUDA;
    // Cut into equal runs of the largest head groups, or one CTA for each
    // (sequence, head group) of some size: whichever takes less by these costs,
    // in tiles of a warp (about 0.35 us): what a launch takes besides its tiles
    // 10, a merge 11, each further (sequence, group) of a CTA 6, fitted to what
    // was measured.  Cut runs take the tiles there are, whole ones those of the
    // longest sequence.  The lengths are on the device, so a sequence is taken for
    // half of max_seq_len on average, as in a batch of requests of any age, and a
    // list for full.  (Cut and whole: 152 sequences of 41 tokens, 5 kv heads 33
    // and 5.6 us; 64 lists of 64 16-token blocks, 8 kv heads 32.7 and 28.4 us; 37
    // sequences of 3120 to 24966 tokens, 6 kv heads of 64 49 and 158 us.)  Where
    // all are as long as max_seq_len the cut is priced too low: at worst 256
    // sequences of 512 tokens, 64 query and 8 kv heads, are cut in 55.2 us and
    // would take 47.0 whole; 18 of 120 such batches lose more than 3 % by it.
    // tiles of a sequence, for this choice: a list rarely names a block twice
    const int64_t usual = std::min(most, cap / kTile + 1);
    int heads = heads_together(num_kv_heads), at_once = tiles_at_once(heads);
    const auto resident = dtype == PA_BF16 ? block_decode_resident_bf16 : block_decode_resident_f16;
    const int per_sm = resident(kv_scales != nullptr, head_size, heads * at_once, at_once > 1);
    if (!per_sm)
        return PA_ERR_CUDA;
    const int slots = std::min(per_sm * sms, max_ctas(heads, head_size));
    const int64_t groups = (int64_t)num_seqs * (num_kv_heads / heads);
    double best = 21 + (double)groups * usual * (lists ? 1 : 0.5) / ((double)slots * at_once) +
                  6.0 * groups / slots;
    bool whole = false;
    for (int h = heads; h >= 1; --h) {
        if (num_kv_heads % h)
            continue;
        const int64_t ctas = (int64_t)num_seqs * (num_kv_heads / h);
        const int t = tiles_at_once(h);
        const int64_t once = (int64_t)resident(kv_scales != nullptr, head_size, h * t, t > 1) * sms;
        if (!once)
            return PA_ERR_CUDA;
        const double cost = (double)((ctas + once - 1) / once) * (10 + (usual + t - 1) / t);
        if (cost < best && ctas <= INT32_MAX) {
            best = cost;
            whole = true;
            heads = h;
            at_once = t;
        }
    }
    const int64_t tiles = most * num_seqs * (num_kv_heads / heads);
    DecodeArgs p = {};
    p.err = device_error_word(&e);
    if (!p.err)
        return PA_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    p.out = out;
    p.lse = lse;
    p.q = q;
    p.scales = kv_scales;
    p.tables = tables;
    p.seq_lens = seq_lens;
    p.lists = lists;
    p.list_lens = list_lens;
    p.cuts = reinterpret_cast<int4 *>(ws);
    p.ws_ml = reinterpret_cast<float *>(ws + w.ml);
    p.ws_o = reinterpret_cast<float *>(ws + w.o);
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = group;
    p.heads = heads;
    p.tiles_at_once = at_once;
    p.num_groups = num_kv_heads / heads;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks;
    p.block_log2 = block_size == 16 ? 4 : 5;
    p.max_listed = max_listed;
    p.len_cap = (int)cap;
    p.qscale = scale * 1.4426950408889634f;
    p.whole = whole;
    // Else equal runs, of at least kMinRun tiles a warp.
    const int64_t ctas = whole ? (int64_t)num_seqs * p.num_groups
                               : std::min<int64_t>(tiles / (kMinRun * at_once) + 1, slots);
    // the most tiles that a warp can have of one (sequence, head group)
    const int64_t run = whole ? most : std::min(most, (tiles + ctas - 1) / ctas);
    const bool nearest = run > (int64_t)kTruncated * at_once;
    alignas(64) CUtensorMap map;
    if (!make_map(&map, kv_cache, kv_scales != nullptr, dtype, num_blocks, block_size,
                  num_kv_heads, head_size))
        return PA_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const auto launch = dtype == PA_BF16 ? launch_block_decode_bf16 : launch_block_decode_f16;
    e = launch(kv_scales != nullptr, nearest, head_size, map, p, (int)ctas, st);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
#endif

} // namespace block
} // namespace pa

#if PA_INST_DTYPE == 0
using namespace pa;
using namespace pa::block;

extern "C" {

size_t pa_block_decode_workspace_size(int num_heads, int num_kv_heads, int head_size)
{
    if (num_heads <= 0 || num_kv_heads <= 0 || head_size <= 0 || num_heads % num_kv_heads)
        return 0;
    return layout(num_heads, num_kv_heads, head_size).total;
}

pa_status pa_decode_fp8_block(void *out, float *lse, const void *q, const void *kv_cache,
                              const float *kv_scales, const int32_t *block_tables,
                              const int32_t *seq_lens, int num_seqs, int num_heads,
                              int num_kv_heads, int head_size, int block_size, int num_blocks,
                              int max_blocks_per_seq, float scale, pa_dtype dtype,
                              int max_seq_len, void *workspace, size_t workspace_bytes,
                              void *stream)
{
    if (max_seq_len < 0 || (num_seqs > 0 && !kv_scales))
        return PA_ERR_INVALID_ARG;
    return decode(out, lse, q, kv_cache, kv_scales, block_tables, seq_lens, nullptr, nullptr,
                  num_seqs, num_heads, num_kv_heads, head_size, block_size, num_blocks,
                  max_blocks_per_seq, 0, scale, dtype, max_seq_len, workspace, workspace_bytes,
                  stream);
}

pa_status pa_decode_sparse(void *out, float *lse, const void *q, const void *kv_cache,
                           const float *kv_scales, const int32_t *block_tables,
                           const int32_t *seq_lens, const int32_t *block_lists,
                           const int32_t *list_lens, int num_seqs, int num_heads,
                           int num_kv_heads, int head_size, int block_size, int num_blocks,
                           int max_blocks_per_seq, int max_selected, float scale, pa_dtype dtype,
                           void *workspace, size_t workspace_bytes, void *stream)
{
    if (max_selected <= 0 || (num_seqs > 0 && (!block_lists || !list_lens)))
        return PA_ERR_INVALID_ARG;
    return decode(out, lse, q, kv_cache, kv_scales, block_tables, seq_lens, block_lists, list_lens,
                  num_seqs, num_heads, num_kv_heads, head_size, block_size, num_blocks,
                  max_blocks_per_seq, max_selected, scale, dtype,
                  (int64_t)max_blocks_per_seq * block_size, workspace, workspace_bytes, stream);
}

} // extern "C"
#endif
