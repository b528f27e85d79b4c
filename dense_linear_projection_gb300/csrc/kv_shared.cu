// C ABI of attention over a shared prefix (proj_kv_attend_shared): argument checks and launches.
// See include/proj.h for the contract.
#include <cuda.h>
#include <cuda_runtime.h>

#include "kv_host.cuh"
#include "kv_prefix.cuh"
#include "proj.h"

using namespace projgb;

namespace {

using PrefixKernel = void (*)(KvPrefixParams, CUtensorMap, CUtensorMap);
using CombineKernel = void (*)(KvCombineParams);
struct PrefixInstance {
    PrefixKernel kernel;
    CombineKernel combine, combine_many;  // for a few parts of a unit, for many
    int smem, tokens, part, columns;  // shared memory, tokens of a tile, floats of a part, elements of a row in it
};

template <bool kE4m3, int kDim>
PrefixInstance prefix_of() {
    using Shape = dev::PrefixShape<kE4m3, kDim>;
    return {dev::kv_prefix_kernel<kE4m3, kDim>, dev::kv_combine_kernel<kDim, 1>, dev::kv_combine_kernel<kDim, dev::kCombineMost>, Shape::kSmem, Shape::kTokens, Shape::kPart, kDim};
}

template <bool kE4m3>
PrefixInstance prefix_for(int head_dim) {
    return head_dim <= 64 ? prefix_of<kE4m3, 64>() : head_dim <= 128 ? prefix_of<kE4m3, 128>() : prefix_of<kE4m3, 256>();
}

PrefixInstance prefix_for(const proj_kv_s *h) {
    return h->d.kv_dtype == PROJ_E4M3 ? prefix_for<true>(h->d.head_dim) : prefix_for<false>(h->d.head_dim);
}

// How the prefix's products are cut, and where the parts lie in the workspace:
// every row's own maximum and sum, its own output, then the prefix's parts.
struct SharedPlan {
    PrefixInstance instance;
    int64_t row_tiles = 0, tiles = 0, combine_blocks = 0;
    int ctas = 0;
    size_t tops = 0, own = 0, parts = 0;
};

// False where the rows of a key head are too many, or all of them for the join's grid (and for
// the prefix's 32-bit numbers of units, of 128 rows where a block of the join has 8).
bool shared_plan(const proj_kv_s *h, int64_t sequences, int64_t prefix_len, SharedPlan &s) {
    const proj_kv_desc_t &d = h->d;
    s.instance = prefix_for(h);
    const int64_t rows = sequences * (d.q_heads / d.kv_heads);
    s.combine_blocks = d.kv_heads * ((rows + dev::kCombineRows - 1) / dev::kCombineRows);
    if (rows > kMaxDim - 256 || s.combine_blocks > kMaxDim) return false;
    s.row_tiles = (rows + dev::kPrefixRows - 1) / dev::kPrefixRows;
    s.tiles = (prefix_len + s.instance.tokens - 1) / s.instance.tokens;
    const int64_t units = d.kv_heads * s.row_tiles;
    s.ctas = static_cast<int>(units * s.tiles < h->sm_count ? units * s.tiles : h->sm_count);
    s.tops = rounded(static_cast<size_t>(sequences) * d.q_heads * sizeof(float2));
    s.own = rounded(static_cast<size_t>(sequences) * d.q_heads * d.head_dim * 4);
    s.parts = static_cast<size_t>(units + s.ctas) * s.instance.part * 4;
    return true;
}

}  // namespace

namespace projgb {
bool prepare_shared(const proj_kv_s *h) {
    const PrefixInstance a = prefix_for(h);
    if (prepare_attend<kAttendPart>(h) &&
        cudaFuncSetAttribute(a.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, a.smem) == cudaSuccess)
        return true;
    cudaGetLastError();
    return false;
}
}  // namespace projgb

extern "C" {

proj_status_t proj_kv_shared_workspace(proj_kv_handle_t h, int64_t sequences, int64_t prefix_len, size_t *bytes) {
    if (!bytes) return PROJ_ERR_INVALID_ARG;
    *bytes = 0;
    SharedPlan s;
    if (!h || sequences < 0 || sequences > h->d.max_sequences || prefix_len < 0 || prefix_len > kMaxDim - 4095) return PROJ_ERR_INVALID_ARG;
    if (!shared_plan(h, sequences, prefix_len, s)) return PROJ_ERR_UNSUPPORTED;
    if (sequences > 0 && prefix_len > 0) *bytes = s.tops + s.own + s.parts;
    return PROJ_OK;
}

proj_status_t proj_kv_attend_shared(proj_kv_handle_t h, int64_t sequences, const void *q, int64_t q_stride,
                                    const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
                                    const int32_t *prefix_pages, int64_t prefix_width, int64_t prefix_len,
                                    const int32_t *page_table, int64_t table_width, const int32_t *seq_lens, float scale,
                                    void *workspace, void *out, int64_t out_stride, float *lse, void *stream) {
    KvAttendParams p{};
    const proj_status_t st = attend_params(h, {sequences, q, q_stride, k_cache, v_cache, k_scale, v_scale, page_table, table_width,
                                               seq_lens, 0, scale, out, out_stride, lse}, p);
    if (st != PROJ_OK) return st;
    if (!fits_table(prefix_width, h->d.page_size) || prefix_len < 0 || prefix_len > prefix_width * h->d.page_size)
        return PROJ_ERR_INVALID_ARG;
    if (sequences == 0) return PROJ_OK;
    if (prefix_len == 0)
        return proj_kv_attend(h, sequences, q, q_stride, k_cache, v_cache, k_scale, v_scale, page_table, table_width, seq_lens, 0,
                              scale, out, out_stride, lse, stream);
    if (!prefix_pages || !workspace || !k_cache || !v_cache) return PROJ_ERR_INVALID_ARG;
    if (!aligned16(workspace) || reinterpret_cast<uintptr_t>(prefix_pages) % 4 != 0) return PROJ_ERR_MISALIGNED;
    SharedPlan s;
    if (!shared_plan(h, sequences, prefix_len, s)) return PROJ_ERR_UNSUPPORTED;
    uint8_t *at = static_cast<uint8_t *>(workspace);

    KvPrefixParams x{};
    x.cache = view_of(h, prefix_pages, prefix_width);
    x.sequences = sequences;
    x.prefix = prefix_len;
    x.q = p.q;
    x.q_stride = q_stride;
    x.k_cache = k_cache;
    x.v_cache = v_cache;
    x.k_scale = k_scale;
    x.v_scale = v_scale;
    x.scale = scale;
    x.group = p.group;
    x.row_tiles = s.row_tiles;
    x.tiles = s.tiles;
    x.partials = reinterpret_cast<float *>(at + s.tops + s.own);
    x.status = h->status;
    x.wait_limit_ns = dev::kPrefixWaitNs;
    x.fault_place = -1;
    if (h->fault_place >= 0) {
        x.wait_limit_ns = dev::kPrefixFaultNs;
        x.fault_place = h->fault_place;
        h->fault_place = -1;  // (the next calls are as ever)
    }
    // Boxes of whole 8-row groups of the swizzle, within a loading warp's tokens.  Without TMA
    // (other page sizes, strides that a tensor map cannot have): 16-byte copies.
    CUtensorMap maps[2] = {};
    const int32_t most = s.instance.tokens / dev::kPrefixLoadWarps;
    for (x.box = most; x.box >= 8 && h->d.page_size % x.box != 0;) x.box /= 2;
    const proj_kv_desc_t &d = h->d;
    const uint64_t dims[4] = {static_cast<uint64_t>(d.head_dim), static_cast<uint64_t>(d.page_size), static_cast<uint64_t>(d.kv_heads),
                              static_cast<uint64_t>(d.num_pages)};
    const uint64_t strides[3] = {static_cast<uint64_t>(d.token_stride) * h->elem, static_cast<uint64_t>(d.head_stride) * h->elem,
                                 static_cast<uint64_t>(d.page_stride) * h->elem};
    const uint32_t inner = h->elem == 2 ? 64 : s.instance.columns;
    if (x.box < 8 || !encode_4d(&maps[0], k_cache, h->elem, dims, strides, inner, x.box) ||
        !encode_4d(&maps[1], v_cache, h->elem, dims, strides, inner, x.box))
        x.box = 0;
    const proj_status_t first = launch(s.instance.kernel, dim3(static_cast<unsigned>(s.ctas)), dev::kPrefixThreads,
                                       static_cast<size_t>(s.instance.smem), stream, x, maps[0], maps[1]);
    if (first != PROJ_OK) return first;

    p.top = reinterpret_cast<float2 *>(at);
    p.out32 = reinterpret_cast<float *>(at + s.tops);
    p.lse = nullptr;  // of all tokens: the join's
    const proj_status_t second = launch_attend<kAttendPart>(h, p, stream);
    if (second != PROJ_OK) return second;

    KvCombineParams c{};
    c.partials = x.partials;
    c.top = p.top;
    c.out32 = p.out32;
    c.sequences = sequences;
    c.row_tiles = s.row_tiles;
    c.tiles = s.tiles;
    c.ctas = s.ctas;
    c.kv_heads = h->d.kv_heads;
    c.group = p.group;
    c.head_dim = h->d.head_dim;
    c.out = p.out;
    c.out_stride = out_stride;
    c.lse = lse;
    const int64_t units = h->d.kv_heads * s.row_tiles;
    const bool few = (s.ctas + units - 1) / units + 1 <= dev::kCombineFew;
    return launch(few ? s.instance.combine : s.instance.combine_many, dim3(static_cast<unsigned>(s.combine_blocks)),
                  dev::kCombineThreads * (few ? 1 : dev::kCombineMost), 0, stream, c);
}

}  // extern "C"
