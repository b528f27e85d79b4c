// C ABI of the 4-bit projection (proj_q4_*): argument checks, packing and
// launches.  See include/proj.h for the contract.
#include <cuda_runtime.h>

#include <new>

#include "proj.h"
#include "proj_host.h"
#include "q4_internal.h"
#include "q4_kernels.cuh"

using namespace projgb;

// How a run of up to 8, 16 or 32 tokens (and of more, in passes) is shared out.
struct Q4Plan {
    int splits = 1;  // CTAs of a cluster, that share a tile's K range
    int per_sm = 1;  // CTAs that an SM takes at once
};

struct proj_q4_s {
    int64_t max_tokens = 0, N = 0, K = 0, group = 0;
    int has_zeros = 0, y_dtype = PROJ_BF16, has_bias = 0;
    int sm_count = 0, device = 0;
    Q4Shape shape{};
    Q4Plan plans[3];
};

namespace {

proj_status_t check_shape(int64_t N, int64_t K, int64_t group, int has_zeros) {
    if (N < 0 || K < 0 || N > kMaxDim || K > kMaxDim || (has_zeros != 0 && has_zeros != 1)) return PROJ_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return PROJ_ERR_UNSUPPORTED;
    return K % group == 0 ? PROJ_OK : PROJ_ERR_INVALID_ARG;
}

int pack_blocks(int64_t items, int sm_count) {
    const int64_t want = (items + 255) / 256;
    return static_cast<int>(want < int64_t(sm_count) * 16 ? want : int64_t(sm_count) * 16);
}

using Q4Kernel = void (*)(Q4Params);
struct Q4Instance {
    Q4Kernel kernel;
    int warps, row_blocks, per_sm, k_steps, red;  // row blocks of a warp; of a CTA; bytes of its join
};

template <int kNT>
Q4Instance instance_nt(int64_t group, bool zeros) {
    using Tile = dev::Q4Tile<kNT>;
    Q4Kernel k;
    if (group == 128)
        k = zeros ? dev::q4_kernel<kNT, 1, true> : dev::q4_kernel<kNT, 1, false>;
    else if (group == 64)
        k = zeros ? dev::q4_kernel<kNT, 2, true> : dev::q4_kernel<kNT, 2, false>;
    else
        k = zeros ? dev::q4_kernel<kNT, 4, true> : dev::q4_kernel<kNT, 4, false>;
    return {k, Tile::kWarps, Tile::kR, Tile::kPerSm, Tile::kKW, Tile::kRed};
}

Q4Instance instance_for(int64_t M, int64_t group, bool zeros) {
    return M <= 8 ? instance_nt<1>(group, zeros) : M <= 16 ? instance_nt<2>(group, zeros) : instance_nt<4>(group, zeros);
}

constexpr int kSmemOfSm = 228 * 1024;  // shared memory of an SM, 1 KiB of it reserved for each CTA
// So much shared memory for a CTA that one more of them does not fit on an SM.
constexpr int smem_for_at_most(int per_sm) { return kSmemOfSm / (per_sm + 1) - 1024 + 256; }

// Clusters that stand on the GPU at once, with `per_sm` CTAs an SM.
int64_t clusters_at_once(const Q4Instance &q, int splits, int per_sm) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute cluster;
    cfg.gridDim = dim3(static_cast<unsigned>(splits));
    cfg.blockDim = dim3(static_cast<unsigned>(32 * q.warps));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem_for_at_most(per_sm));
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = static_cast<unsigned>(splits);
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, q.kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return clusters;
}

Q4Plan plan_for(const Q4Shape &shape, const Q4Instance &q, int sm_count) {
    Q4Plan plan;
    plan.per_sm = q.per_sm;
    const int64_t tiles = shape.row_tiles, steps = (shape.k_blocks + 1) / 2;
    if (tiles == 0 || steps == 0) return plan;
    // CTAs of one K range: as many as stand on the GPU at once, while every
    // warp has a step.  (31 tokens, 12300 rows, 193 tiles: 3 a range 16.2 us, 2
    // 17.9, 1 21.9, and 6, that is two waves, 19.6.)
    int64_t most = q.per_sm * int64_t(sm_count) / tiles;
    if (most > steps / q.k_steps) most = steps / q.k_steps;
    if (most > kQ4MaxSplits) most = kQ4MaxSplits;
    int s = static_cast<int>(most);
    while (s > 1 && clusters_at_once(q, s, q.per_sm) < tiles) --s;
    // With four rounds of K steps or fewer, a join takes more than a split saves
    // that takes no work off the busiest SM (one token, K 2048: 16384 rows 6.0 us
    // whole, 7.1 split; 4096 rows, where it does take work off, 4.0 and 3.5).
    const auto busiest = [&](int64_t ctas) { return (ctas + sm_count - 1) / sm_count; };
    if (s > 1 && steps <= 4 * q.k_steps && busiest(tiles * s) >= s * busiest(tiles)) s = 1;
    if (s > 1) plan.splits = s;
    // As few CTAs an SM as hold them all at once: left to themselves, some SMs
    // take four and others none (one token, 28672 × 8192, 448 tiles: 21.2 us
    // instead of 26.2; 2048 rows, 32 clusters of 8, 4.3 instead of 5.4).
    while (plan.per_sm > 1 && clusters_at_once(q, plan.splits, plan.per_sm - 1) >= tiles) --plan.per_sm;
    return plan;
}

}  // namespace

extern "C" {

proj_status_t proj_q4_packed_bytes(int64_t N, int64_t K, int64_t group, int has_zeros, size_t *bytes) {
    if (!bytes) return PROJ_ERR_INVALID_ARG;
    *bytes = 0;
    const proj_status_t st = check_shape(N, K, group, has_zeros);
    if (st != PROJ_OK) return st;
    const Q4Shape s = q4_shape(N, K, group, has_zeros != 0);
    *bytes = static_cast<size_t>(s.codes_bytes + s.scales_bytes + s.zeros_bytes);
    return PROJ_OK;
}

proj_status_t proj_q4_create(proj_q4_handle_t *out, int64_t max_tokens, int64_t N, int64_t K, int64_t group,
                             int has_zeros, proj_dtype_t y_dtype, int has_bias, void *stream) {
    (void)stream;
    if (!out) return PROJ_ERR_INVALID_ARG;
    *out = nullptr;
    const proj_status_t st = check_shape(N, K, group, has_zeros);
    if (st != PROJ_OK) return st;
    if (max_tokens < 0 || max_tokens > kMaxDim || (has_bias != 0 && has_bias != 1) ||
        (y_dtype != PROJ_BF16 && y_dtype != PROJ_F32))
        return PROJ_ERR_INVALID_ARG;
    if (max_tokens > int64_t(65535) * kQ4MaxTokens) return PROJ_ERR_UNSUPPORTED;  // passes: the grid's second dimension
    const int sms = gb300_sm_count();
    if (sms <= 0) return sms < 0 ? PROJ_ERR_CUDA : PROJ_ERR_UNSUPPORTED;
    for (int64_t m = 8; m <= kQ4MaxTokens; m *= 2)
        if (cudaFuncSetAttribute(instance_for(m, group, has_zeros != 0).kernel,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOfSm - 1024) != cudaSuccess) {
            cudaGetLastError();
            return PROJ_ERR_CUDA;
        }
    proj_q4_s *h = new (std::nothrow) proj_q4_s();
    if (!h) return PROJ_ERR_OUT_OF_MEMORY;
    h->max_tokens = max_tokens;
    h->N = N;
    h->K = K;
    h->group = group;
    h->has_zeros = has_zeros;
    h->y_dtype = y_dtype;
    h->has_bias = has_bias;
    h->sm_count = sms;
    h->device = device_of_handle();
    h->shape = q4_shape(N, K, group, has_zeros != 0);
    for (int i = 0; i < 3; ++i) h->plans[i] = plan_for(h->shape, instance_for(8 << i, group, has_zeros != 0), sms);
    *out = h;
    return PROJ_OK;
}

proj_status_t proj_q4_pack(proj_q4_handle_t h, const void *codes, const void *scales, const void *zeros, void *packed,
                           void *stream) {
    if (!h || !is_current(h->device)) return PROJ_ERR_INVALID_ARG;
    const Q4Shape &s = h->shape;
    if (s.codes_bytes == 0) return PROJ_OK;
    if (!codes || !scales || !packed || (zeros != nullptr) != (h->has_zeros != 0)) return PROJ_ERR_INVALID_ARG;
    if (!aligned16(packed) || reinterpret_cast<uintptr_t>(scales) % 2 != 0) return PROJ_ERR_MISALIGNED;
    if (launch_faulted()) return PROJ_ERR_CUDA;
    uint8_t *at = static_cast<uint8_t *>(packed);
    const int64_t items = s.codes_bytes / 16, pairs = s.scales_bytes / 4;
    dev::q4_pack_codes_kernel<<<pack_blocks(items, h->sm_count), 256, 0, as_stream(stream)>>>(
        static_cast<const uint8_t *>(codes), reinterpret_cast<uint4 *>(at), h->N, h->K, s.k_blocks, items);
    dev::q4_pack_scales_kernel<<<pack_blocks(pairs, h->sm_count), 256, 0, as_stream(stream)>>>(
        static_cast<const uint16_t *>(scales), static_cast<const uint8_t *>(zeros),
        reinterpret_cast<uint32_t *>(at + s.codes_bytes),
        h->has_zeros ? at + s.codes_bytes + s.scales_bytes : nullptr, h->N, s.groups, s.groups_padded, pairs);
    return cudaGetLastError() == cudaSuccess ? PROJ_OK : PROJ_ERR_CUDA;
}

proj_status_t proj_q4_run(proj_q4_handle_t h, int64_t M, const void *X, const void *packed, const void *bias, void *Y,
                          void *stream) {
    if (!h || !is_current(h->device) || M < 0 || M > h->max_tokens) return PROJ_ERR_INVALID_ARG;
    if (M == 0 || h->N == 0) return PROJ_OK;
    if ((bias != nullptr) != (h->has_bias != 0) || !Y) return PROJ_ERR_INVALID_ARG;
    if (h->K > 0 && (!X || !packed)) return PROJ_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(packed) || reinterpret_cast<uintptr_t>(Y) % (h->y_dtype == PROJ_F32 ? 4 : 2) != 0 ||
        reinterpret_cast<uintptr_t>(bias) % 2 != 0)
        return PROJ_ERR_MISALIGNED;
    if (launch_faulted()) return PROJ_ERR_CUDA;
    const uint8_t *at = static_cast<const uint8_t *>(packed);
    Q4Params p{};
    p.M = M;
    p.N = h->N;
    p.K = h->K;
    p.row_tiles = h->shape.row_tiles;
    p.k_blocks = h->shape.k_blocks;
    p.groups_padded = h->shape.groups_padded;
    p.y_f32 = h->y_dtype == PROJ_F32;
    p.y_vec = h->N % 4 == 0 && reinterpret_cast<uintptr_t>(Y) % (p.y_f32 ? 16 : 8) == 0;
    p.X = static_cast<const uint16_t *>(X);
    p.codes = reinterpret_cast<const uint4 *>(at);
    p.scales = reinterpret_cast<const uint32_t *>(at + h->shape.codes_bytes);
    p.zeros = h->has_zeros ? at + h->shape.codes_bytes + h->shape.scales_bytes : nullptr;
    p.bias = static_cast<const uint16_t *>(bias);
    p.Y = Y;

    const Q4Instance q = instance_for(M, h->group, h->has_zeros != 0);
    const Q4Plan &plan = h->plans[M <= 8 ? 0 : M <= 16 ? 1 : 2];
    const int64_t passes = (M + kQ4MaxTokens - 1) / kQ4MaxTokens;
    const int per_sm = passes == 1 ? plan.per_sm : q.per_sm;
    p.splits = static_cast<uint32_t>(plan.splits);
    // Two stages where 16 warps stand on an SM (64 KiB of codes are on their
    // way then, and three are slower), three where fewer do (12 warps: 21.2 us
    // against 21.7 for one token, 28672 × 8192).
    const int tokens = static_cast<int>(M < kQ4MaxTokens ? M : kQ4MaxTokens);
    const int groups = static_cast<int>(128 / h->group);
    const int weights = q.warps * q.row_blocks * (1024 + groups * (32 + (h->has_zeros ? 8 : 0)));
    const int stage = (weights + 255) / 256 * 256 + q.k_steps * tokens * kQ4XPitch;  // X on a 256-byte boundary
    const int fit = (kSmemOfSm / per_sm - 1024) / stage, most = q.warps * per_sm > 12 ? 2 : 3;
    p.stages = fit < 2 ? 2 : fit < most ? fit : most;
    int smem = p.stages * stage;
    if (smem < q.red) smem = q.red;
    if (per_sm < q.per_sm && smem < smem_for_at_most(per_sm)) smem = smem_for_at_most(per_sm);

    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(p.row_tiles * p.splits), static_cast<unsigned>(passes));
    cfg.blockDim = dim3(static_cast<unsigned>(32 * q.warps));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = as_stream(stream);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.splits > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, q.kernel, p) != cudaSuccess) {
        cudaGetLastError();
        return PROJ_ERR_CUDA;
    }
    return PROJ_OK;
}

proj_status_t proj_q4_destroy(proj_q4_handle_t h) {
    delete h;
    return PROJ_OK;
}

}  // extern "C"
