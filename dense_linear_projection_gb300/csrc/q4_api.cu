// C ABI of the 4-bit projection (proj_q4_*): argument checks, packing and
// launches.  See include/proj.h for the contract.
#include <cuda_runtime.h>

#include <new>

#include "proj.h"
#include "proj_host.h"
#include "q4_internal.h"
#include "q4_kernels.cuh"

using namespace projgb;

struct proj_q4_s {
    int64_t max_tokens = 0, N = 0, K = 0, group = 0;
    int has_zeros = 0, y_dtype = PROJ_BF16, has_bias = 0;
    int sm_count = 0;
    Q4Shape shape{};
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
    int device = 0;
    cudaDeviceProp prop;
    if (cudaGetDevice(&device) != cudaSuccess || cudaGetDeviceProperties(&prop, device) != cudaSuccess)
        return PROJ_ERR_CUDA;
    if (prop.major != 10 || prop.minor != 3) return PROJ_ERR_UNSUPPORTED;  // built for sm_103a
    proj_q4_s *h = new (std::nothrow) proj_q4_s();
    if (!h) return PROJ_ERR_OUT_OF_MEMORY;
    h->max_tokens = max_tokens;
    h->N = N;
    h->K = K;
    h->group = group;
    h->has_zeros = has_zeros;
    h->y_dtype = y_dtype;
    h->has_bias = has_bias;
    h->sm_count = prop.multiProcessorCount;
    h->shape = q4_shape(N, K, group, has_zeros != 0);
    *out = h;
    return PROJ_OK;
}

proj_status_t proj_q4_pack(proj_q4_handle_t h, const void *codes, const void *scales, const void *zeros, void *packed,
                           void *stream) {
    if (!h) return PROJ_ERR_INVALID_ARG;
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
    if (!h || M < 0 || M > h->max_tokens) return PROJ_ERR_INVALID_ARG;
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
    p.k_blocks = h->shape.k_blocks;
    p.groups_padded = h->shape.groups_padded;
    p.group = static_cast<int32_t>(h->group);
    p.y_f32 = h->y_dtype == PROJ_F32;
    p.X = static_cast<const uint16_t *>(X);
    p.codes = reinterpret_cast<const uint4 *>(at);
    p.scales = reinterpret_cast<const uint32_t *>(at + h->shape.codes_bytes);
    p.zeros = h->has_zeros ? at + h->shape.codes_bytes + h->shape.scales_bytes : nullptr;
    p.bias = static_cast<const uint16_t *>(bias);
    p.Y = Y;
    const dim3 grid(static_cast<unsigned>((h->N + 7) / 8), static_cast<unsigned>(M < 32 ? M : 32));
    dev::q4_kernel<<<grid, 256, 0, as_stream(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? PROJ_OK : PROJ_ERR_CUDA;
}

proj_status_t proj_q4_destroy(proj_q4_handle_t h) {
    delete h;
    return PROJ_OK;
}

}  // extern "C"
