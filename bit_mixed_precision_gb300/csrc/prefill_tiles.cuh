// Tiles of the prefill kernels, both directions: 128 rows of D 16-bit elements as D / 64 halves of 64 columns,
// 128-byte swizzled, their matrix descriptors and their tensor maps.
#pragma once

#include <mutex>

#include "kvq_common.cuh"

namespace kvq {

namespace {

constexpr int kTile = 128;                 // rows per tile (queries or keys)
constexpr uint32_t kHalfBytes = 128 * 128;       // one 128-row x 64-column 128B-swizzled half
constexpr float kLog2e = 1.4426950408889634f;

template <typename T> struct Pack2;
template <> struct Pack2<__half> {
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    }
};
template <> struct Pack2<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    }
};

// K-major operand (rows x 128 elements as two 128B-swizzled 64-column halves):
// descriptor of the 16-element K slice kk (0..7).
__device__ __forceinline__ uint64_t kmajor_desc(uint32_t tile, int kk, uint32_t half = kHalfBytes) {
    return sdesc_sw128(tile + (uint32_t)(kk >> 2) * half + (uint32_t)(kk & 3) * 32u, 16u,
                       1024u);
}

// MN-major operand (128 K-rows of 128 N-elements, two 64-column halves):
// descriptor of K rows 16*kk .. 16*kk+15.  LBO = stride between the N
// halves, SBO = stride between groups of 8 K rows.
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t tile, int kk, uint32_t half = kHalfBytes) {
    return sdesc_sw128(tile + (uint32_t)kk * 16u * 128u, half, 1024u);
}

// ------------------------------------------------------------------ host

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// [rows = BH][T][D] 16-bit tensor, box 64 x box_rows x 1, 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* ptr, int dt, int BH, int T, int D, int box_rows = kTile) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)T, (cuuint64_t)BH};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)T * D * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = enc(m, dt == KVQ_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                     3, const_cast<void*>(ptr), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

}  // namespace

}  // namespace kvq
