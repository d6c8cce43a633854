// Varlen sequences cut into pieces of equal size, and tensor maps of (token, head, dim) tensors: what the chunked kernels share.
#pragma once

#include "ccv_layer.h"
#include "ccv_tcgen05.cuh"

namespace ccv {

// Piece (chunk, or segment) j of sequence i is in slot first_slot(i) + j.  floor(s / u) + i, with u the tokens of a piece,
// leaves every sequence room for its ceil(n / u) pieces, needs no sum over the lengths, and total / u + batch slots in all.
__device__ __forceinline__ int first_slot(int start, int i, int unit) { return start / unit + i; }

// The sequence of a slot, the last i with first_slot(i) <= slot, and its tokens; by a whole warp, 32 candidates at a time.
__device__ __forceinline__ void find_sequence(const int32_t *query_start_loc, int batch, int slot, int unit, int lane, int &seq, int &start,
                                              int &end) {
    int lo = 0, hi = batch;  // the answer is in [lo, hi)
    do {
        const int step = (hi - lo + 31) / 32;
        const int i = min(lo + lane * step, batch), next = max(i, min(i + step, hi));
        const int at = query_start_loc[i], to = query_start_loc[next];
        const bool below = i < hi && first_slot(at, i, unit) <= slot;
        const int last = 31 - __clz(__ballot_sync(kFullMask, below) | 1);
        lo += last * step;
        hi = min(hi, lo + step);
        start = __shfl_sync(kFullMask, at, last);
        end = __shfl_sync(kFullMask, to, last);
    } while (hi - lo > 1);
    seq = lo;
}

__device__ __forceinline__ bool sequence_ok(int s, int e, int total) { return s >= 0 && e >= s && e <= total; }

// ------------------------------------------------------------ host side ----

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// CUDA's encoder, looked up once (the library links none of libcuda's symbols).
inline EncodeTiled tensor_map_encoder() {
    static const EncodeTiled fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

// Map (dim, head, token) of a bf16 tensor with boxes of 64 values x `rows` tokens; false where its strides do not allow one.
inline bool encode_heads_map(CUtensorMap *map, const ccv_heads_view &v, int dim, int heads, int tokens, int rows) {
    const cuuint64_t size[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
    const cuuint64_t stride[2] = {static_cast<cuuint64_t>(v.stride_head) * 2, static_cast<cuuint64_t>(v.stride_tok) * 2};
    if ((stride[0] == 0 && heads > 1) || stride[1] == 0 || stride[0] >= 1ull << 40 || stride[1] >= 1ull << 40) return false;
    const cuuint64_t strides[2] = {heads > 1 ? stride[0] : 16, stride[1]};
    const cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(rows)}, one[3] = {1, 1, 1};
    const EncodeTiled encode = tensor_map_encoder();
    return encode != nullptr &&
           encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(v.data), size, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace ccv
