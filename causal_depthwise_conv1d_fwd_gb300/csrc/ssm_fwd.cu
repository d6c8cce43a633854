// Selective state space scan over varlen sequences (prefill): the choice of form, and contiguous copies where the chunked one
// needs them.
#include <cstdlib>
#include <cstring>

#include "ssm_fwd.cuh"

namespace ccv {
namespace {

// ------------------------------------------------------------------ copies ----

// dst (tokens, heads, padded dim) from a view with any strides, by tiles of 32 tokens x 32 channels: read along the axis whose
// stride is smaller, written along channels.
__global__ void __launch_bounds__(256) ssm_copy_kernel(ccv_heads_view v, uint16_t *dst, int tokens, int heads, int dim, int padded, int along_tokens) {
    __shared__ uint16_t tile[32][33];
    wait_prior_grid();
    release_next_grid();
    const int width = heads * padded, across = (width + 31) / 32;
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int t0 = blockIdx.x / across * 32, c0 = blockIdx.x % across * 32;
    const uint16_t *src = static_cast<const uint16_t *>(v.data);
    for (int i = y; i < 32; i += 8) {
        const int t = along_tokens ? x : i, c = along_tokens ? i : x;
        const int h = (c0 + c) / padded, d = (c0 + c) % padded;
        uint16_t w = 0;
        if (t0 + t < tokens && h < heads && d < dim) w = src[(t0 + t) * v.stride_tok + h * v.stride_head + d * v.stride_dim];
        tile[t][c] = w;
    }
    __syncthreads();
    for (int i = y; i < 32; i += 8)
        if (t0 + i < tokens && c0 + x < width) dst[static_cast<int64_t>(t0 + i) * width + c0 + x] = tile[i][x];
}

int padded_dim(int dim) { return (dim + 7) / 8 * 8; }
int64_t copy_bytes(int64_t tokens, int heads, int dim) { return (tokens * heads * padded_dim(dim) * 2 + 127) / 128 * 128; }

int copy_view(ccv_heads_view &v, uint8_t *to, int tokens, int heads, int dim, cudaStream_t stream) {
    const int padded = padded_dim(dim);
    const int64_t blocks = (static_cast<int64_t>(tokens) + 31) / 32 * ((static_cast<int64_t>(heads) * padded + 31) / 32);
    if (blocks > 0x7fffffff || static_cast<int64_t>(heads) * padded > 0x7fffffff) return CCV_ERR_SIZE;
    const int status = launch_pdl(ssm_copy_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, v,
                                  reinterpret_cast<uint16_t *>(to), tokens, heads, dim, padded, v.stride_tok < v.stride_dim ? 1 : 0);
    v = ccv_heads_view{to, 0, static_cast<int64_t>(heads) * padded, padded, 1};
    return status;
}

// Whether tensor maps take the view as it is.
bool mapped(const ccv_heads_view &v, int heads) {
    return aligned16(v.data) && v.stride_dim == 1 && v.stride_tok > 0 && v.stride_tok % 8 == 0 &&
           (heads == 1 || (v.stride_head > 0 && v.stride_head % 8 == 0));
}

// -------------------------------------------------------------------- form ----

enum Form { kRecurrent, kChunked, kScan };

// Up to 8 tokens a sequence the recurrent form, whose blocks read and write a state as they are and start at once: 16 (128)
// sequences of 8 tokens of 32 heads of 64 channels with 128 states take 21 (123) us, chunked 27 (166), and of 16 tokens 35 (215)
// and 27 (168); 128 of 8 tokens of 4096 channels with 16 states 51, by the scan 126 (a single one 10 and 8).  Above that the
// tensor cores where one decay a head and the states allow it: 8 x 500 tokens of 32 heads with 16 states take 34 us and by the
// scan 118, with 64 35 and 214; heads of 8 channels (256 of them, whose tiles are an eighth full) 197 and 442 (but 32 x 60 tokens
// 314 and 232), and of 4 (512) 450 and 662, but 32 x 60 tokens of those 649 and 332.  The average is all that the sizes tell: 255
// sequences of one token and one of 1700, 32 heads, go token by token and take 1263 us, by the chunked form 358.
// CCV_SSM_PATH=recurrent, =chunked or =scan, read at each call, forces a form where it can run (for testing and tuning).
Form choose(int total_tokens, int batch, int head_dim, int dim_state, int a_per_state) {
    const char *path = std::getenv("CCV_SSM_PATH");
    const bool chunks = ssm_chunked_dims(dim_state, a_per_state);
    if (path != nullptr && std::strcmp(path, "recurrent") == 0) return kRecurrent;
    if (path != nullptr && std::strcmp(path, "scan") == 0) return kScan;
    if (path != nullptr && std::strcmp(path, "chunked") == 0 && chunks) return kChunked;
    if (total_tokens <= static_cast<int64_t>(8) * batch) return kRecurrent;
    return chunks && head_dim >= 8 ? kChunked : kScan;
}

}  // namespace
}  // namespace ccv

extern "C" int64_t ssm_fwd_workspace(int total_tokens, int batch, int num_heads, int num_groups, int head_dim, int dim_state,
                                     int a_per_state, int copies) {
    using namespace ccv;
    if (total_tokens <= 0 || total_tokens > (1 << 30) || batch <= 0 || num_heads <= 0 || num_groups <= 0 || num_heads % num_groups != 0 ||
        head_dim <= 0 || head_dim > kSsmMaxDim || dim_state <= 0 || dim_state > kSsmMaxStates)
        return 0;
    const Form form = choose(total_tokens, batch, head_dim, dim_state, a_per_state);
    if (form == kRecurrent) return 0;
    if (form == kScan)
        return ssm_scan_workspace(total_tokens, batch, num_heads, head_dim, dim_state,
                                  ssm_scan_segments(total_tokens, batch, num_heads, num_groups, head_dim, dim_state));
    int64_t bytes = ssm_chunked_workspace(total_tokens, batch, num_heads, head_dim,
                                          ssm_chunked_segments(total_tokens, batch, num_heads, head_dim));
    if (copies) bytes += copy_bytes(total_tokens, num_heads, head_dim) + 2 * copy_bytes(total_tokens, num_groups, dim_state);
    return bytes;
}

extern "C" int ssm_fwd(const ccv_ssm_args *args, const int32_t *query_start_loc, int batch, const int32_t *cache_indices,
                       const uint8_t *has_initial_state, int total_tokens, void *workspace, int64_t workspace_bytes, int *err_count,
                       ccv_stream_t stream) {
    using namespace ccv;
    if (batch < 0 || total_tokens < 0 || total_tokens > (1 << 30)) return CCV_ERR_SIZE;
    int status = ssm_check(args, 1, total_tokens);
    if (status != CCV_OK) return status;
    if (args->state == nullptr && has_initial_state != nullptr) return CCV_ERR_ARGUMENT;
    if (batch == 0 || total_tokens == 0 || args->num_heads == 0 || args->head_dim == 0 || args->dim_state == 0) return CCV_OK;
    if (query_start_loc == nullptr) return CCV_ERR_NULL_POINTER;
    if ((status = ssm_check_written(*args, 1, total_tokens)) != CCV_OK) return status;
    const ccv_ssm_args a = ssm_ordered(*args);
    const bool copies = !mapped(a.x, a.num_heads) || !mapped(a.B, a.num_groups) || !mapped(a.C, a.num_groups);
    const int64_t need = ssm_fwd_workspace(total_tokens, batch, a.num_heads, a.num_groups, a.head_dim, a.dim_state, a.a_per_state, copies);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 127u) != 0))
        return CCV_ERR_WORKSPACE;
    const Form form = choose(total_tokens, batch, a.head_dim, a.dim_state, a.a_per_state);
    if (form == kRecurrent) {
        const SsmRows rows{query_start_loc, cache_indices, has_initial_state, nullptr, nullptr, 0, 0, 0, batch, 0, total_tokens, err_count};
        return ssm_launch_recurrent(a, rows, stream);
    }
    SsmFwd p{a, query_start_loc, cache_indices, has_initial_state, batch, total_tokens, err_count,
             form == kScan ? ssm_scan_segments(total_tokens, batch, a.num_heads, a.num_groups, a.head_dim, a.dim_state)
                           : ssm_chunked_segments(total_tokens, batch, a.num_heads, a.head_dim),
             nullptr, nullptr};
    if (form == kScan) return ssm_launch_scan(p, workspace, stream);
    if (copies) {
        uint8_t *to = static_cast<uint8_t *>(workspace) + ssm_chunked_workspace(total_tokens, batch, a.num_heads, a.head_dim, p.seg_chunks);
        if ((status = copy_view(p.a.x, to, total_tokens, a.num_heads, a.head_dim, stream)) != CCV_OK) return status;
        to += copy_bytes(total_tokens, a.num_heads, a.head_dim);
        if ((status = copy_view(p.a.B, to, total_tokens, a.num_groups, a.dim_state, stream)) != CCV_OK) return status;
        to += copy_bytes(total_tokens, a.num_groups, a.dim_state);
        if ((status = copy_view(p.a.C, to, total_tokens, a.num_groups, a.dim_state, stream)) != CCV_OK) return status;
    }
    return ssm_launch_chunked(p, workspace, stream);
}
