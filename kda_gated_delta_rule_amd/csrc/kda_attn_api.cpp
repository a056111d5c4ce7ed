// kda_attn_api.cpp -- the extern "C" entry points of the softmax-attention operators declared in
// include/kda.h.  As in kda_api.cpp, every argument check runs here before any HIP call.
#include "kda.h"

#include <float.h>
#include <math.h>

#include "kda_check.hpp"
#include "kda_internal.hpp"

using namespace kda::check;

namespace {

// n rows of `width` contiguous elements every ld elements: 16-byte loads need both aligned.  No
// rows may come with a null pointer.
bool valid_rows(const void* p, int64_t n, int64_t ld, int64_t width, int dtype) {
    const int64_t per = dtype == KDA_BF16 ? 8 : 4;
    return (p || n == 0) && aligned16(p) && ld >= width && ld % per == 0;
}

// What the prompt entry points share: KDA_OK, or the error.
int prompt_args(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv, int dtype,
                const int32_t* cu_q, const int32_t* cu_k, int num_seqs, int64_t total_q, int64_t total_k, int H,
                int Hk, int dk, int dv, float scale) {
    if (!valid_dtype(dtype)) return KDA_ERR_INVALID_ARG;
    if (num_seqs < 0 || total_q < 0 || total_k < 0 || H < 1 || Hk < 1 || H % Hk) return KDA_ERR_INVALID_ARG;
    if (!isfinite(scale)) return KDA_ERR_INVALID_ARG;
    if (!supported_dim(dk) || !supported_dim(dv)) return KDA_ERR_UNSUPPORTED;
    if (!valid_rows(q, total_q, ldq, static_cast<int64_t>(H) * dk, dtype)) return KDA_ERR_INVALID_ARG;
    if (!valid_rows(k, total_k, ldk, static_cast<int64_t>(Hk) * dk, dtype)) return KDA_ERR_INVALID_ARG;
    if (!valid_rows(v, total_k, ldv, static_cast<int64_t>(Hk) * dv, dtype)) return KDA_ERR_INVALID_ARG;
    if (!cu_q || !aligned16(cu_q) || !cu_k || !aligned16(cu_k)) return KDA_ERR_INVALID_ARG;
    // offsets inside a tile of 128 tokens in bf16, of 64 in fp32, are 32-bit
    if (ldq > (1 << 22) || ldk > (1 << 22) || ldv > (1 << 22) || static_cast<int64_t>(H) * dv > (1 << 22))
        return KDA_ERR_INVALID_ARG;
    // token counts as in cu_seqlens (int32), element offsets within int64
    if (total_q > INT32_MAX || total_k > INT32_MAX || H > 65535) return KDA_ERR_INVALID_ARG;
    if (checked_mul(total_q, ldq) < 0 || checked_mul(total_k, ldk) < 0 || checked_mul(total_k, ldv) < 0)
        return KDA_ERR_INVALID_ARG;
    if (num_seqs == 0 && (total_q > 0 || total_k > 0)) return KDA_ERR_INVALID_ARG;
    // launch size: tiles of 64 tokens or more, 256 threads each, within 32-bit work-items
    if (checked_mul((total_q > total_k ? total_q : total_k) / 64 + num_seqs, H) > (1ll << 22))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

bool prompt_sizes(int64_t total_q, int64_t total_k, int H, int Hk, int dk, int dv, int dtype) {
    return total_q >= 0 && total_q <= INT32_MAX && total_k >= 0 && total_k <= INT32_MAX && H >= 1 && H <= 65535 &&
           Hk >= 1 && H % Hk == 0 && supported_dim(dk) && supported_dim(dv) && valid_dtype(dtype);
}

// |scale| as the kernels take it: a masked score is -inf, which a factor of zero would turn to NaN.  The
// smallest number above zero stands for it: the largest product q.k there is then scores 2^-20.
float nonzero(float scale) { return fmaxf(fabsf(scale), FLT_TRUE_MIN); }

}  // namespace

KDA_EXPORT size_t kda_attn_prefill_workspace_size(int num_seqs, int64_t total_q, int64_t total_k, int H, int Hk,
                                                  int dk, int dv, int dtype) {
    if (num_seqs < 0 || !prompt_sizes(total_q, total_k, H, Hk, dk, dv, dtype)) return 0;
    return kda::attn_prefill_workspace_bytes(num_seqs, total_q, total_k, H, dv, dtype == KDA_BF16);
}

KDA_EXPORT int kda_attn_prefill(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                                int dtype, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int num_seqs,
                                int64_t total_q, int64_t total_k, int H, int Hk, int dk, int dv, float scale,
                                void* o, float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const int st = prompt_args(q, ldq, k, ldk, v, ldv, dtype, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                               H, Hk, dk, dv, scale);
    if (st != KDA_OK) return st;
    if (total_q == 0) return KDA_OK;
    if (!o || !aligned16(o) || (lse && !aligned16(lse))) return KDA_ERR_INVALID_ARG;
    const size_t need = kda::attn_prefill_workspace_bytes(num_seqs, total_q, total_k, H, dv, dtype == KDA_BF16);
    if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    kda::AttnPrefillArgs a{q, k, v, ldq, ldk, ldv, cu_seqlens_q, cu_seqlens_k, num_seqs,
                           static_cast<int>(total_q), static_cast<int>(total_k), H, Hk, nonzero(scale), scale < 0.f,
                           o, lse, workspace};
    return to_status(kda::launch_attn_prefill(a, dtype == KDA_BF16, dk, dv, stream));
}

KDA_EXPORT size_t kda_attn_backward_workspace_size(int num_seqs, int64_t total_q, int64_t total_k, int H, int Hk,
                                                   int dk, int dv, int dtype) {
    if (num_seqs < 0 || !prompt_sizes(total_q, total_k, H, Hk, dk, dv, dtype)) return 0;
    return kda::attn_backward_workspace_bytes(num_seqs, total_q, total_k, H, Hk, dk, dv, dtype == KDA_BF16);
}

KDA_EXPORT int kda_attn_backward(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                                 int dtype, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int num_seqs,
                                 int64_t total_q, int64_t total_k, int H, int Hk, int dk, int dv, float scale,
                                 const void* o, const float* lse, const void* dout, void* dq, void* dk_out,
                                 void* dv_out, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const int st = prompt_args(q, ldq, k, ldk, v, ldv, dtype, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                               H, Hk, dk, dv, scale);
    if (st != KDA_OK) return st;
    if (total_q > 0)
        for (const void* p : {o, static_cast<const void*>(lse), dout, static_cast<const void*>(dq)})
            if (!p || !aligned16(p)) return KDA_ERR_INVALID_ARG;
    if (total_k > 0)
        for (const void* p : {dk_out, dv_out})
            if (!p || !aligned16(p)) return KDA_ERR_INVALID_ARG;
    if (total_q == 0 && total_k == 0) return KDA_OK;
    const size_t need =
        kda::attn_backward_workspace_bytes(num_seqs, total_q, total_k, H, Hk, dk, dv, dtype == KDA_BF16);
    if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    kda::AttnBackwardArgs b{{q, k, v, ldq, ldk, ldv, cu_seqlens_q, cu_seqlens_k, num_seqs,
                             static_cast<int>(total_q), static_cast<int>(total_k), H, Hk, nonzero(scale),
                             scale < 0.f, nullptr, nullptr, nullptr},
                            o, lse, dout, scale, dq, dk_out, dv_out, workspace};
    return to_status(kda::launch_attn_backward(b, dtype == KDA_BF16, dk, dv, stream));
}

namespace {

constexpr int64_t kMaxPositions = 1ll << 30;  // of a sequence: positions a step ahead stay within 32 bits
constexpr int64_t kMaxBatch = 1ll << 38;      // of a decode batch: its steps of 256 are counted in 32 bits

int log2_of(int bt) { return bt == 16 ? 4 : bt == 32 ? 5 : bt == 64 ? 6 : bt == 128 ? 7 : -1; }

// The paged cache's arguments: KDA_OK, or the error.
int cache_args(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale, int num_blocks,
               int block_tokens, const int32_t* block_table, int max_blocks, int Hk, int dk, int dv) {
    if (num_blocks < 1 || max_blocks < 1 || Hk < 1) return KDA_ERR_INVALID_ARG;
    if (!supported_dim(dk) || !supported_dim(dv) || log2_of(block_tokens) < 0) return KDA_ERR_UNSUPPORTED;
    for (const void* p : {k_cache, v_cache, static_cast<const void*>(k_scale), static_cast<const void*>(v_scale),
                          static_cast<const void*>(block_table)})
        if (!p || !aligned16(p)) return KDA_ERR_INVALID_ARG;
    if (Hk > 65535 || static_cast<int64_t>(max_blocks) * block_tokens > kMaxPositions) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

bool decode_sizes(int N, int T, int H, int Hk, int dtype, int block_tokens, int max_blocks) {
    return valid_dtype(dtype) && N >= 0 && T >= 1 && T <= 8 && H >= 1 && H <= 65535 && Hk >= 1 && H % Hk == 0 &&
           log2_of(block_tokens) >= 0 && max_blocks >= 1 &&
           static_cast<int64_t>(max_blocks) * block_tokens <= kMaxPositions &&
           static_cast<int64_t>(N) * T * H <= (1ll << 22) &&
           static_cast<int64_t>(max_blocks) * block_tokens * N <= kMaxBatch;
}

size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

int cache_append(const void* k, int64_t ldk, const void* v, int64_t ldv, int dtype, const int32_t* cu_seqlens,
                 const int32_t* start_len, int N, int64_t total_tokens, void* k_cache, void* v_cache, float* k_scale,
                 float* v_scale, int num_blocks, int block_tokens, const int32_t* block_table, int max_blocks, int Hk,
                 int dk, int dv, bool clear, hipStream_t stream) {
    if (!valid_dtype(dtype) || N < 0 || total_tokens < 0 || total_tokens > INT32_MAX) return KDA_ERR_INVALID_ARG;
    if (N == 0) return total_tokens == 0 ? KDA_OK : KDA_ERR_INVALID_ARG;
    const int st = cache_args(k_cache, v_cache, k_scale, v_scale, num_blocks, block_tokens, block_table, max_blocks,
                              Hk, dk, dv);
    if (st != KDA_OK) return st;
    if (!valid_rows(k, total_tokens, ldk, static_cast<int64_t>(Hk) * dk, dtype)) return KDA_ERR_INVALID_ARG;
    if (!valid_rows(v, total_tokens, ldv, static_cast<int64_t>(Hk) * dv, dtype)) return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens || !aligned16(cu_seqlens) || !start_len || !aligned16(start_len)) return KDA_ERR_INVALID_ARG;
    if (checked_mul(total_tokens, ldk) < 0 || checked_mul(total_tokens, ldv) < 0) return KDA_ERR_INVALID_ARG;
    // launch size: two workgroups of 256 threads for each block written into and head
    if (checked_mul(total_tokens / block_tokens + 2ll * N, Hk) > (1ll << 22)) return KDA_ERR_INVALID_ARG;
    if (total_tokens == 0) return KDA_OK;
    kda::AttnAppendArgs a{k, v, ldk, ldv, cu_seqlens, start_len, N, static_cast<int>(total_tokens), Hk,
                          static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), k_scale, v_scale,
                          num_blocks, block_tokens, block_table, max_blocks, clear};
    return to_status(kda::launch_attn_append(a, dtype == KDA_BF16, dk, dv, stream));
}

}  // namespace

KDA_EXPORT int kda_attn_cache_append(const void* k, int64_t ldk, const void* v, int64_t ldv, int dtype,
                                     const int32_t* cu_seqlens, const int32_t* start_len, int N, int64_t total_tokens,
                                     void* k_cache, void* v_cache, float* k_scale, float* v_scale, int num_blocks,
                                     int block_tokens, const int32_t* block_table, int max_blocks, int Hk, int dk,
                                     int dv, hipStream_t stream) {
    return cache_append(k, ldk, v, ldv, dtype, cu_seqlens, start_len, N, total_tokens, k_cache, v_cache, k_scale,
                        v_scale, num_blocks, block_tokens, block_table, max_blocks, Hk, dk, dv, false, stream);
}

KDA_EXPORT int kda_attn_cache_append_clear(const void* k, int64_t ldk, const void* v, int64_t ldv, int dtype,
                                           const int32_t* cu_seqlens, const int32_t* start_len, int N,
                                           int64_t total_tokens, void* k_cache, void* v_cache, float* k_scale,
                                           float* v_scale, int num_blocks, int block_tokens,
                                           const int32_t* block_table, int max_blocks, int Hk, int dk, int dv,
                                           hipStream_t stream) {
    return cache_append(k, ldk, v, ldv, dtype, cu_seqlens, start_len, N, total_tokens, k_cache, v_cache, k_scale,
                        v_scale, num_blocks, block_tokens, block_table, max_blocks, Hk, dk, dv, true, stream);
}

KDA_EXPORT size_t kda_attn_decode_workspace_size(int N, int T, int H, int Hk, int dv, int dtype, int block_tokens,
                                                 int max_blocks) {
    if (!decode_sizes(N, T, H, Hk, dtype, block_tokens, max_blocks) || !supported_dim(dv)) return 0;
    const int pieces = kda::attn_decode_pieces(N, T, H, Hk, block_tokens, max_blocks);
    if (N == 0 || pieces == 0) return 0;
    const size_t parts = static_cast<size_t>(kda::attn_decode_most_pieces(N, pieces)) * T * H;
    return round16(parts * sizeof(float2)) + parts * dv * sizeof(float);
}

KDA_EXPORT int kda_attn_decode(const void* q, int64_t ldq, int dtype, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, int num_blocks, int block_tokens,
                               const int32_t* block_table, int max_blocks, const int32_t* context_len, int N, int T,
                               int H, int Hk, int dk, int dv, float scale, void* o, void* workspace,
                               size_t workspace_bytes, hipStream_t stream) {
    if (!valid_dtype(dtype) || N < 0 || T < 1 || T > 8 || H < 1 || Hk < 1 || H % Hk || !isfinite(scale))
        return KDA_ERR_INVALID_ARG;
    if (N == 0) return KDA_OK;
    const int st = cache_args(k_cache, v_cache, k_scale, v_scale, num_blocks, block_tokens, block_table, max_blocks,
                              Hk, dk, dv);
    if (st != KDA_OK) return st;
    if (!decode_sizes(N, T, H, Hk, dtype, block_tokens, max_blocks)) return KDA_ERR_INVALID_ARG;
    if (!valid_rows(q, 1, ldq, static_cast<int64_t>(H) * dk, dtype) || checked_mul(static_cast<int64_t>(N) * T, ldq) < 0)
        return KDA_ERR_INVALID_ARG;
    if (!context_len || !aligned16(context_len) || !o || !aligned16(o)) return KDA_ERR_INVALID_ARG;
    const int bf16 = dtype == KDA_BF16;
    const int pieces = kda::attn_decode_pieces(N, T, H, Hk, block_tokens, max_blocks);
    const size_t need = kda_attn_decode_workspace_size(N, T, H, Hk, dv, dtype, block_tokens, max_blocks);
    if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    const size_t parts = static_cast<size_t>(kda::attn_decode_most_pieces(N, pieces)) * T * H;
    kda::AttnDecodeArgs a{q, ldq, static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache), k_scale,
                          v_scale, num_blocks, block_tokens, log2_of(block_tokens), block_table, max_blocks,
                          context_len, N, T, H, Hk, scale, o, kda::attn_decode_row_groups(T, H, Hk), pieces,
                          pieces ? reinterpret_cast<float*>(ws + round16(parts * sizeof(float2))) : nullptr,
                          pieces ? reinterpret_cast<float2*>(ws) : nullptr};
    return to_status(kda::launch_attn_decode(a, bf16, dk, dv, stream));
}
