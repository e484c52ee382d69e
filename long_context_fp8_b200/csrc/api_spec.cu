// C entry points of speculative decoding: argument checks and launches.
#include <algorithm>
#include <cmath>

#include "kernels.h"

using namespace dsa;

namespace {

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }
inline dsa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA; }

constexpr int64_t kInt32Max = 0x7fffffff;
constexpr int64_t kMaxVocab = 1 << 30;

// Block tables and their pool: shapes shared by the entry points below.
dsa_status check_pages(int max_pages, int64_t num_pages, int page_size)
{
    if (max_pages <= 0 || num_pages <= 0 || page_size <= 0) return DSA_ERR_INVALID_ARG;
    if (num_pages > kInt32Max / page_size || (int64_t)max_pages * page_size > kInt32Max) return DSA_ERR_UNSUPPORTED;
    return DSA_OK;
}

}  // namespace

extern "C" {

dsa_status dsa_rope_freqs(int rot_dim, double base, dsa_rope_scaling scaling, double factor,
                          int64_t original_context, double beta_fast, double beta_slow, uint64_t *turns_out)
{
    if (!turns_out || rot_dim < 2 || rot_dim > 256 || rot_dim % 2 != 0 || !(base > 1.0) || !std::isfinite(base))
        return DSA_ERR_INVALID_ARG;
    if (scaling != DSA_ROPE_NONE && scaling != DSA_ROPE_LINEAR && scaling != DSA_ROPE_YARN) return DSA_ERR_INVALID_ARG;
    if (scaling != DSA_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return DSA_ERR_INVALID_ARG;
    constexpr double kTwoPi = 6.283185307179586476925;
    double low = 0.0, high = 0.0;
    if (scaling == DSA_ROPE_YARN) {
        if (original_context < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast))
            return DSA_ERR_INVALID_ARG;
        auto dim_of = [&](double beta) {
            return rot_dim * std::log((double)original_context / (kTwoPi * beta)) / (2.0 * std::log(base));
        };
        low = std::max(std::floor(dim_of(beta_fast)), 0.0);
        high = std::min(std::ceil(dim_of(beta_slow)), (double)(rot_dim - 1));
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == DSA_ROPE_LINEAR) {
            f /= factor;
        } else if (scaling == DSA_ROPE_YARN) {
            const double r = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001)));
            f = f * (1.0 - r) + f / factor * r;
        }
        // f <= 1 radian, so the fraction of a turn is below 1/6 and fits 64 bits
        turns_out[i] = (uint64_t)std::nearbyint(std::ldexp(f / kTwoPi, 64));
    }
    return DSA_OK;
}

dsa_status dsa_rope(const void *q, int64_t q_stride, int H_q, const void *k, int64_t k_stride, int H_k,
                    const int32_t *positions, int64_t rows, int d, int rot_begin, int rot_dim, int interleaved,
                    const uint64_t *turns, float attn_factor, int inverse, void *q_out, int64_t q_out_stride,
                    void *k_out, int64_t k_out_stride, dsa_dtype dtype, void *stream)
{
    if (dtype != DSA_BF16 && dtype != DSA_F32) return DSA_ERR_UNSUPPORTED;
    if (rows < 0 || d <= 0 || H_q <= 0 || H_k < 0 || rot_begin < 0 || rot_dim <= 0 || !turns ||
        !std::isfinite(attn_factor))
        return DSA_ERR_INVALID_ARG;
    if ((k == nullptr) != (H_k == 0) || (k_out == nullptr) != (H_k == 0)) return DSA_ERR_INVALID_ARG;
    if (d % 8 != 0 || d > 1024 || rot_begin % 8 != 0 || rot_dim % 16 != 0 || rot_dim > 256 || rot_begin + rot_dim > d ||
        H_q > 32768 || H_k > 32768)
        return DSA_ERR_UNSUPPORTED;
    if (q_stride % 8 != 0 || q_out_stride % 8 != 0 || q_stride < (int64_t)H_q * d || q_out_stride < (int64_t)H_q * d)
        return DSA_ERR_INVALID_ARG;
    if (H_k > 0 && (k_stride % 8 != 0 || k_out_stride % 8 != 0 || k_stride < (int64_t)H_k * d ||
                    k_out_stride < (int64_t)H_k * d))
        return DSA_ERR_INVALID_ARG;
    if (rows == 0) return DSA_OK;
    if (rows > kInt32Max) return DSA_ERR_UNSUPPORTED;
    if (!q || !q_out || !positions || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(k_out, 16) ||
        !aligned(positions, 4))
        return DSA_ERR_INVALID_ARG;
    // in place means the same rows
    if ((q == q_out && q_stride != q_out_stride) || (k && k == k_out && k_stride != k_out_stride)) return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_rope(q, q_stride, H_q, k, k_stride, H_k, positions, rows, d, rot_begin, rot_dim,
                                   interleaved != 0, turns, attn_factor, inverse != 0, q_out, q_out_stride, k_out,
                                   k_out_stride, dtype == DSA_BF16, as_stream(stream)));
}

dsa_status dsa_blocks_extend(const int32_t *new_lens, int32_t *context_lens, int32_t *pages_held,
                             int32_t *block_table, const int32_t *free_pages, int64_t free_capacity,
                             int32_t *free_count, int B, int max_pages_per_seq, int64_t num_pages, int page_size,
                             int64_t max_tokens, int32_t *token_start, int32_t *seq_ids, int32_t *positions,
                             int64_t *slots, uint32_t *status, void *stream)
{
    if (B < 0 || free_capacity < 0 || max_tokens < 0) return DSA_ERR_INVALID_ARG;
    if (B == 0) return DSA_OK;
    const dsa_status s = check_pages(max_pages_per_seq, num_pages, page_size);
    if (s != DSA_OK) return s;
    if (free_capacity > kInt32Max || max_tokens > kInt32Max) return DSA_ERR_UNSUPPORTED;
    if (!new_lens || !context_lens || !pages_held || !block_table || (free_capacity > 0 && !free_pages) || !free_count ||
        !token_start || (max_tokens > 0 && (!seq_ids || !positions)))
        return DSA_ERR_INVALID_ARG;
    if (!aligned(new_lens, 16) || !aligned(context_lens, 16) || !aligned(pages_held, 16) || !aligned(block_table, 16) ||
        !aligned(free_pages, 16) || !aligned(free_count, 4) || !aligned(token_start, 16) || !aligned(seq_ids, 16) ||
        !aligned(positions, 16) || !aligned(slots, 16) || !aligned(status, 4))
        return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_blocks_extend(new_lens, context_lens, pages_held, block_table, free_pages, free_capacity,
                                            free_count, B, max_pages_per_seq, num_pages, page_size, max_tokens,
                                            token_start, seq_ids, positions, slots, status, as_stream(stream)));
}

dsa_status dsa_blocks_trim(const int32_t *keep_lens, int32_t *context_lens, int32_t *pages_held,
                           int32_t *block_table, int32_t *free_pages, int64_t free_capacity, int32_t *free_count,
                           int B, int max_pages_per_seq, int64_t num_pages, int page_size, uint32_t *status,
                           void *stream)
{
    if (B < 0 || free_capacity < 0) return DSA_ERR_INVALID_ARG;
    if (B == 0) return DSA_OK;
    const dsa_status s = check_pages(max_pages_per_seq, num_pages, page_size);
    if (s != DSA_OK) return s;
    if (free_capacity > kInt32Max) return DSA_ERR_UNSUPPORTED;
    if (!keep_lens || !context_lens || !pages_held || !block_table || (free_capacity > 0 && !free_pages) || !free_count)
        return DSA_ERR_INVALID_ARG;
    if (!aligned(keep_lens, 16) || !aligned(context_lens, 16) || !aligned(pages_held, 16) || !aligned(block_table, 16) ||
        !aligned(free_pages, 16) || !aligned(free_count, 4) || !aligned(status, 4))
        return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_blocks_trim(keep_lens, context_lens, pages_held, block_table, free_pages, free_capacity,
                                          free_count, B, max_pages_per_seq, num_pages, page_size, status,
                                          as_stream(stream)));
}

size_t dsa_tree_attn_workspace_size(int B, int64_t N, int H_q, int H_kv, int d)
{
    if (B <= 0 || N <= 0 || H_q <= 0 || H_kv <= 0 || (d != 64 && d != 128)) return 0;
    return tree_attn_ws_bytes(d);
}

dsa_status dsa_tree_attn(const void *q, const void *k_cache, const float *k_cache_scale, const void *v_cache,
                         const float *v_cache_scale, const int32_t *block_table, const int32_t *context_lens,
                         const int32_t *token_start, const int32_t *parents, int64_t num_pages,
                         int max_pages_per_seq, int page_size, int B, int64_t N, int max_tree, int64_t max_context,
                         int H_q, int H_kv, int d, float sm_scale, void *out, float *lse_out, void *workspace,
                         size_t ws_bytes, void *stream)
{
    if (B < 0 || N < 0) return DSA_ERR_INVALID_ARG;
    if (B == 0 || N == 0) return DSA_OK;
    if (H_q <= 0 || H_kv <= 0 || d <= 0 || max_tree <= 0 || max_context <= 0 || !std::isfinite(sm_scale) ||
        !(sm_scale > 0.f))
        return DSA_ERR_INVALID_ARG;
    const dsa_status s = check_pages(max_pages_per_seq, num_pages, page_size);
    if (s != DSA_OK) return s;
    if (max_tree > DSA_MAX_TREE || (d != 64 && d != 128) || page_size % 16 != 0 || H_q % H_kv != 0 || H_q > 32768 ||
        B > 65536 || N > kInt32Max)
        return DSA_ERR_UNSUPPORTED;
    // the kernel's positions are 32 bits wide, to the end of a context's last block of 128
    if (std::min(max_context, (int64_t)max_pages_per_seq * page_size) > kInt32Max - 127) return DSA_ERR_UNSUPPORTED;
    if (!q || !k_cache || !v_cache || !block_table || !context_lens || !token_start || !parents || !out ||
        (k_cache_scale == nullptr) != (v_cache_scale == nullptr))
        return DSA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(lse_out, 4) ||
        !aligned(k_cache_scale, 4) || !aligned(v_cache_scale, 4) || !aligned(block_table, 4) ||
        !aligned(context_lens, 4) || !aligned(token_start, 4) || !aligned(parents, 4))
        return DSA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || ws_bytes < dsa_tree_attn_workspace_size(B, N, H_q, H_kv, d))
        return DSA_ERR_WORKSPACE;
    return cuda_status(launch_tree_attn((const uint16_t *)q, k_cache, k_cache_scale, v_cache, v_cache_scale, block_table,
                                        context_lens, token_start, parents, num_pages, max_pages_per_seq, page_size, B,
                                        N, max_tree, max_context, H_q, H_kv, d, sm_scale, (uint16_t *)out, lse_out,
                                        workspace, as_stream(stream)));
}

dsa_status dsa_verify_tree(const float *target_probs, const float *draft_probs, const int32_t *tokens,
                           const int32_t *parents, const int32_t *token_start, const float *u_accept,
                           const float *u_sample, int B, int64_t N, int64_t V, int max_path, int32_t *path_out,
                           int32_t *accept_len, int32_t *next_token, uint32_t *status, void *stream)
{
    if (B < 0 || N < 0 || V < 1 || max_path < 1) return DSA_ERR_INVALID_ARG;
    if (B == 0) return DSA_OK;
    if (V > kMaxVocab || N > kInt32Max || (int64_t)B * 8 > kInt32Max) return DSA_ERR_UNSUPPORTED;
    if (!token_start || !u_sample || !path_out || !accept_len || !next_token ||
        (N > 0 && (!target_probs || !tokens || !parents || !u_accept)))
        return DSA_ERR_INVALID_ARG;
    if (!aligned(target_probs, 16) || !aligned(draft_probs, 16) || !aligned(tokens, 4) || !aligned(parents, 4) ||
        !aligned(token_start, 4) || !aligned(u_accept, 4) || !aligned(u_sample, 4) || !aligned(path_out, 4) ||
        !aligned(accept_len, 4) || !aligned(next_token, 4) || !aligned(status, 4))
        return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_verify_tree(target_probs, draft_probs, tokens, parents, token_start, u_accept, u_sample, B,
                                          N, V, max_path, path_out, accept_len, next_token, status, as_stream(stream)));
}

dsa_status dsa_cache_compact(const int32_t *block_table, const int32_t *context_lens, const int32_t *token_start,
                             const int32_t *path, const int32_t *accept_len, int B, int64_t N, int max_path,
                             int max_pages_per_seq, int64_t num_pages, int page_size, int d_I, int d,
                             void *kidx_cache, float *kscale_cache, void *k_cache, float *k_cache_scale,
                             void *v_cache, float *v_cache_scale, int32_t *keep_lens_out, uint32_t *status,
                             void *stream)
{
    if (B < 0 || N < 0 || max_path < 1 || d <= 0) return DSA_ERR_INVALID_ARG;
    if (B == 0) return DSA_OK;
    const dsa_status s = check_pages(max_pages_per_seq, num_pages, page_size);
    if (s != DSA_OK) return s;
    if (!block_table || !context_lens || !token_start || !path || !accept_len || !k_cache || !v_cache ||
        (kidx_cache == nullptr) != (kscale_cache == nullptr) || (k_cache_scale == nullptr) != (v_cache_scale == nullptr) ||
        (kidx_cache && d_I <= 0))
        return DSA_ERR_INVALID_ARG;
    if ((kidx_cache && (d_I % 8 != 0 || d_I > 65536)) || d > 65536 ||
        d % (k_cache_scale ? 8 : 4) != 0)
        return DSA_ERR_UNSUPPORTED;
    if (!aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(token_start, 4) || !aligned(path, 4) ||
        !aligned(accept_len, 4) || !aligned(kidx_cache, 8) || !aligned(kscale_cache, 4) || !aligned(k_cache, 8) ||
        !aligned(k_cache_scale, 4) || !aligned(v_cache, 8) || !aligned(v_cache_scale, 4) || !aligned(keep_lens_out, 4) ||
        !aligned(status, 4))
        return DSA_ERR_INVALID_ARG;
    return cuda_status(launch_cache_compact(block_table, context_lens, token_start, path, accept_len, B, N, max_path,
                                            max_pages_per_seq, num_pages, page_size, d_I, d, kidx_cache, kscale_cache,
                                            k_cache, k_cache_scale, v_cache, v_cache_scale, keep_lens_out, status,
                                            as_stream(stream)));
}

}  // extern "C"
