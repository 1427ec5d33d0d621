// api_attn.hip -- the C ABI of the attention half (declared in
// include/moe.h): argument checks and launches.  Nothing here allocates memory
// or synchronises; every call only enqueues on `stream`.
#include "../../include/moe.h"
#include "attn.h"

#include <cmath>

namespace {

bool aligned16(const void* p) { return p == nullptr || ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return p == nullptr || ((uintptr_t)p & 3u) == 0; }
hipStream_t S(moe_stream s) { return (hipStream_t)s; }
moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// log2 of a page size the kernels take, or -1
int page_shift_of(int page_size) {
    for (int s = 4; s <= 10; s++)
        if (page_size == 1 << s) return s;
    return -1;
}

moe_status cache_view(const moe_kv_cache* c, KvView* v) {
    if (!c || !c->k || !c->v || c->num_pages <= 0 || c->page_size <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0)
        return MOE_ERR_INVALID_ARG;
    if (c->dtype != MOE_BF16 && c->dtype != MOE_FP8_E4M3)
        return c->dtype >= MOE_F32 && c->dtype <= MOE_FP8_E4M3 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
    const bool f8 = c->dtype == MOE_FP8_E4M3;
    if (f8 != (c->k_scale != nullptr) || f8 != (c->v_scale != nullptr)) return MOE_ERR_INVALID_ARG;
    const int shift = page_shift_of(c->page_size);
    if (shift < 0 || (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) ||
        (int64_t)c->num_pages * c->page_size > INT32_MAX)
        return MOE_ERR_UNSUPPORTED;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale))
        return MOE_ERR_UNSUPPORTED;
    *v = KvView{c->k, c->v, c->k_scale, c->v_scale, c->num_pages, shift, c->n_kv_heads, c->head_dim};
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_kv_plan(const int32_t* cached_len, const int32_t* new_len, int32_t S_, const int32_t* free_pages,
                       int32_t n_free, int32_t page_size, int32_t T, int32_t* page_table, int32_t W,
                       int32_t* q_offsets, int32_t* kv_len, int32_t* positions, int32_t* slots, int32_t* counts,
                       moe_stream stream) {
    if (S_ <= 0 || T < 0 || W <= 0 || n_free < 0 || page_size <= 0) return MOE_ERR_INVALID_ARG;
    if (!cached_len || !new_len || !page_table || !q_offsets || !kv_len || !counts || (n_free > 0 && !free_pages) ||
        (T > 0 && (!positions || !slots)))
        return MOE_ERR_INVALID_ARG;
    const int shift = page_shift_of(page_size);
    if (shift < 0 || S_ > MAX_REQUESTS || (int64_t)W * page_size > ((int64_t)1 << 30)) return MOE_ERR_UNSUPPORTED;
    if (!aligned4(cached_len) || !aligned4(new_len) || !aligned4(free_pages) || !aligned4(page_table) ||
        !aligned4(q_offsets) || !aligned4(kv_len) || !aligned4(positions) || !aligned4(slots) || !aligned4(counts))
        return MOE_ERR_UNSUPPORTED;
    // every block reads the lengths while the first one writes these
    if (kv_len == cached_len || kv_len == new_len || q_offsets == cached_len || q_offsets == new_len) return MOE_ERR_INVALID_ARG;
    return hip_status(launch_kv_plan(cached_len, new_len, S_, free_pages, n_free, shift, T, page_table, W, q_offsets,
                                     kv_len, positions, slots, counts, S(stream)));
}

moe_status moe_qk_norm_rope(const void* qkv, int32_t x_dtype, int64_t qkv_stride, int32_t T, int32_t n_heads,
                            const moe_kv_cache* cache, const float* q_weight, const float* k_weight, float eps,
                            const float* inv_freq, int32_t rope_dim, int32_t rope_layout, float rope_scale,
                            const int32_t* positions, const int32_t* slots, void* q_out, moe_stream stream) {
    if (T < 0 || n_heads <= 0 || rope_dim < 0 || !(eps >= 0.0f) || !std::isfinite(eps) || !std::isfinite(rope_scale))
        return MOE_ERR_INVALID_ARG;
    if (x_dtype != MOE_F32 && x_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (rope_layout != MOE_ROPE_HALF && rope_layout != MOE_ROPE_INTERLEAVED) return MOE_ERR_INVALID_ARG;
    KvView kv;
    const moe_status chk = cache_view(cache, &kv);
    if (chk != MOE_OK) return chk;
    const int64_t heads = (int64_t)n_heads + 2 * (int64_t)kv.n_kv_heads;
    if (rope_dim > kv.head_dim || (rope_dim > 0 && !inv_freq)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!qkv || !slots || !q_out || (rope_dim > 0 && !positions))) return MOE_ERR_INVALID_ARG;
    if (qkv_stride < heads * kv.head_dim) return MOE_ERR_INVALID_ARG;
    if (x_dtype != MOE_BF16 || rope_dim % 16 != 0 || qkv_stride % 8 != 0 || heads > 1024) return MOE_ERR_UNSUPPORTED;
    if (!aligned16(qkv) || !aligned16(q_out) || !aligned16(q_weight) || !aligned16(k_weight) || !aligned4(inv_freq) ||
        !aligned4(positions) || !aligned4(slots))
        return MOE_ERR_UNSUPPORTED;
    return hip_status(launch_qk_norm_rope((const uint16_t*)qkv, qkv_stride, T, n_heads, kv, q_weight, k_weight, eps,
                                          inv_freq, rope_dim, rope_layout == MOE_ROPE_INTERLEAVED, rope_scale,
                                          positions, slots, (uint16_t*)q_out, S(stream)));
}

size_t moe_paged_attn_workspace_size(int32_t T, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t S_) {
    if (T < 0 || n_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 || S_ <= 0 || n_heads % n_kv_heads != 0) return 0;
    return paged_attn_workspace_bytes(T, n_heads, n_kv_heads, head_dim, S_);
}

moe_status moe_paged_attn(const void* q, int32_t q_dtype, int64_t q_stride, int32_t T, int32_t n_heads,
                          const moe_kv_cache* cache, const int32_t* page_table, int32_t W, const int32_t* q_offsets,
                          const int32_t* kv_len, int32_t S_, float scale, float softcap, int32_t window, void* out,
                          void* workspace, size_t ws_bytes, moe_stream stream) {
    if (T < 0 || n_heads <= 0 || W <= 0 || S_ <= 0 || window < 0 || !(softcap >= 0.0f) || !std::isfinite(softcap) ||
        !std::isfinite(scale))
        return MOE_ERR_INVALID_ARG;
    // the kernel's own factors, in units of log2, must be finite too
    const float log2e = 1.44269504088896341f;
    if (!std::isfinite(scale * log2e) || !std::isfinite(softcap * log2e) || (softcap > 0.0f && !std::isfinite(scale / softcap)))
        return MOE_ERR_INVALID_ARG;
    if (q_dtype != MOE_F32 && q_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    KvView kv;
    const moe_status chk = cache_view(cache, &kv);
    if (chk != MOE_OK) return chk;
    if (!page_table || !q_offsets || !kv_len || (T > 0 && (!q || !out))) return MOE_ERR_INVALID_ARG;
    if (q_stride < (int64_t)n_heads * kv.head_dim || (int64_t)T * n_heads > (int64_t)1 << 30) return MOE_ERR_INVALID_ARG;
    if (q_dtype != MOE_BF16 || S_ > MAX_REQUESTS || n_heads % kv.n_kv_heads != 0 ||
        n_heads / kv.n_kv_heads > MAX_GROUP || q_stride % 8 != 0 || (int64_t)n_heads * kv.head_dim > 64 * 65535 ||
        (int64_t)W * (1 << kv.page_shift) > ((int64_t)1 << 30))
        return MOE_ERR_UNSUPPORTED;
    // the steps of all units (16 rows of a key-value head, 32 positions at least) are counted in int32
    if ((((int64_t)T * n_heads + 15) / 16 + (int64_t)S_ * kv.n_kv_heads) * (((int64_t)W << kv.page_shift) / 32 + 9) > INT32_MAX)
        return MOE_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(out) || !aligned4(page_table) || !aligned4(q_offsets) || !aligned4(kv_len))
        return MOE_ERR_UNSUPPORTED;
    if (!workspace || !aligned16(workspace) ||
        ws_bytes < moe_paged_attn_workspace_size(T, n_heads, kv.n_kv_heads, kv.head_dim, S_))
        return MOE_ERR_WORKSPACE;
    return hip_status(launch_paged_attn((const uint16_t*)q, q_stride, T, n_heads, kv, page_table, W, q_offsets, kv_len,
                                        S_, scale, softcap, window, (uint16_t*)out, workspace, S(stream)));
}

size_t moe_linear_workspace_size(int32_t T, int32_t N, int32_t K) {
    if (T < 0 || N <= 0 || K <= 0) return 0;
    return linear_workspace_bytes(T, N, K);
}

moe_status moe_linear(const void* x, int32_t x_dtype, int64_t x_stride, const void* w, int32_t w_dtype,
                      const float* bias, int32_t act, const void* residual, int32_t T, int32_t N, int32_t K, void* out,
                      int32_t out_dtype, void* workspace, size_t ws_bytes, moe_stream stream) {
    if (T < 0 || N <= 0 || K <= 0 || x_stride < K) return MOE_ERR_INVALID_ARG;
    if (!w || (T > 0 && (!x || !out))) return MOE_ERR_INVALID_ARG;
    if ((x_dtype != MOE_F32 && x_dtype != MOE_BF16) || (out_dtype != MOE_F32 && out_dtype != MOE_BF16) ||
        w_dtype < MOE_F32 || w_dtype > MOE_FP8_E4M3 || act < MOE_ACT_NONE || act > MOE_ACT_RELU)
        return MOE_ERR_INVALID_ARG;
    if (x_dtype != MOE_BF16 || w_dtype != MOE_BF16 || K % 64 != 0 || N % 8 != 0 || x_stride % 8 != 0)
        return MOE_ERR_UNSUPPORTED;
    // 32-bit byte offsets within a tile of 256 rows, and tiles (64 x 64 at least) counted in int32
    if (K > 1 << 22 || x_stride > 1 << 22 || ((int64_t)T / 64 + 1) * ((int64_t)N / 64 + 1) > INT32_MAX / 16)
        return MOE_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(w) || !aligned16(bias) || !aligned16(residual) || !aligned16(out))
        return MOE_ERR_UNSUPPORTED;
    const size_t need = moe_linear_workspace_size(T, N, K);
    if (need > 0 && (!workspace || !aligned16(workspace) || ws_bytes < need)) return MOE_ERR_WORKSPACE;
    return hip_status(launch_linear((const uint16_t*)x, x_stride, (const uint16_t*)w, bias, act, residual, T, N, K,
                                    out, out_dtype == MOE_BF16, workspace, S(stream)));
}

}  // extern "C"
