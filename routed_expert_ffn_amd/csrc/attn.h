// attn.h -- internal host-side launchers of the attention half's kernels
// (page tables, head norms + rotation, paged attention, dense products); not
// part of the ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

// A key-value cache as the kernels take it (moe_kv_cache, checked).
struct KvView {
    void* k;
    void* v;
    float* k_scale;   // null: bf16 elements
    float* v_scale;
    int num_pages, page_shift, n_kv_heads, head_dim;
};

// kv_plan.hip
constexpr int MAX_REQUESTS = 4096;
hipError_t launch_kv_plan(const int32_t* cached_len, const int32_t* new_len, int S, const int32_t* free_pages,
                          int n_free, int page_shift, int T, int32_t* table, int W, int32_t* q_offsets,
                          int32_t* kv_len, int32_t* positions, int32_t* slots, int32_t* counts, hipStream_t st);

// rope.hip
hipError_t launch_qk_norm_rope(const uint16_t* qkv, int64_t stride, int T, int n_heads, const KvView& cache,
                               const float* q_weight, const float* k_weight, float eps, const float* inv_freq,
                               int rope_dim, int interleaved, float rope_scale, const int32_t* positions,
                               const int32_t* slots, uint16_t* q_out, hipStream_t st);

// paged_attn.hip
constexpr int MAX_GROUP = 64;   // query heads per key-value head
size_t paged_attn_workspace_bytes(int T, int n_heads, int n_kv_heads, int head_dim, int S);
hipError_t launch_paged_attn(const uint16_t* q, int64_t q_stride, int T, int n_heads, const KvView& cache,
                             const int32_t* table, int W, const int32_t* q_offsets, const int32_t* kv_len, int S,
                             float scale, float softcap, int window, uint16_t* out, void* ws, hipStream_t st);

// linear.hip
size_t linear_workspace_bytes(int T, int N, int K);
hipError_t launch_linear(const uint16_t* x, int64_t x_stride, const uint16_t* w, const float* bias, int act,
                         const void* residual, int T, int N, int K, void* out, int out_bf16, void* ws,
                         hipStream_t st);
