// rope.hip -- per-head norms of queries and keys, the position rotation and
// the write into the paged cache, in one pass over the projection's rows
// (gfx950).
//
//   q, k: y = x rsqrt(mean x^2 + eps) w, then (a, b) -> f (a cos - b sin, b cos + a sin)
//   v:    as it is;  q -> q_out (bf16), k and v -> their cache slot (bf16, or e4m3 with scale max|y| / 448)
//
// HBM-bound: a row of 20 heads of 256 is read once (10 KB) and written once.
// A lane holds 8 consecutive elements of a head (16-byte loads and stores), a
// head is head_dim / 8 lanes, so a wave does 2 to 8 heads at a time; sums and
// maxima over a head are lane exchanges.  The angles depend on the row only:
// the block forms its rows' cos and sin once, in LDS, and every head reuses
// them.  position * inv_freq and its remainder modulo 2 pi are taken in fp64
// (at position 250,000 the fp32 product alone is off by 2^-24 * 250,000 =
// 0.015 radians), the sine and cosine of the remainder in fp32.
#include "attn.h"
#include "common.h"

namespace {

constexpr int ROPE_THREADS = 256;
typedef uint32_t u32x2_r __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_r __attribute__((ext_vector_type(2)));

MOE_DEV uint32_t pack2(float lo, float hi) {
    const bf16x2_r v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

// D: head_dim; F8: e4m3 cache; TB: rows per block
template <int D, int F8, int TB>
__global__ __launch_bounds__(ROPE_THREADS) void k_qk_norm_rope(
    const uint16_t* __restrict__ qkv, int64_t stride, int T, int n_heads, KvView cache,
    const float* __restrict__ q_weight, const float* __restrict__ k_weight, float eps,
    const float* __restrict__ inv_freq, int R, int interleaved, float rope_scale, const int32_t* __restrict__ positions,
    const int32_t* __restrict__ slots, uint16_t* __restrict__ q_out, int heads_per_block) {
    constexpr int LPH = D / 8;             // lanes per head
    constexpr int HPW = WAVE / LPH;        // heads per wave
    __shared__ float2 cs[TB * (D / 2)];    // (cos, sin) * rope_scale of the block's rows
    const int t0 = blockIdx.x * TB;
    const int rows = min(TB, T - t0);
    const int half = R / 2;
    for (int i = threadIdx.x; i < rows * half; i += ROPE_THREADS) {
        const int r = i / half, p = i - r * half;
        const double a = (double)positions[t0 + r] * (double)inv_freq[p];
        const double n = rint(a * 0.15915494309189533577);                 // turns
        const double rem = fma(n, -2.4492935982947064e-16, fma(n, -6.28318530717958623, a));
        float s, c;
        sincosf((float)rem, &s, &c);
        cs[r * (D / 2) + p] = make_float2(c * rope_scale, s * rope_scale);
    }
    __syncthreads();
    const int nk = cache.n_kv_heads, heads = n_heads + 2 * nk;
    const int l = lane_id(), w = threadIdx.x / WAVE;
    const int c8 = l % LPH, sub = l / LPH;
    const int h_begin = blockIdx.y * heads_per_block, h_end = min(heads, h_begin + heads_per_block);
    const int groups = (h_end - h_begin + HPW - 1) / HPW;
    const int page_mask = (1 << cache.page_shift) - 1;
    const int64_t cache_slots = (int64_t)cache.num_pages << cache.page_shift;
    for (int u = w; u < rows * groups; u += ROPE_THREADS / WAVE) {
        const int r = u / groups, h = h_begin + (u - r * groups) * HPW + sub;
        const int t = t0 + r, slot = slots[t];
        if (slot < 0 || slot >= cache_slots) continue;                     // a padding row (the same for the whole wave)
        const bool have = h < h_end;
        const uint4 raw = *reinterpret_cast<const uint4*>(qkv + (int64_t)t * stride + (have ? h : h_begin) * D + c8 * 8);
        float x[8];
        const uint32_t u4[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; i++) { x[2 * i] = bf16lo_to_f32(u4[i]); x[2 * i + 1] = bf16hi_to_f32(u4[i]); }
        const bool is_q = h < n_heads, is_v = h >= n_heads + nk;
        const float* wt = is_q ? q_weight : k_weight;
        if (q_weight || k_weight) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; i++) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int d = 1; d < LPH; d <<= 1) ss += wave_xor(ss, d);
            if (wt && !is_v) {
                const float inv = 1.0f / sqrtf(ss * (1.0f / D) + eps);
                const float4 wa = *reinterpret_cast<const float4*>(wt + c8 * 8);
                const float4 wb = *reinterpret_cast<const float4*>(wt + c8 * 8 + 4);
                const float ww[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
                for (int i = 0; i < 8; i++) x[i] = x[i] * inv * ww[i];
            }
        }
        const bool rot = !is_v && c8 * 8 < R;
        if (interleaved) {
            if (rot) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float2 a = cs[r * (D / 2) + c8 * 4 + i];
                    const float p = x[2 * i], q = x[2 * i + 1];
                    x[2 * i] = p * a.x - q * a.y;
                    x[2 * i + 1] = q * a.x + p * a.y;
                }
            }
        } else if (R > 0) {
            // the pair of chunk c is chunk c +- R / 16 of the same head
            const int pc = c8 < R / 16 ? c8 + R / 16 : c8 - R / 16;
            const int src = sub * LPH + (rot ? pc : c8);
            const bool second = c8 >= R / 16;
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; i++) y[i] = __shfl(x[i], src, WAVE);
            if (rot) {
                const int p0 = r * (D / 2) + (second ? c8 - R / 16 : c8) * 8;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float2 a = cs[p0 + i];
                    x[i] = second ? x[i] * a.x + y[i] * a.y : x[i] * a.x - y[i] * a.y;
                }
            }
        }
        float amax = 0.f;
        if constexpr (F8) {
            bool nan = false;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                amax = fmaxf(amax, fabsf(x[i]));
                nan |= x[i] != x[i];
            }
            if (nan) amax = __builtin_nanf("");
#pragma unroll
            for (int d = 1; d < LPH; d <<= 1) {
                const float o = wave_xor(amax, d);
                amax = (o != o || amax != amax) ? __builtin_nanf("") : fmaxf(amax, o);
            }
        }
        if (!have) continue;
        if (is_q) {
            uint4 o;
            o.x = pack2(x[0], x[1]); o.y = pack2(x[2], x[3]); o.z = pack2(x[4], x[5]); o.w = pack2(x[6], x[7]);
            *reinterpret_cast<uint4*>(q_out + ((int64_t)t * n_heads + h) * D + c8 * 8) = o;
            continue;
        }
        const int kh = is_v ? h - n_heads - nk : h - n_heads;
        const int64_t ph = (int64_t)(slot >> cache.page_shift) * nk + kh;    // (page, head)
        const int off = slot & page_mask;
        if constexpr (F8) {
            // a head of zeros (or so small that its scale would be subnormal) is stored as zeros of scale 0
            float sc = amax / 448.0f;
            if (sc < 1.17549435e-38f) sc = 0.f;
            const float dv = sc == 0.f ? 1.0f : sc;
            uint32_t a = 0, b = 0;
            a = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] / dv, x[1] / dv, a, false);
            a = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] / dv, x[3] / dv, a, true);
            b = __builtin_amdgcn_cvt_pk_fp8_f32(x[4] / dv, x[5] / dv, b, false);
            b = __builtin_amdgcn_cvt_pk_fp8_f32(x[6] / dv, x[7] / dv, b, true);
            // k: 16-element chunks, page_size of them side by side; v: rows
            const int64_t at = is_v ? (((ph << cache.page_shift) + off) * D + c8 * 8)
                                    : ((((ph * (D / 16) + (c8 >> 1)) << cache.page_shift) + off) * 16 + (c8 & 1) * 8);
            *reinterpret_cast<u32x2_r*>((uint8_t*)(is_v ? cache.v : cache.k) + at) = u32x2_r{a, b};
            if (c8 == 0) (is_v ? cache.v_scale : cache.k_scale)[(ph << cache.page_shift) + off] = sc;
        } else {
            uint4 o;
            o.x = pack2(x[0], x[1]); o.y = pack2(x[2], x[3]); o.z = pack2(x[4], x[5]); o.w = pack2(x[6], x[7]);
            const int64_t at = is_v ? (((ph << cache.page_shift) + off) * D + c8 * 8)
                                    : ((((ph * (D / 8) + c8) << cache.page_shift) + off) * 8);
            *reinterpret_cast<uint4*>((uint16_t*)(is_v ? cache.v : cache.k) + at) = o;
        }
    }
}

template <int D, int F8>
hipError_t launch_d(const uint16_t* qkv, int64_t stride, int T, int n_heads, const KvView& cache, const float* qw,
                    const float* kw, float eps, const float* inv_freq, int R, int inter, float rope_scale,
                    const int32_t* positions, const int32_t* slots, uint16_t* q_out, hipStream_t st) {
    constexpr int HPW = WAVE / (D / 8);
    const int heads = n_heads + 2 * cache.n_kv_heads;
    if (T <= 256) {
        // few rows: one row's heads over several blocks, one wave pass each
        const int hpb = HPW * (ROPE_THREADS / WAVE);
        hipLaunchKernelGGL((k_qk_norm_rope<D, F8, 1>), dim3(T, (heads + hpb - 1) / hpb), dim3(ROPE_THREADS), 0, st, qkv,
                           stride, T, n_heads, cache, qw, kw, eps, inv_freq, R, inter, rope_scale, positions, slots,
                           q_out, hpb);
    } else {
        constexpr int TB = 16;
        hipLaunchKernelGGL((k_qk_norm_rope<D, F8, TB>), dim3((T + TB - 1) / TB, 1), dim3(ROPE_THREADS), 0, st, qkv,
                           stride, T, n_heads, cache, qw, kw, eps, inv_freq, R, inter, rope_scale, positions, slots,
                           q_out, heads);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_norm_rope(const uint16_t* qkv, int64_t stride, int T, int n_heads, const KvView& cache,
                               const float* q_weight, const float* k_weight, float eps, const float* inv_freq,
                               int rope_dim, int interleaved, float rope_scale, const int32_t* positions,
                               const int32_t* slots, uint16_t* q_out, hipStream_t st) {
    if (T == 0) return hipSuccess;
    auto go = [&](auto fn) {
        return fn(qkv, stride, T, n_heads, cache, q_weight, k_weight, eps, inv_freq, rope_dim, interleaved, rope_scale,
                  positions, slots, q_out, st);
    };
    const bool f8 = cache.k_scale != nullptr;
    switch (cache.head_dim) {
        case 64: return f8 ? go(launch_d<64, 1>) : go(launch_d<64, 0>);
        case 128: return f8 ? go(launch_d<128, 1>) : go(launch_d<128, 0>);
        case 256: return f8 ? go(launch_d<256, 1>) : go(launch_d<256, 0>);
    }
    return hipErrorInvalidValue;
}
