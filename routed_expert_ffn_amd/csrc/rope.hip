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
//   8,192 rows of 20 heads of 256 (168 MB): 34.4 us, 4.9 TB/s (a plain copy reaches 5.1);
// 5 rows 3.6 us and 777 rows of 48 heads of 128 into an e4m3 cache (17.6 MB) 9.3 us are
// latency: a load, the angles, two passes of lane moves and a store.
#include "attn.h"
#include "common.h"
#include "stream.h"

#include <algorithm>

namespace {

constexpr int ROPE_THREADS = 256;
typedef uint32_t u32x2_r __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_r __attribute__((ext_vector_type(2)));

// Sum over the LPH lanes of a head (8, 16 or 32), in every one of them: partners
// by DPP within 16 lanes (each step's partner lies in the other half, whose
// lanes already hold one value), across 16 by a lane swap.
template <int LPH>
MOE_DEV float head_sum(float v) {
    v += tr_partner<1>(v);
    v += tr_partner<2>(v);
    v += tr_partner<4>(v);
    if constexpr (LPH >= 16) v += tr_partner<8>(v);
    if constexpr (LPH >= 32) v += tr_partner<16>(v);
    return v;
}

MOE_DEV uint32_t pack2(float lo, float hi) {
    const bf16x2_r v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

// D: head_dim; F8: e4m3 cache; TB: rows per block.  blockIdx.x: rows, blockIdx.y:
// groups_per_block of the row's groups of HPW heads.  A wave takes every fourth
// unit (row, group of heads) of the block, UN of them loaded together, the
// next UN under the current ones; the first loads go out before the angles
// are formed.
template <int D, int F8, int TB, int UN>
__global__ __launch_bounds__(ROPE_THREADS) void k_qk_norm_rope(
    const uint16_t* __restrict__ qkv, int64_t stride, int T, int n_heads, KvView cache,
    const float* __restrict__ q_weight, const float* __restrict__ k_weight, float eps,
    const float* __restrict__ inv_freq, int R, int interleaved, float rope_scale, const int32_t* __restrict__ positions,
    const int32_t* __restrict__ slots, uint16_t* __restrict__ q_out, int groups_per_block) {
    constexpr int LPH = D / 8;             // lanes per head
    constexpr int HPW = WAVE / LPH;        // heads per wave
    constexpr int NWV = ROPE_THREADS / WAVE;
    __shared__ __attribute__((aligned(16))) float2 cs[TB * (D / 2)];   // (cos, sin) * rope_scale of the block's rows
    __shared__ int row_slot[TB];
    const int t0 = blockIdx.x * TB;
    const int rows = min(TB, T - t0);
    const int nk = cache.n_kv_heads, heads = n_heads + 2 * nk;
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int c8 = l % LPH, sub = l / LPH;
    const int g_begin = blockIdx.y * groups_per_block;
    const int groups = min((heads + HPW - 1) / HPW - g_begin, groups_per_block);
    const int units = rows * groups;
    auto load = [&](int u) __attribute__((always_inline)) -> uint4 {
        u = min(u, units - 1);             // past the end: the last unit again, not used
        const int r = u / groups, h = min((g_begin + u - r * groups) * HPW + sub, heads - 1);
        return ldnt16(qkv + (int64_t)(t0 + r) * stride + h * D + c8 * 8);
    };
    uint4 raw[UN];
#pragma unroll
    for (int i = 0; i < UN; i++) raw[i] = load(w + i * NWV);
    float qw[8], kw[8];
    const bool qn = q_weight != nullptr, kn = k_weight != nullptr;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const float4 a = qn ? *reinterpret_cast<const float4*>(q_weight + c8 * 8 + 4 * i) : make_float4(1, 1, 1, 1);
        const float4 b = kn ? *reinterpret_cast<const float4*>(k_weight + c8 * 8 + 4 * i) : make_float4(1, 1, 1, 1);
        qw[4 * i] = a.x; qw[4 * i + 1] = a.y; qw[4 * i + 2] = a.z; qw[4 * i + 3] = a.w;
        kw[4 * i] = b.x; kw[4 * i + 1] = b.y; kw[4 * i + 2] = b.z; kw[4 * i + 3] = b.w;
    }
    const int half = R / 2;
    if ((int)threadIdx.x < rows) row_slot[threadIdx.x] = slots[t0 + threadIdx.x];
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
    const int page_mask = (1 << cache.page_shift) - 1;
    const int64_t cache_slots = (int64_t)cache.num_pages << cache.page_shift;
    // the pair of chunk c in the half layout is chunk c +- R / 16 of the same head
    const bool turned = c8 * 8 < R, second = c8 >= R / 16;
    const int pair_lane = sub * LPH + (turned ? (second ? c8 - R / 16 : c8 + R / 16) : c8);
    const int pair_chunk = second ? c8 - R / 16 : c8;
    auto unit = [&](int u, uint4 rw) __attribute__((always_inline)) {
        const int r = u / groups, h = (g_begin + u - r * groups) * HPW + sub;
        const int t = t0 + r, slot = __builtin_amdgcn_readfirstlane(row_slot[r]);
        if (slot < 0 || slot >= cache_slots) return;                       // a padding row (the same for the whole wave)
        float x[8];
        const uint32_t u4[4] = {rw.x, rw.y, rw.z, rw.w};
#pragma unroll
        for (int i = 0; i < 4; i++) { x[2 * i] = bf16lo_to_f32(u4[i]); x[2 * i + 1] = bf16hi_to_f32(u4[i]); }
        const bool is_q = h < n_heads, is_v = h >= n_heads + nk;
        const bool all_q = (g_begin + u - r * groups) * HPW + HPW <= n_heads;
        if (qn || kn) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; i++) ss = fmaf(x[i], x[i], ss);
            ss = head_sum<LPH>(ss);
            const float inv = __builtin_amdgcn_rsqf(ss * (1.0f / D) + eps);
            if (!is_v && (is_q ? qn : kn)) {
#pragma unroll
                for (int i = 0; i < 8; i++) x[i] = x[i] * inv * (is_q ? qw[i] : kw[i]);
            }
        }
        if (interleaved) {
            if (!is_v && turned) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float4 a2 = reinterpret_cast<const float4*>(cs + r * (D / 2) + c8 * 4)[i / 2];
                    const float2 a = i % 2 ? make_float2(a2.z, a2.w) : make_float2(a2.x, a2.y);
                    const float p = x[2 * i], q = x[2 * i + 1];
                    x[2 * i] = p * a.x - q * a.y;
                    x[2 * i + 1] = q * a.x + p * a.y;
                }
            }
        } else if (R > 0) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; i++) y[i] = __shfl(x[i], pair_lane, WAVE);
            if (!is_v && turned) {
                const float4* ang = reinterpret_cast<const float4*>(cs + r * (D / 2) + pair_chunk * 8);
                const float sign = second ? 1.f : -1.f;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float4 a = ang[i];
                    x[2 * i] = fmaf(x[2 * i], a.x, sign * y[2 * i] * a.y);
                    x[2 * i + 1] = fmaf(x[2 * i + 1], a.z, sign * y[2 * i + 1] * a.w);
                }
            }
        }
        if (is_q) {
            uint4 o;
            o.x = pack2(x[0], x[1]); o.y = pack2(x[2], x[3]); o.z = pack2(x[4], x[5]); o.w = pack2(x[6], x[7]);
            *reinterpret_cast<uint4*>(q_out + ((int64_t)t * n_heads + h) * D + c8 * 8) = o;
        }
        if (all_q) return;
        const int kh = is_v ? h - n_heads - nk : h - n_heads;
        const int64_t ph = (int64_t)(slot >> cache.page_shift) * nk + kh;  // (page, head)
        const int off = slot & page_mask;
        const bool kv = !is_q && h < heads;
        if constexpr (F8) {
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < 8; i++) amax = (x[i] != x[i] || amax != amax) ? __builtin_nanf("") : fmaxf(amax, fabsf(x[i]));
#pragma unroll
            for (int d = 1; d < LPH; d <<= 1) {
                const float o = wave_xor(amax, d);
                amax = (o != o || amax != amax) ? __builtin_nanf("") : fmaxf(amax, o);
            }
            // element = x / (amax / 448) as (7/8 x) / (amax / 512): both operands are
            // exact for a bf16 x, so only the quotient rounds and a value that lies
            // halfway between two e4m3 goes to the even one.  A head of zeros (or so
            // small that amax / 512 would be subnormal) is stored as zeros of scale 0.
            float sc = amax / 448.0f, dv = amax * (1.0f / 512);
            if (sc < 2.36e-38f) { sc = 0.f; dv = 1.f; }
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; i++) y[i] = 0.875f * x[i] / dv;
            uint32_t a = 0, b = 0;
            a = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], a, false);
            a = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], a, true);
            b = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], b, false);
            b = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], b, true);
            // k: 16-element chunks, page_size of them side by side; v: rows
            const int64_t at = is_v ? (((ph << cache.page_shift) + off) * D + c8 * 8)
                                    : ((((ph * (D / 16) + (c8 >> 1)) << cache.page_shift) + off) * 16 + (c8 & 1) * 8);
            if (kv) {
                *reinterpret_cast<u32x2_r*>((uint8_t*)(is_v ? cache.v : cache.k) + at) = u32x2_r{a, b};
                if (c8 == 0) (is_v ? cache.v_scale : cache.k_scale)[(ph << cache.page_shift) + off] = sc;
            }
        } else {
            uint4 o;
            o.x = pack2(x[0], x[1]); o.y = pack2(x[2], x[3]); o.z = pack2(x[4], x[5]); o.w = pack2(x[6], x[7]);
            const int64_t at = is_v ? (((ph << cache.page_shift) + off) * D + c8 * 8)
                                    : ((((ph * (D / 8) + c8) << cache.page_shift) + off) * 8);
            if (kv) *reinterpret_cast<uint4*>((uint16_t*)(is_v ? cache.v : cache.k) + at) = o;
        }
    };
    for (int u0 = w; u0 < units; u0 += UN * NWV) {
        uint4 next[UN];
        if (u0 + UN * NWV < units) {
#pragma unroll
            for (int i = 0; i < UN; i++) next[i] = load(u0 + (UN + i) * NWV);
        }
#pragma unroll
        for (int i = 0; i < UN; i++)
            if (u0 + i * NWV < units) unit(u0 + i * NWV, raw[i]);
#pragma unroll
        for (int i = 0; i < UN; i++) raw[i] = next[i];
    }
}

template <int D, int F8, int TB, int UN>
void launch_t(int groups_per_block, const uint16_t* qkv, int64_t stride, int T, int n_heads, const KvView& cache,
              const float* qw, const float* kw, float eps, const float* inv_freq, int R, int inter, float rope_scale,
              const int32_t* positions, const int32_t* slots, uint16_t* q_out, hipStream_t st) {
    constexpr int HPW = WAVE / (D / 8);
    const int groups = (n_heads + 2 * cache.n_kv_heads + HPW - 1) / HPW;
    hipLaunchKernelGGL((k_qk_norm_rope<D, F8, TB, UN>),
                       dim3((T + TB - 1) / TB, (groups + groups_per_block - 1) / groups_per_block), dim3(ROPE_THREADS), 0,
                       st, qkv, stride, T, n_heads, cache, qw, kw, eps, inv_freq, R, inter, rope_scale, positions, slots,
                       q_out, groups_per_block);
}

template <int D, int F8>
hipError_t launch_d(const uint16_t* qkv, int64_t stride, int T, int n_heads, const KvView& cache, const float* qw,
                    const float* kw, float eps, const float* inv_freq, int R, int inter, float rope_scale,
                    const int32_t* positions, const int32_t* slots, uint16_t* q_out, hipStream_t st) {
    constexpr int HPW = WAVE / (D / 8);
    const int groups = (n_heads + 2 * cache.n_kv_heads + HPW - 1) / HPW;
    // 8 rows per block (their keys' 16-byte chunks fill whole lines), the heads
    // split until there are about 1024 blocks; few rows: one row and one group
    // of heads per wave.  Both sides, one row a wave first: 256 rows x 10 groups 4.7 us against 6.1,
    // 777 x 10 8.5 against 8.3, 777 x 12 (e4m3) 10.1 against 10.5, 1600 x 10 14.1 against 11.3, 8192 x 10 52
    // against 39.
    if ((int64_t)T * groups <= 10240)
        launch_t<D, F8, 1, 1>(4, qkv, stride, T, n_heads, cache, qw, kw, eps, inv_freq, R, inter, rope_scale, positions,
                              slots, q_out, st);
    else
        launch_t<D, F8, 8, 4>((int)std::max<int64_t>(std::min<int64_t>((int64_t)groups * ((T + 7) / 8) / 1024, groups), 2),
                              qkv, stride, T, n_heads, cache, qw, kw, eps, inv_freq, R, inter, rope_scale, positions,
                              slots, q_out, st);
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
