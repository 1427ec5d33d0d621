// linear.hip -- dense products with bias, activation and residual (gfx950).
//
//   out[t][n] = cast( act( sum_k x[t][k] w[n][k] + bias[n] ) + residual[t][n] )
//
// 64 x 64 output tiles, K steps of 64 through LDS, MFMA 16x16x32 bf16 with the
// weight as its first operand, so a lane's four results are consecutive
// outputs of one row.  Rows behind T and N are read as row 0 and not stored.
#include "attn.h"
#include "common.h"

namespace {

constexpr int LT_THREADS = 256;
typedef uint32_t u32x2_l __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_l __attribute__((ext_vector_type(2)));

enum { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_RELU = 4 };

MOE_DEV float activate(float z, int act) {
    switch (act) {
        case ACT_SILU: return z / (1.0f + expf(-z));
        case ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
        case ACT_GELU_TANH: return 0.5f * z * (1.0f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
        case ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    }
    return z;
}

MOE_DEV uint32_t pk(float lo, float hi) {
    const bf16x2_l v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

// four consecutive outputs of row t from n on (n % 4 == 0, N % 8 == 0)
template <int OB>
MOE_DEV void finish4(f32x4_t z, int64_t t, int n, int N, const float* bias, int act, const void* residual, void* out) {
    if (bias) z += *reinterpret_cast<const f32x4_t*>(bias + n);
#pragma unroll
    for (int i = 0; i < 4; i++) z[i] = activate(z[i], act);
    const int64_t o = t * N + n;
    if constexpr (OB) {
        if (residual) {
            const u32x2_l r = *reinterpret_cast<const u32x2_l*>((const uint16_t*)residual + o);
            z += f32x4_t{bf16lo_to_f32(r[0]), bf16hi_to_f32(r[0]), bf16lo_to_f32(r[1]), bf16hi_to_f32(r[1])};
        }
        *reinterpret_cast<u32x2_l*>((uint16_t*)out + o) = u32x2_l{pk(z[0], z[1]), pk(z[2], z[3])};
    } else {
        if (residual) z += *reinterpret_cast<const f32x4_t*>((const float*)residual + o);
        *reinterpret_cast<f32x4_t*>((float*)out + o) = z;
    }
}

template <int OB>
__global__ __launch_bounds__(LT_THREADS) void k_linear(const uint16_t* __restrict__ x, int64_t x_stride,
                                                       const uint16_t* __restrict__ w, const float* __restrict__ bias,
                                                       int act, const void* residual, int T, int N, int K, void* out) {
    constexpr int BT = 64, BN = 64, BK = 64, LR = BK + 8;       // padded LDS rows
    __shared__ __attribute__((aligned(16))) uint16_t xs[BT * LR], ws[BN * LR];
    const int n0 = blockIdx.x * BN;
    const int64_t t0 = (int64_t)blockIdx.y * BT;
    const int tid = threadIdx.x, l = lane_id(), wv = tid / WAVE;
    const int wn = (wv & 1) * 32, wt = (wv >> 1) * 32;
    f32x4_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < K; k0 += BK) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 2; c++) {
            const int q = c * LT_THREADS + tid, r = q >> 3, ch = q & 7;
            const int64_t t = t0 + r < T ? t0 + r : 0;
            const int64_t n = n0 + r < N ? n0 + r : 0;
            *reinterpret_cast<uint4*>(xs + r * LR + ch * 8) = *reinterpret_cast<const uint4*>(x + t * x_stride + k0 + ch * 8);
            *reinterpret_cast<uint4*>(ws + r * LR + ch * 8) = *reinterpret_cast<const uint4*>(w + n * K + k0 + ch * 8);
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < BK; kk += 32) {
            bf16x8_t a[2], b[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                a[i] = *reinterpret_cast<const bf16x8_t*>(ws + (wn + i * 16 + (l & 15)) * LR + kk + (l >> 4) * 8);
                b[i] = *reinterpret_cast<const bf16x8_t*>(xs + (wt + i * 16 + (l & 15)) * LR + kk + (l >> 4) * 8);
            }
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int j = 0; j < 2; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int64_t t = t0 + wt + j * 16 + (l & 15);
            const int n = n0 + wn + i * 16 + (l >> 4) * 4;
            if (t < T && n < N) finish4<OB>(acc[i][j], t, n, N, bias, act, residual, out);
        }
}

}  // namespace

size_t linear_workspace_bytes(int T, int N, int K) {
    (void)T; (void)N; (void)K;
    return 0;
}

hipError_t launch_linear(const uint16_t* x, int64_t x_stride, const uint16_t* w, const float* bias, int act,
                         const void* residual, int T, int N, int K, void* out, int out_bf16, void* ws,
                         hipStream_t st) {
    (void)ws;
    if (T == 0) return hipSuccess;
    const dim3 grid((N + 63) / 64, (T + 63) / 64);
    if (out_bf16) hipLaunchKernelGGL((k_linear<1>), grid, dim3(LT_THREADS), 0, st, x, x_stride, w, bias, act, residual, T, N, K, out);
    else hipLaunchKernelGGL((k_linear<0>), grid, dim3(LT_THREADS), 0, st, x, x_stride, w, bias, act, residual, T, N, K, out);
    return hipGetLastError();
}
