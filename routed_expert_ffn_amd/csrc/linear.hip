// linear.hip -- dense products with bias, activation and residual (gfx950).
//
//   out[t][n] = cast( act( sum_k x[t][k] w[n][k] + bias[n] ) + residual[t][n] )
//
// Two kernels.  Few rows (T <= 16): the weights are read once and that is the
// time, so k_linear_rows streams them through registers.  More rows: tiles of x
// and w through LDS, k_linear_tile.  Sums, bias, activation and residual in fp32,
// one rounding at the end.
#include "attn.h"
#include "common.h"
#include "device.h"

#include <algorithm>
#include <type_traits>

namespace {

typedef uint32_t u32x2_l __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_l __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_l __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_ptr;
typedef __amdgpu_buffer_rsrc_t rsrc_t;

enum { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_RELU = 4 };

// z / (1 + e^-y) by the hardware's exp2 and reciprocal (about 1 unit each)
MOE_DEV float gated(float z, float y) {
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896341f * y));
}
MOE_DEV float activate(float z, int act) {
    switch (act) {
        case ACT_SILU: return gated(z, z);
        case ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
        // 0.5 z (1 + tanh u) = z / (1 + e^-2u)
        case ACT_GELU_TANH: return gated(z, 1.59576912160573071f * (z + 0.044715f * z * z * z));
        case ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    }
    return z;
}

MOE_DEV uint32_t pk(float lo, float hi) {
    const bf16x2_l v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}
MOE_DEV int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// ------------------------------------------------------------------ few rows
// A block takes 4 RG weight rows, its 8 waves a share of k each: K is cut into
// steps of 128, wave w takes steps w KS .. w KS + KS - 1 of every 8 KS.  One load
// instruction of a wave is 4 rows x 128 k, 256 contiguous bytes a row: lane
// (r, g) = (l & 15, l >> 4) holds row r >> 2, chunk (16 bytes) 4 g + (r & 3).  As the
// MFMA's first operand that is a 16-row matrix whose row r holds the k of
// part r & 3 only, so there is one MFMA per part p, with the matching x chunks
// as its second operand, and of its 16 result rows those with r & 3 = p count:
// in result element i = p of each lane, row g, token l & 15.  Three quarters of
// the MFMA's work is thrown away, which costs nothing (T <= 16 leaves the matrix
// cores idle), and in return the loads need neither LDS nor narrow rows.
// A pass's loads go out at once: up to K = 2048 all of the block's.
// More than 16 rows: TT tiles of 16, each with its own second operands and results.
//   Bound: the weight's bytes, cold (a decode step reads each weight once).
// 5 x 5120 x 2048: 21 MB in 6.0 us, 3.5 TB/s, of which about 2.5 us are the launch and
// the first load's way to memory and back; the library's product of the same size
// is 8.9.
//   KS, the k steps per wave and pass, and so the loads in flight: 5 x 5120 x 2048 6.7 us
// with 1, 5.7 with 2, 7.6 with 4 (more registers, half of the steps past the end); 5 x 5120 x 8192 21.9,
// 17.6, 18.2; 16 x 5120 x 8192 26.2, 22.0, 21.5; at K = 512 1 and 2 are the same.
constexpr int ROWS_MAX_T = 32;
constexpr int RW = 8;                      // waves per block

template <int RG, int KS, int TT, int OB>
__global__ __launch_bounds__(RW * WAVE, 2) void k_linear_rows(const uint16_t* __restrict__ x, int x_stride,
                                                              const uint16_t* __restrict__ w, const float* __restrict__ bias,
                                                              int act, const void* residual, int T, int N, int K,
                                                              int rows_per_block, void* out) {
    __shared__ float red[RW][RG][TT][WAVE];
    const int l = lane_id(), wv = uni(threadIdx.x / WAVE), r = l & 15, g = l >> 4;
    const int n0 = blockIdx.x * rows_per_block, rows = min(rows_per_block, N - n0);
    const int kc = K / 8;                  // 16-byte chunks of a row
    // (chunks and rows past the end read as 0 without touching memory)
    const rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(w + (int64_t)n0 * K), 0, rows * K * 2, 0x00027000);
    const rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(x), 0, ((T - 1) * x_stride + K) * 2, 0x00027000);
    const int chunk = 4 * g + (r & 3);
    float val[RG][TT];
#pragma unroll
    for (int i = 0; i < RG; i++)
#pragma unroll
        for (int t = 0; t < TT; t++) val[i][t] = 0.f;
    for (int s0 = wv * KS; s0 * 16 < kc; s0 += RW * KS) {
        u32x4_l xf[TT][KS][4], wf[RG][KS];
#pragma unroll
        for (int t = 0; t < TT; t++)
#pragma unroll
            for (int s = 0; s < KS; s++)
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    const int c = (s0 + s) * 16 + 4 * g + p, row = 16 * t + r;
                    xf[t][s][p] = __builtin_bit_cast(u32x4_l, __builtin_amdgcn_raw_buffer_load_b128(
                                                                  xr, c < kc && row < T ? (row * x_stride + c * 8) * 2 : -16, 0, 0));
                }
#pragma unroll
        for (int i = 0; i < RG; i++)
#pragma unroll
            for (int s = 0; s < KS; s++) {
                const int c = (s0 + s) * 16 + chunk, row = 4 * i + (r >> 2);
                wf[i][s] = __builtin_bit_cast(u32x4_l, __builtin_amdgcn_raw_buffer_load_b128(
                                                           wr, c < kc && row < rows ? (row * K + c * 8) * 2 : -16, 0, 2));
            }
#pragma unroll
        for (int i = 0; i < RG; i++)
#pragma unroll
            for (int t = 0; t < TT; t++) {
                f32x4_t acc[4];
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    acc[p] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < KS; s++)
                        acc[p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, wf[i][s]),
                                                                         __builtin_bit_cast(bf16x8_t, xf[t][s][p]), acc[p], 0, 0, 0);
                }
                val[i][t] += (acc[0][0] + acc[1][1]) + (acc[2][2] + acc[3][3]);
            }
    }
#pragma unroll
    for (int i = 0; i < RG; i++)
#pragma unroll
        for (int t = 0; t < TT; t++) red[wv][i][t][l] = val[i][t];
    __syncthreads();
    // thread: output (t, row), the rows of a token side by side
    for (int id = threadIdx.x; id < T * rows; id += RW * WAVE) {
        const int t = id / rows, row = id - t * rows;
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < RW; i++) z += red[i][row >> 2][t >> 4][(row & 3) * 16 + (t & 15)];
        const int n = n0 + row;
        if (bias) z += bias[n];
        z = activate(z, act);
        const int64_t o = (int64_t)t * N + n;
        if constexpr (OB) {
            if (residual) z += bf16_to_f32(((const uint16_t*)residual)[o]);
            ((uint16_t*)out)[o] = (uint16_t)pk(z, 0.f);
        } else {
            if (residual) z += ((const float*)residual)[o];
            ((float*)out)[o] = z;
        }
    }
}

// ------------------------------------------------------------------ many rows
// BT x BN output tiles, K steps of BK through ST LDS stages filled by the LDS DMA
// (16 bytes a lane), ST - 1 steps ahead: a stage is waited for ST - 2 steps after
// its loads went out.  2 x WN waves, MFMA 16x16x32 with the weight as the
// first operand, so a lane's results are 4 consecutive outputs of one row.  The fragments of the next K step are read from LDS under the MFMAs of the
// current one, in two register sets.
//   LDS rows are BK elements; their 16-byte chunks are swizzled (on the global
// side of the DMA) so that the 16 lanes that a 16-byte read serves together fall
// into the 16 slots of 256 bytes (lanes 0-3, 12-15 and 20-27 are served together,
// 4-11, 16-19 and 28-31, and so on): BK 64, chunk ^ ((row >> 1) & 7); BK 32, chunk ^
// {0, 2, 3, 1}[(row >> 2) & 3].  No conflicts counted.
//   KG 2: two groups of waves take half of each K step each and add their sums at
// the end through LDS: with one block per CU twice the waves hide what a K step
// waits for (48 x 1000 x 8192, 4 stages each: 33 us with one group, 21 with two).
//   Bound: with many tiles the matrix cores and their feeding.  8192 x 2048 x 4096
// 115 us, 1.19 PFLOP/s (1.36 PFLOP/s is what a large library product reaches; its
// own time here is 92); 8 waves of 128 x 64 outputs each, two per SIMD, so that one
// issues MFMAs while the other waits at the barrier (4 waves of 128 x 128 reach 1.1 at
// best).  With few tiles the latency of a K step, 0.37 us per 128 of k and group.
//   Blocks: tiles of one XCD (block mod 8) are neighbours, in panels of 8 column
// tiles, so that they share x and w in its L2.
// s_waitcnt vmcnt(N) lgkmcnt(0): this wave's older loads have landed, its LDS reads
// are done (they went out a step of MFMAs ago; said here, or the compiler would
// wait for the next step's reads too)
template <int N>
MOE_DEV void wait_vm() {
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4));
}
MOE_DEV void dma16(const void* g, lds_ptr* l) { __builtin_amdgcn_global_load_lds(g, l, 16, 0, 0); }

template <int BT, int BN, int BK, int ST, int WN, int KG>
struct TileGeo {
    static constexpr int NWV = 2 * WN * KG;                  // waves: 2 along the rows, WN along the columns, KG along k
    static constexpr int WT = BT / 2, WNC = BN / WN;         // a wave's rows and columns
    static constexpr int IT = WT / 16, JT = WNC / 16;        // its MFMA tiles
    static constexpr int ROWB = BK * 2;                      // LDS row bytes
    static constexpr int STAGE = (BT + BN) * ROWB;
    static constexpr int RPI = 1024 / ROWB;                  // rows per DMA instruction (1 KB)
    static constexpr int DX = BT / RPI / NWV, DW = BN / RPI / NWV, DMA = DX + DW;   // per wave
    static_assert(DX * RPI * NWV == BT && DW * RPI * NWV == BN, "whole DMA instructions per wave");
    // epilogue: 32 rows x WNC columns fp32 per wave, rows padded by 16 bytes
    static constexpr int EROW = WNC * 4 + 16, EPI = 2 * WN * 32 * EROW;
    static constexpr int XCH = KG > 1 ? (KG - 1) * 2 * WN * IT * JT * 1024 : 0;      // sums of the other k groups
    static constexpr int LDS = STAGE * ST > EPI + XCH ? STAGE * ST : EPI + XCH;
};

template <int BT, int BN, int BK, int ST, int WN, int KG, int OB, int BPC>
__global__ __launch_bounds__(2 * WN * KG * WAVE, BPC * WN * KG / 2) void k_linear_tile(const uint16_t* __restrict__ x, int x_stride,
                                                                   const uint16_t* __restrict__ w,
                                                                   const float* __restrict__ bias, int act,
                                                                   const void* residual, int T, int N, int K, int tiles_t,
                                                                   int tiles_n, void* out) {
    using G = TileGeo<BT, BN, BK, ST, WN, KG>;
    constexpr int IT = G::IT, JT = G::JT, KQ = BK / 32 / KG; // MFMA steps per K step and wave
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int l = lane_id(), wv = uni(threadIdx.x / WAVE), kg = wv / (2 * WN), w4 = wv % (2 * WN), wt = w4 / WN, wn = w4 % WN;
    // tile of this block
    const int tiles = tiles_t * tiles_n, per = (tiles + 7) / 8;
    const int id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || id >= tiles) return;
    constexpr int PN = 8;
    const int panel = id / (tiles_t * PN), pw = min(PN, tiles_n - panel * PN), in = id - panel * tiles_t * PN;
    const int64_t t0 = (int64_t)(in / pw) * BT;
    const int n0 = (panel * PN + in % pw) * BN;
    const int rows_t = (int)min((int64_t)BT, T - t0), rows_n = min(BN, N - n0);

    // DMA: lane -> row l / CPR of the instruction's rows, LDS chunk l % CPR, which
    // holds global chunk (l % CPR) ^ swizzle(row).  Rows past the end repeat the last.
    constexpr int CPR = G::ROWB / 16;
    auto swz = [](int row) __attribute__((always_inline)) {
        return BK == 128 ? row & 15 : BK == 64 ? (row >> 1) & 7 : (((row >> 2) ^ (row >> 3)) & 1) * 2 + ((row >> 3) & 1);
    };
    const unsigned char* xb = (const unsigned char*)(x + t0 * x_stride);
    const unsigned char* wb = (const unsigned char*)(w + (int64_t)n0 * K);
    uint32_t xo[G::DX], wo[G::DW];
#pragma unroll
    for (int i = 0; i < G::DX; i++) {
        const int r = (wv * G::DX + i) * G::RPI + l / CPR;
        xo[i] = (uint32_t)min(r, rows_t - 1) * (uint32_t)(x_stride * 2) + (uint32_t)(((l % CPR) ^ swz(r)) * 16);
    }
#pragma unroll
    for (int i = 0; i < G::DW; i++) {
        const int r = (wv * G::DW + i) * G::RPI + l / CPR;
        wo[i] = (uint32_t)min(r, rows_n - 1) * (uint32_t)(K * 2) + (uint32_t)(((l % CPR) ^ swz(r)) * 16);
    }
    const int nk = K / BK;                  // whole steps; BK 128: K may leave half a step over
    const bool rest = BK == 128 && K % BK != 0;
    const int last = rest ? nk : nk - 1;
    auto issue = [&](int k) __attribute__((always_inline)) {
        unsigned char* st = smem + (k % ST) * G::STAGE;
        k = min(k, last);
        // (in the half step the second half's lanes load the first half again, unused)
#pragma unroll
        for (int i = 0; i < G::DX; i++) {
            uint32_t o = xo[i];
            if (BK == 128 && rest && k == nk && (((l % CPR) ^ swz((wv * G::DX + i) * G::RPI + l / CPR)) >= 8)) o -= 128;
            dma16(xb + (int64_t)k * G::ROWB + o, (lds_ptr*)(st + (wv * G::DX + i) * 1024));
        }
#pragma unroll
        for (int i = 0; i < G::DW; i++) {
            uint32_t o = wo[i];
            if (BK == 128 && rest && k == nk && (((l % CPR) ^ swz((wv * G::DW + i) * G::RPI + l / CPR)) >= 8)) o -= 128;
            dma16(wb + (int64_t)k * G::ROWB + o, (lds_ptr*)(st + BT * G::ROWB + (wv * G::DW + i) * 1024));
        }
    };
    const int fr = l & 15, fh = l >> 4;
    struct Frag { bf16x8_t x[IT][KQ], w[JT][KQ]; };
    auto read = [&](Frag& f, int k) __attribute__((always_inline)) {
        const unsigned char* st = smem + (k % ST) * G::STAGE;
#pragma unroll
        for (int q = 0; q < KQ; q++) {
            const int c = (kg * KQ + q) * 4 + fh;
#pragma unroll
            for (int i = 0; i < IT; i++) {
                const int r = wt * G::WT + i * 16 + fr;
                f.x[i][q] = *reinterpret_cast<const bf16x8_t*>(st + r * G::ROWB + ((c ^ swz(r)) * 16));
            }
#pragma unroll
            for (int j = 0; j < JT; j++) {
                const int r = wn * G::WNC + j * 16 + fr;
                f.w[j][q] = *reinterpret_cast<const bf16x8_t*>(st + BT * G::ROWB + r * G::ROWB + ((c ^ swz(r)) * 16));
            }
        }
    };
    f32x4_t acc[IT][JT];
#pragma unroll
    for (int i = 0; i < IT; i++)
#pragma unroll
        for (int j = 0; j < JT; j++) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto mma = [&](const Frag& f) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < KQ; q++)
#pragma unroll
            for (int i = 0; i < IT; i++)
#pragma unroll
                for (int j = 0; j < JT; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.w[j][q], f.x[i][q], acc[i][j], 0, 0, 0);
    };
    // One K step: stage k + 1 has landed everywhere (each wave waits for its own
    // loads, then the barrier); the next fragments are read under this step's
    // MFMAs; stage k - 1, read one step earlier still, is free and takes the loads
    // of step k + ST - 1.  Every step is the same, with no branch that would make
    // the MFMAs wait: behind the last one the last K block is loaded again and the
    // fragments read go unused.
    auto step = [&](int k, Frag& cur, Frag& nxt) __attribute__((always_inline)) {
        wait_vm<G::DMA * (ST - 3)>();
        __builtin_amdgcn_s_barrier();
        read(nxt, k + 1);
        issue(k + ST - 1);
        mma(cur);
        constexpr int NM = IT * JT * KQ, NR = (IT + JT) * KQ, H = NM / 2 < 16 ? NM / 2 : 16;
#pragma unroll
        for (int q = 0; q < H; q++) {
            __builtin_amdgcn_sched_group_barrier(0x100, (NR + H - 1) / H, 0);        // LDS reads
            __builtin_amdgcn_sched_group_barrier(0x008, NM / H / 2, 0);              // MFMA
        }
#pragma unroll
        for (int q = 0; q < H; q++) {
            __builtin_amdgcn_sched_group_barrier(0x020, (G::DMA + H - 1) / H, 0);    // LDS DMA
            __builtin_amdgcn_sched_group_barrier(0x008, NM / H / 2, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int s = 0; s < ST - 1; s++) issue(s);
    Frag f0, f1;
    wait_vm<G::DMA * (ST - 2)>();
    __builtin_amdgcn_s_barrier();
    read(f0, 0);
    for (int k = 0; k + 1 < nk; k += 2) {
        step(k, f0, f1);
        step(k + 1, f1, f0);
    }
    if constexpr (BK >= 64) {               // (K is a multiple of 64: an even number of steps of 32)
        if (nk & 1) step(nk - 1, f0, f1);
        if (rest && kg == 0) mma(nk & 1 ? f1 : f0);          // the half step, read under the last whole one
    }
    wait_vm<0>();

    // ---- epilogue: 32 rows of the wave's tile at a time through its part of the
    // LDS, then 8 consecutive outputs a lane
    __syncthreads();                                          // every wave has read its last fragments, every load has landed
    if constexpr (KG > 1) {                                   // the k groups' sums meet in the first
        f32x4_t* xch = reinterpret_cast<f32x4_t*>(smem + G::EPI);
        if (kg > 0) {
#pragma unroll
            for (int i = 0; i < IT; i++)
#pragma unroll
                for (int j = 0; j < JT; j++) xch[((wv - 2 * WN) * IT * JT + i * JT + j) * WAVE + l] = acc[i][j];
        }
        __syncthreads();
        if (kg > 0) return;
#pragma unroll
        for (int k2 = 0; k2 < KG - 1; k2++)
#pragma unroll
            for (int i = 0; i < IT; i++)
#pragma unroll
                for (int j = 0; j < JT; j++) acc[i][j] += xch[((k2 * 2 * WN + w4) * IT * JT + i * JT + j) * WAVE + l];
    }
    unsigned char* ep = smem + w4 * 32 * G::EROW;
    constexpr int LPR = G::WNC / 8, RPP = WAVE / LPR, NP = 32 / RPP;     // lanes per row, rows per pass, passes
    const int er = l / LPR, ec = l % LPR * 8, n = n0 + wn * G::WNC + ec;
    f32x4_t b[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if (bias && n < N) {
        b[0] = *reinterpret_cast<const f32x4_t*>(bias + n);
        b[1] = *reinterpret_cast<const f32x4_t*>(bias + n + 4);
    }
    auto fence = [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
        __builtin_amdgcn_wave_barrier();
    };
#pragma unroll 1
    for (int i = 0; i < IT / 2; i++) {
        // all of the block's residual goes out first
        const int64_t tw = t0 + wt * G::WT + i * 32 + er, ow = tw * N + n;
        u32x4_l rv[NP][OB ? 1 : 2];
        if (residual) {
#pragma unroll
            for (int q = 0; q < NP; q++) {
                if (tw + q * RPP < T && n < N) {
                    const int64_t o = ow + (int64_t)q * RPP * N;
                    if constexpr (OB) {
                        rv[q][0] = *reinterpret_cast<const u32x4_l*>((const uint16_t*)residual + o);
                    } else {
                        rv[q][0] = *reinterpret_cast<const u32x4_l*>((const float*)residual + o);
                        rv[q][OB ? 0 : 1] = *reinterpret_cast<const u32x4_l*>((const float*)residual + o + 4);
                    }
                }
            }
        }
#pragma unroll
        for (int q = 0; q < IT; q++) {
            if (i != q / 2) continue;                         // uniform
#pragma unroll
            for (int j = 0; j < JT; j++)
                *reinterpret_cast<f32x4_t*>(ep + (q % 2 * 16 + fr) * G::EROW + (j * 16 + fh * 4) * 4) = acc[q][j];
        }
        fence();
        if (act != ACT_NONE) {                                // in place, a loop of its own
#pragma unroll 1
            for (int q = 0; q < 2 * NP; q++) {
                f32x4_t* z = reinterpret_cast<f32x4_t*>(ep + (q / 2 * RPP + er) * G::EROW + ec * 4 + (q & 1) * 16);
                f32x4_t y = *z + (q & 1 ? b[1] : b[0]);
#pragma unroll
                for (int e = 0; e < 4; e++) y[e] = activate(y[e], act);
                *z = y;
            }
            fence();
        }
#pragma unroll
        for (int q = 0; q < NP; q++) {
            const float* src = reinterpret_cast<const float*>(ep + (q * RPP + er) * G::EROW + ec * 4);
            f32x4_t z[2] = {*reinterpret_cast<const f32x4_t*>(src), *reinterpret_cast<const f32x4_t*>(src + 4)};
            if (tw + q * RPP >= T || n >= N) continue;
            if (act == ACT_NONE) {
                z[0] += b[0];
                z[1] += b[1];
            }
            const int64_t o = ow + (int64_t)q * RPP * N;
            if constexpr (OB) {
                if (residual) {
                    const u32x4_l r = rv[q][0];
                    z[0] += f32x4_t{bf16lo_to_f32(r[0]), bf16hi_to_f32(r[0]), bf16lo_to_f32(r[1]), bf16hi_to_f32(r[1])};
                    z[1] += f32x4_t{bf16lo_to_f32(r[2]), bf16hi_to_f32(r[2]), bf16lo_to_f32(r[3]), bf16hi_to_f32(r[3])};
                }
                *reinterpret_cast<u32x4_l*>((uint16_t*)out + o) =
                    u32x4_l{pk(z[0][0], z[0][1]), pk(z[0][2], z[0][3]), pk(z[1][0], z[1][1]), pk(z[1][2], z[1][3])};
            } else {
                if (residual) {
                    z[0] += __builtin_bit_cast(f32x4_t, rv[q][0]);
                    z[1] += __builtin_bit_cast(f32x4_t, rv[q][OB ? 0 : 1]);
                }
                *reinterpret_cast<f32x4_t*>((float*)out + o) = z[0];
                *reinterpret_cast<f32x4_t*>((float*)out + o + 4) = z[1];
            }
        }
        fence();
    }
}

struct LinearArgs {
    const uint16_t* x;
    int x_stride;
    const uint16_t* w;
    const float* bias;
    int act;
    const void* residual;
    int T, N, K;
    void* out;
};

template <int RG, int KS, int TT, int OB>
hipError_t launch_rows(const LinearArgs& a, int rows_per_block, hipStream_t st) {
    hipLaunchKernelGGL((k_linear_rows<RG, KS, TT, OB>), dim3((a.N + rows_per_block - 1) / rows_per_block), dim3(RW * WAVE),
                       0, st, a.x, a.x_stride, a.w, a.bias, a.act, a.residual, a.T, a.N, a.K, rows_per_block, a.out);
    return hipGetLastError();
}

template <int OB>
hipError_t launch_few(const LinearArgs& a, hipStream_t st) {
    // one block per CU while it has at most 32 weight rows
    const int groups = (a.N + 3) / 4, rg = std::min(std::max((groups + 255) / 256, 1), 8);
    if (a.T > 16) return launch_rows<2, 1, 2, OB>(a, 4 * rg, st);            // (N <= 2048: rg is 1 or 2)
    if (rg == 1) return launch_rows<1, 2, 1, OB>(a, 4, st);
    if (rg == 2) return launch_rows<2, 2, 1, OB>(a, 8, st);
    if (rg <= 4) return launch_rows<4, 2, 1, OB>(a, 4 * rg, st);
    return launch_rows<8, 2, 1, OB>(a, 4 * rg, st);
}

template <int BT, int BN, int BK, int ST, int WN, int KG, int BPC, int OB>
hipError_t launch_tile(const LinearArgs& a, hipStream_t st) {
    auto kern = k_linear_tile<BT, BN, BK, ST, WN, KG, OB, BPC>;
    static LdsLimit lim;
    constexpr int lds = TileGeo<BT, BN, BK, ST, WN, KG>::LDS;
    hipError_t e = lim.ensure((const void*)kern, lds);
    if (e != hipSuccess) return e;
    const int tt = (a.T + BT - 1) / BT, tn = (a.N + BN - 1) / BN, per = (tt * tn + 7) / 8;
    hipLaunchKernelGGL(kern, dim3(per * 8), dim3(2 * WN * KG * WAVE), lds, st, a.x, a.x_stride, a.w, a.bias, a.act, a.residual,
                       a.T, a.N, a.K, tt, tn, a.out);
    return hipGetLastError();
}

template <int OB>
hipError_t launch_ob(const LinearArgs& a, hipStream_t st) {
    // Few rows: 17 to 32 rows cost the rows kernel a second product per weight, which
    // narrow weights hide (24 x 2048 x 8192: 19.5 us, tiles 23) and wide ones do not (24 x 5120 x 8192:
    // 38, tiles 24); from 33 rows on tiles are as good throughout.
    if (a.T <= 16 || (a.T <= ROWS_MAX_T && a.N <= 2048)) {
        return launch_few<OB>(a, st);
    }
    auto tiles = [&](int b) { return (int64_t)((a.T + b - 1) / b) * ((a.N + b - 1) / b); };
    auto rounds = [&](int b) { return (tiles(b) + 255) / 256; };             // tiles a CU is given
    // Which tile: a CU works off its tiles one after the other or two side by side,
    // and the time of a round is that of its slowest CU, so each size's time is that of
    // a round times the rounds, in units that fit the times at K = 2048 (us: 64-square 9
    // for a lone tile, 7 per tile and CU after that, 128-square 23 and 18, 256-square
    // 44).  Both sides: 1600 x 5120 x 2048, 256-square 46 us, 128 57, 64 57; 3200 x 5120 x 512
    // (260 of the largest, a second round for four of them) 36, 28, 38; 3200 x 2048 x 2048 45, 37, 48;
    // 800 x 2048 x 8192 137, 74, 48.  Over 90 sizes up to 8192 rows the choice was the best
    // one or within 8 percent of it, but for 4000 x 768 x 1024 (15.4 against 12.3).
    const int64_t c64 = rounds(64) == 1 ? 9 : rounds(64) * 7, c128 = rounds(128) == 1 ? 23 : rounds(128) * 18,
                  c256 = rounds(256) * 44;
    if (c256 < c128 && c256 < c64) return launch_tile<256, 256, 32, 4, 4, 1, 1, OB>(a, st);
    if (c128 < c64) return launch_tile<128, 128, 32, 4, 2, 1, 2, OB>(a, st);
    // One 64-square tile per CU: six stages, or from K = 2048 on two k groups.  Weights
    // from memory, 4 stages against 6: 333 x 1000 x 1088 7.8 us and 6.9, 333 x 1000 x 1920 13.9 and 11.2
    // (8 stages: 7.2 and 11.4).  Six stages against two groups: weights in the caches, 48 x 1000 x 8192
    // 26.2 us and 21.2, 400 x 2048 x 8192 31.7 and 26.9, 333 x 1000 x 2048 9.5 and 8.8; from memory the two
    // are within 5 percent (32.9 and 34.1, 35.8 and 35.3, 11.3 and 11.7).
    if (tiles(64) <= 256)
        return a.K >= 2048 ? launch_tile<64, 64, 128, 4, 2, 2, 1, OB>(a, st) : launch_tile<64, 64, 64, 6, 2, 1, 1, OB>(a, st);
    return launch_tile<64, 64, 64, 4, 2, 1, 2, OB>(a, st);
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
    const LinearArgs a{x, (int)x_stride, w, bias, act, residual, T, N, K, out};
    return out_bf16 ? launch_ob<1>(a, st) : launch_ob<0>(a, st);
}
