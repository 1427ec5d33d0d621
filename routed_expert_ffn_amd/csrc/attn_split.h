// attn_split.h -- what the two attention kernels share: their arguments, the cutting
// of the work into shares, and the kernel that joins a unit's shares.
#pragma once
#include "attn.h"
#include "common.h"
#include "stream.h"

struct AttnArgs {
    const uint16_t* q;
    int64_t q_stride;
    int T, n_heads;
    KvView kv;
    const int32_t* table;
    int W;
    const int32_t* q_offsets;
    const int32_t* kv_len;
    int S;
    float scale, softcap;
    int window;
    uint16_t* out;
    int G;                                  // query heads per key-value head
    int G16;                                // ceil(2^16 / G): x / G = x G16 >> 16 for x < 1024
    int whole;                              // no unit is split: each goes to the share that its first step lies in
    int shares;                             // blocks of the attention launch
    int* share;                             // [1] steps per share, written by block 0 for the join
    int* base;                              // [S] first step of each request
    float* part;                            // [2 shares][rows][D] unnormalised sums
    float2* ml;                             // [2 shares][rows] (maximum, sum)
};

// prompt_attn.hip
struct PromptShape { int rows, shares; };
PromptShape prompt_attn_shape();
hipError_t launch_prompt_attn(const AttnArgs& a, hipStream_t st);

namespace {

constexpr int AT_THREADS = 256;             // of the few-row kernel and of the one-wave joins
// What a piece costs besides its own positions (its q rows, first loads and
// join), in positions: short requests would otherwise pile up in few shares (40 requests of
// up to 600 positions 14 us; at 512 positions a piece 16).
constexpr int PIECE_COST = 128;
constexpr float LOG2E = 1.44269504088896341f;

typedef uint32_t u32x2_a __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_a __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_a __attribute__((ext_vector_type(2)));
typedef short s16x4_a __attribute__((ext_vector_type(4)));

MOE_DEV int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
MOE_DEV uint32_t pk_bf16(float lo, float hi) {
    const bf16x2_a v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}
// two e4m3 of word w (its low or high half) -> packed bf16 (exact)
template <bool HI>
MOE_DEV uint32_t fp8x2_bf16(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}

// What a block needs of a request: its row range, positions and units.
struct Request {
    int row0, n, first;                     // first batch row, rows, position of its first row
    int len;                                // positions that the table can hold
    int units;                              // row groups * key-value heads
    int steps;                              // cost of each unit of its first row group, in steps
    int grow;                               // what a unit of the next row group costs more
};
// RB rows per unit.  GROW: a request's row groups see more positions the later
// they are (a prompt's first rows next to nothing), and their cost follows.
template <int RB, int STEP, bool GROW>
MOE_DEV Request request_of(const AttnArgs& a, int s) {
    Request r;
    const int b = min(max(a.q_offsets[s], 0), a.T), e = min(max(a.q_offsets[s + 1], 0), a.T);
    const int L = min(max(a.kv_len[s], 0), 1 << 30);
    r.row0 = b;
    r.n = max(e - b, 0);
    r.first = L - r.n;
    r.len = (int)min((int64_t)L, (int64_t)a.W << a.kv.page_shift);
    const int lo = a.window > 0 ? max(r.first - a.window + 1, 0) : 0;
    // (rows before position 0 or behind the table see nothing more: their cost would outgrow int32)
    r.grow = GROW && a.window == 0 && r.first >= 0 && r.len == L ? (RB + STEP * a.G / 2) / (STEP * a.G) : 0;
    const int hi = GROW ? (int)min((int64_t)r.len, (int64_t)max(r.first, 0) + RB / a.G) : r.len;
    r.units = (int)(((uint32_t)(r.n * a.G) + RB - 1) / RB) * a.kv.n_kv_heads;      // (T * n_heads fits int32)
    r.steps = (max(hi - lo, 0) + STEP - 1) / STEP + PIECE_COST / STEP;
    return r;
}
// steps of the units before row group grp
MOE_DEV int steps_before(const Request& r, int nkv, int grp) {
    return nkv * (r.steps * grp + r.grow * (int)((uint32_t)grp * (uint32_t)(grp - 1) / 2));
}

// the page table through the scalar cache (nothing writes it while the kernel runs)
typedef const __attribute__((address_space(4))) int32_t* table_ptr;

// First element of four consecutive results c of a row as the second product
// leaves them, (h, e, 4 g + i): elements 16 E h + E (4 g + i) + e, i = 0 .. 3.
template <int D>
MOE_DEV int dim_of(int c) {
    constexpr int E = D == 64 ? 4 : 8;
    const int g = c & 3, e = (c >> 2) % E, h = (c >> 2) / E;
    return 16 * E * h + 4 * E * g + e;
}

// The request that batch row t lies in, searched by a wave: 64 offsets at a time.
MOE_DEV int request_with(const AttnArgs& a, int t) {
    const int l = lane_id();
    int s = 0, stride = 1;
    while (stride * WAVE < a.S) stride *= WAVE;
    for (; stride >= 1; stride /= WAVE) {
        const int i = s + l * stride;
        s += max(__popcll(__ballot(i < a.S && a.q_offsets[min(i, a.S - 1)] <= t)) - 1, 0) * stride;
    }
    return uniform(s);
}

// out = sum_c 2^{m_c - M} acc_c / sum_c 2^{m_c - M} sum_c over the shares c that a
// unit lies in.  WPR waves per (batch row, head, CH elements): CH / 4 lanes of 4
// elements each, the shares dealt to the groups of them in all WPR waves, joined
// across lanes and then through LDS in order.  Few rows take CH 64 and 16 or 4
// waves (a unit in hundreds of shares; one token over 262,144 positions: 11 us
// with 4 waves, 6 with 16), many rows one wave each (most of them in one share,
// with nothing to do).
//   Whole prompts: most rows have nothing to join, and looking that up is all that
// their wave does: four rows a wave (8192 rows of 32 heads of 128: one row a wave
// 86 us, four 56).
constexpr int join_rows(bool GROW, int WPR) { return GROW && WPR == 1 ? 4 : 1; }
template <int D, int RB, int STEP, bool GROW, int CH, int WPR>
__global__ __launch_bounds__(WPR == 1 ? AT_THREADS : WPR * WAVE) void k_attn_join(const AttnArgs a) {
    constexpr int NW = AT_THREADS / WAVE, NC = D / CH, TC = CH / 4, GW = WAVE / TC, NG = GW * WPR;
    constexpr int U = 4;                   // shares in flight per thread
    constexpr int TPW = join_rows(GROW, WPR);
    __shared__ float2 gml[WPR];
    __shared__ f32x4_t go[WPR][TC];
    const int l = lane_id(), w = uniform(threadIdx.x / WAVE);
    const int y = WPR == 1 ? blockIdx.y * NW + w : blockIdx.y, hq = y / NC, c0 = y % NC * TC;
    const int share = a.share[0];
    Request rq;
    int s = 0;
#pragma unroll 1
    for (int n = 0; n < TPW; n++) {
        const int t = blockIdx.x * TPW + n;
        if (TPW > 1 && t >= a.T) return;
        if (n == 0 || t >= rq.row0 + rq.n) {
            s = request_with(a, t);
            rq = request_of<RB, STEP, GROW>(a, s);
        }
        if (hq >= a.n_heads || t < rq.row0 || t >= rq.row0 + rq.n) continue;
        const int nkv = a.kv.n_kv_heads, G = a.G;
        const int head = hq / G, row = (t - rq.row0) * G + (hq - head * G);
        const int grp = row / RB, rr = row - grp * RB;
        const int cost = rq.steps + rq.grow * grp;
        const int u0 = a.base[s] + steps_before(rq, nkv, grp) + head * cost;    // the unit's first step
        // (at most shares - 1 <= 511: the fp32 quotient is off by one at most)
        auto share_of = [&](int u) {
            const int q = (int)((float)u * __builtin_amdgcn_rcpf((float)share));
            return q + ((int64_t)(q + 1) * share <= u ? 1 : 0) - ((int64_t)q * share > u ? 1 : 0);
        };
        const int b0 = share_of(u0), np = share_of(u0 + cost - 1) - b0 + 1;
        if (np <= 1 || b0 < 0 || b0 + np > a.shares) continue;   // (past the shares only with offsets that do not ascend)
        const int first_odd = u0 == b0 * share ? 0 : 1;
        const int e = l % TC, gr = (WPR == 1 ? 0 : w * GW) + l / TC;
        float M = -__builtin_inff(), L = 0.f;
        f32x4_t o = {0.f, 0.f, 0.f, 0.f};
        auto add = [&](float m2, float l2, f32x4_t v2) __attribute__((always_inline)) {
            const float mn = fmaxf(M, m2), base = mn == -__builtin_inff() ? 0.f : mn;
            const float f0 = __builtin_amdgcn_exp2f(M - base), f1 = __builtin_amdgcn_exp2f(m2 - base);
            L = L * f0 + l2 * f1;
            o = o * f0 + v2 * f1;
            M = mn;
        };
        for (int p0 = gr; p0 < np; p0 += NG * U) {
            float2 x[U];
            f32x4_t v[U];
#pragma unroll
            for (int i = 0; i < U; i++) {
                const int p = min(p0 + i * NG, np - 1);
                const int64_t at = (2 * (int64_t)(b0 + p) + (p == 0 ? first_odd : 0)) * RB + rr;
                x[i] = a.ml[at];
                v[i] = *reinterpret_cast<const f32x4_t*>(a.part + at * D + (c0 + e) * 4);
            }
#pragma unroll
            for (int i = 0; i < U; i++) {
                if (p0 + i * NG >= np) break;
                add(x[i].x, x[i].y, v[i]);
            }
        }
        // the wave's groups: every lane ends with the sum over them, taken in the
        // same order (its own pair's lower group first)
#pragma unroll
        for (int d = TC; d < WAVE; d <<= 1) {
            const bool low = (l & d) == 0;
            const float m2 = wave_xor(M, d), l2 = wave_xor(L, d);
            f32x4_t v2;
#pragma unroll
            for (int i = 0; i < 4; i++) v2[i] = wave_xor(o[i], d);
            const float m1 = M, l1 = L;
            const f32x4_t v1 = o;
            M = low ? m1 : m2; L = low ? l1 : l2; o = low ? v1 : v2;
            add(low ? m2 : m1, low ? l2 : l1, low ? v2 : v1);
        }
        if constexpr (WPR > 1) {
            if (l < TC) go[w][l] = o;
            if (l == 0) gml[w] = make_float2(M, L);
            __syncthreads();
            if (threadIdx.x >= TC) continue;
            M = -__builtin_inff();
            L = 0.f;
            o = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int i = 0; i < WPR; i++) add(gml[i].x, gml[i].y, go[i][e]);
        } else if (l >= TC) {
            continue;
        }
        const float inv = L == 0.f ? 0.f : __builtin_amdgcn_rcpf(L);
        uint16_t* dst = a.out + ((int64_t)t * a.n_heads + hq) * D + dim_of<D>(c0 + e);
#pragma unroll
        for (int i = 0; i < 4; i++) dst[(D == 64 ? 4 : 8) * i] = (uint16_t)pk_bf16(o[i] * inv, 0.f);
    }
}

}  // namespace
