// prompt_attn.hip -- attention over the paged cache for requests of many new rows
// (gfx950): paged_attn.hip's formulas, arguments and shares, but with the cache's
// tiles in LDS, where all waves of a block use them.
//
// A block takes 256 rows (query token x query head of one key-value head), each of
// its 8 waves 32 of them with their q fragments and sums in registers:
//   S^T[position][row] = K Q^T      MFMA 16x16x32 bf16, 32 positions at a time
//   O^T[d][row]       += V^T P^T    MFMA 16x16x32 bf16, k = the 32 positions
// with the same lane layouts as there: P goes from the first product's result into
// the second's operand within the lane, a byte permute pairs up two positions'
// values.  A wave's fragment of K or V, 1 KB from LDS, meets two row tiles; two waves
// per SIMD, so that one's softmax runs beside the other's MFMAs.
//
// LDS: three stages of 32 positions (64 below head_dim 256), filled by the DMA two
// stages ahead, one barrier a stage.  Keys as in their pages, [chunk][16 positions], so
// that a fragment is 1 KB in a row; of the values' rows, position 4 g + j is row 4 j + g:
// rows read together are neighbours, 256 bytes and more side by side.
//
// Bound by compute: 8192 causal rows over 8192 positions, 32 heads of 128 on 8, 0.55
// TFLOP in 751 us (0.73 PFLOP/s), where the softmax's vector instructions take about as long
// as the MFMAs; 16 heads of 256 on 2 in 1008 us (0.55 PFLOP/s), where by count the LDS
// reads do (each fragment feeds two MFMAs only) and q and the sums fill the registers.
// 256 rows a block, one block per CU: with four waves of 32 rows twice the LDS
// would be filled per row.
#include "attn_split.h"
#include "device.h"

namespace {

constexpr int PROMPT_WAVES = 8, PROMPT_THREADS = PROMPT_WAVES * WAVE;
constexpr int PMT = 2;                      // row tiles per wave
constexpr int PROMPT_ROWS = PROMPT_WAVES * PMT * 16;
constexpr int PROMPT_SHARES = 256;          // one block per CU
constexpr int TICK = 16;                    // positions per step of the shares

template <int D, int F8>
struct Stage {
    static constexpr int ES = F8 ? 1 : 2, X = 16 / ES;       // element bytes, elements per key chunk
    static constexpr int HALVES = D == 256 ? 1 : 2;          // 32 positions each
    static constexpr int SUB = 2 * HALVES, POS = 16 * SUB;   // sub-tiles of 16 positions
    static constexpr int KB = 16 * D * ES, KI = KB / 1024;   // bytes and DMA instructions of a sub-tile's keys (values the same)
    static constexpr int SCALES = SUB * 2 * KB;              // then [sub-tile][k, v][16] scales
    static constexpr int BYTES = SCALES + (F8 ? SUB * 128 : 0);
    static constexpr int ST = 3;
    static constexpr int DX = SUB * 2 * KI / PROMPT_WAVES;   // DMA instructions per wave
    static constexpr int DMA = DX + (F8 ? HALVES : 0);
    static_assert(DX * PROMPT_WAVES == SUB * 2 * KI && DX <= 2 * KI, "a wave's instructions lie in one sub-tile");
};

typedef __attribute__((address_space(3))) void lds_void;
// s_waitcnt vmcnt(N) lgkmcnt(0)
template <int N>
MOE_DEV void wait_loads() {
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4));
}

MOE_DEV void dma16(const void* g, void* lds) { __builtin_amdgcn_global_load_lds(g, (lds_void*)lds, 16, 0, 0); }
MOE_DEV void dma4(const void* g, void* lds) { __builtin_amdgcn_global_load_lds(g, (lds_void*)lds, 4, 0, 0); }

template <int D, int F8>
__global__ __launch_bounds__(PROMPT_THREADS, 2) void k_prompt_attn(const AttnArgs a) {
    using SG = Stage<D, F8>;
    constexpr int RB = PROMPT_ROWS, ES = SG::ES, X = SG::X, KB = SG::KB;
    constexpr int E = D == 64 ? 4 : 8;              // value elements per lane and read
    constexpr int NH = D / (16 * E);                // reads per position
    constexpr int EW = F8 ? E / 4 : E / 2;          // their 32-bit words
    constexpr int PER = F8 ? 4 : 2;                 // elements per word
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    int* base = (int*)(smem + SG::BYTES * SG::ST);  // [S] first steps
    __shared__ int sc32[PROMPT_WAVES];

    const int tid = threadIdx.x, l = lane_id(), w = uniform(tid / WAVE), r16 = l & 15, g4 = l >> 4;
    const int G = a.G, nkv = a.kv.n_kv_heads;

    // ---- first step of every request
    int total = 0;
    for (int s0 = 0; s0 < a.S; s0 += PROMPT_THREADS) {
        const int s = s0 + tid;
        int c = 0;
        if (s < a.S) {
            const Request r = request_of<RB, TICK, true>(a, s);
            c = steps_before(r, nkv, r.units / nkv);
        }
        const int incl = wave_incl_scan(c);
        __syncthreads();                    // the scratch's last readers are done
        if (l == WAVE - 1) sc32[w] = incl;
        __syncthreads();
        int b = total;
#pragma unroll
        for (int i = 0; i < PROMPT_WAVES; i++) {
            if (i < w) b += sc32[i];
            total += sc32[i];
        }
        if (s < a.S) {
            base[s] = b + incl - c;
            if (blockIdx.x == 0) a.base[s] = b + incl - c;
        }
    }
    __syncthreads();
    total = uniform(total);
    const int share = max((int)(((uint32_t)total + a.shares - 1) / a.shares), 1);
    if (blockIdx.x == 0 && tid == 0) a.share[0] = share;
    const int share_lo = min((int64_t)blockIdx.x * share, (int64_t)total);
    const int share_hi = min((int64_t)share_lo + share, (int64_t)total);

    const float qscale = a.softcap > 0.f ? a.scale / a.softcap : a.scale * LOG2E;
    const float capk = a.softcap * LOG2E;
    const int ps = a.kv.page_shift, pmask = (1 << ps) - 1;

    // this wave's DMA instructions: sub-tile, keys or values, source offset per lane
    const int my_sub = w * SG::DX / (2 * SG::KI);
    uint32_t src[SG::DX];
#pragma unroll
    for (int i = 0; i < SG::DX; i++) {
        const int c = (w * SG::DX + i) % (2 * SG::KI), b = (c - SG::KI) * 1024 + l * 16, row = b / (D * ES);
        src[i] = c < SG::KI ? (uint32_t)((((4 * c + g4) << ps) + r16) * 16)
                            : (uint32_t)((4 * (row & 3) + (row >> 2)) * D * ES + b % (D * ES));
    }

    for (int at = share_lo; at < share_hi;) {
        // ---- the piece: steps [st0, st1) of unit (row group, head) of request s
        int s = 0;
        for (int hi = a.S; hi - s > 1;) {
            const int mid = (s + hi) >> 1;
            if (base[mid] <= at) s = mid;
            else hi = mid;
        }
        s = uniform(s);
        Request rq = request_of<RB, TICK, true>(a, s);
        rq.row0 = uniform(rq.row0);
        rq.n = uniform(rq.n);
        rq.first = uniform(rq.first);
        rq.len = uniform(rq.len);
        rq.units = uniform(rq.units);
        rq.steps = uniform(rq.steps);
        rq.grow = uniform(rq.grow);
        const int off = at - uniform(base[s]), groups = (int)((uint32_t)rq.units / (uint32_t)nkv);
        if (off < 0 || off >= steps_before(rq, nkv, groups)) return;     // (offsets that do not ascend, their steps past int32: no row is read)
        int grp = 0;
        for (int hi = groups; hi - grp > 1;) {
            const int mid = (grp + hi) >> 1;
            if (steps_before(rq, nkv, mid) <= off) grp = mid;
            else hi = mid;
        }
        grp = uniform(grp);
        const int cost = rq.steps + rq.grow * grp, in = off - steps_before(rq, nkv, grp);
        const int head = uniform((int)((uint32_t)in / (uint32_t)cost)), st0 = in - head * cost;
        if ((uint32_t)head >= (uint32_t)nkv) return;                     // (the same)
        if (a.whole && st0 > 0) {           // the share before has it
            at += cost - st0;
            continue;
        }
        const int st1 = a.whole ? cost : min(cost, st0 + (share_hi - at));
        const int piece_at = at;
        at += st1 - st0;
        const int row0 = grp * RB, nrows = min(RB, rq.n * G - row0);
        const int i0 = (int)((uint32_t)row0 / (uint32_t)G), r_in = row0 - i0 * G;   // row0 = token i0, its head r_in
        auto token_of = [&](int x) { return i0 + (((r_in + x) * a.G16) >> 16); };    // of the unit's row x
        // positions [see_lo, see_hi) that some row of the unit sees, in stages; the
        // piece takes its part of them
        const int p_lo = rq.first + i0, p_hi = rq.first + token_of(nrows - 1);
        const int see_lo = a.window > 0 ? max(p_lo - a.window + 1, 0) : 0;
        const int see_hi = max(min(p_hi + 1, rq.len), 0);
        const int a0 = see_lo & ~31;
        const int stages = (max(see_hi - a0, 0) + SG::POS - 1) / SG::POS;
        const float stretch = (float)stages / (float)cost;
        auto stage_at = [&](int st) { return st == cost ? stages : min((int)((float)st * stretch), stages); };
        const int k0 = uniform(stage_at(st0)), n = uniform(stage_at(st1)) - k0;
        const int t_lo = a0 + k0 * SG::POS;
        const int t_hi = (int)min((int64_t)t_lo + (int64_t)n * SG::POS, (int64_t)see_hi);

        const table_ptr trow = (table_ptr)(uintptr_t)(a.table + (int64_t)s * a.W);
        auto page_at = [&](int pos) __attribute__((always_inline)) {         // -1: none
            const int v = trow[min(pos >> ps, a.W - 1)];
            return uniform(v >= 0 && v < a.kv.num_pages ? v : -1);
        };
        // stage k's loads; returns which of its sub-tiles have a page (of others page 0
        // is read: what stands there is masked)
        auto issue = [&](int k) __attribute__((always_inline)) {
            const int t0 = t_lo + k * SG::POS;
            unsigned char* st = smem + k % SG::ST * SG::BYTES;
            int ok = 0, page[SG::SUB];
#pragma unroll
            for (int sb = 0; sb < SG::SUB; sb++) {
                page[sb] = page_at(t0 + 16 * sb);
                ok |= (page[sb] >= 0 ? 1 : 0) << sb;
                page[sb] = max(page[sb], 0);
            }
            int mine = page[0];
#pragma unroll
            for (int sb = 1; sb < SG::SUB; sb++) mine = my_sub == sb ? page[sb] : mine;
            const int64_t ph = (int64_t)mine * nkv + head;
            const int po = (t0 + 16 * my_sub) & pmask;
            const char* kb = (const char*)a.kv.k + (((ph * (D / X)) << ps) + po) * 16;
            const char* vb = (const char*)a.kv.v + ((ph << ps) + po) * (D * ES);
#pragma unroll
            for (int i = 0; i < SG::DX; i++) {
                const int id = w * SG::DX + i;
                const char* from = id % (2 * SG::KI) < SG::KI ? kb : vb;
                dma16(from + src[i], st + id * 1024);
            }
            if constexpr (F8) {             // every wave loads all of the stage's scales, to the same place
#pragma unroll
                for (int hf = 0; hf < SG::HALVES; hf++) {
                    const int sb = 2 * hf + (l >> 5);
                    const int64_t at2 = (((int64_t)(l >> 5 ? page[2 * hf + 1] : page[2 * hf]) * nkv + head) << ps) +
                                        ((t0 + 16 * sb) & pmask) + r16;
                    dma4((l & 16 ? a.kv.v_scale : a.kv.k_scale) + at2, st + SG::SCALES + hf * 256);
                }
            }
            return ok;
        };

        // ---- this wave's rows: q fragments, and the positions that each sees
        const int x0 = w * PMT * 16, rows_w = min(max(nrows - x0, 0), PMT * 16);
        const int wp_lo = rq.first + token_of(x0), wp_hi = rows_w > 0 ? rq.first + token_of(x0 + rows_w - 1) : -1;
        const int w_lo = a.window > 0 ? max(wp_lo - a.window + 1, 0) : 0, w_hi = min(wp_hi, rq.len - 1);    // some row sees
        const int full_lo = a.window > 0 ? max(wp_hi - a.window + 1, 0) : 0;
        const int full_hi = min(min(wp_lo + 1, rq.len), t_hi);                                              // every row sees
        lds_barrier();                      // the last piece's stages are read
        int ok[SG::ST - 1] = {};
#pragma unroll
        for (int k = 0; k < SG::ST - 1; k++)
            if (k < n) ok[k] = issue(k);
        bf16x8_t qf[PMT][D / 32];
        int vlo[PMT];
        uint32_t vn[PMT];                   // this lane's rows see [vlo, vlo + vn)
#pragma unroll
        for (int mt = 0; mt < PMT; mt++) {
            const int x = x0 + mt * 16 + r16, xs = r_in + min(x, nrows - 1), i = (xs * a.G16) >> 16;   // (rows past the unit's repeat its last, unused)
            const uint16_t* q = a.q + (int64_t)(rq.row0 + i0 + i) * a.q_stride + (int64_t)(head * G + xs - i * G) * D;
#pragma unroll
            for (int k = 0; k < D / 32; k++)
                qf[mt][k] = *reinterpret_cast<const bf16x8_t*>(q + (F8 ? 16 * (4 * (k >> 1) + g4) + 8 * (k & 1) : 32 * k + 8 * g4));
            const int p = rq.first + i0 + i;
            vlo[mt] = a.window > 0 ? max(p - a.window + 1, 0) : 0;
            vn[mt] = x < nrows ? (uint32_t)max(min(p + 1, t_hi) - vlo[mt], 0) : 0u;
        }
        f32x4_t acc[PMT][NH][E], sum[PMT];
        float m[PMT];
#pragma unroll
        for (int mt = 0; mt < PMT; mt++) {
            m[mt] = -__builtin_inff();
            sum[mt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < NH; h++)
#pragma unroll
                for (int e = 0; e < E; e++) acc[mt][h][e] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
        uint32_t strange = 0;               // not 0: infinite or NaN values in a tile seen in part

        // 32 positions from t0, their sub-tiles at `st`; ok2: which of the two have a page
        auto half = [&](const unsigned char* st, const unsigned char* sc_at, int t0, int ok2) __attribute__((always_inline)) {
            const bool whole = ok2 == 3 && t0 >= full_lo && t0 + 32 <= full_hi;
            f32x4_t sc[PMT][2];
#pragma unroll
            for (int mt = 0; mt < PMT; mt++)
#pragma unroll
                for (int sb = 0; sb < 2; sb++) sc[mt][sb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < D / 32; k++) {
#pragma unroll
                for (int sb = 0; sb < 2; sb++) {
                    bf16x8_t kf;
                    if constexpr (F8) {
                        const u32x2_a x = *reinterpret_cast<const u32x2_a*>(st + sb * 2 * KB + (k >> 1) * 1024 + l * 16 + (k & 1) * 8);
                        kf = __builtin_bit_cast(bf16x8_t, u32x4_a{fp8x2_bf16<false>(x[0]), fp8x2_bf16<true>(x[0]),
                                                                  fp8x2_bf16<false>(x[1]), fp8x2_bf16<true>(x[1])});
                    } else {
                        kf = *reinterpret_cast<const bf16x8_t*>(st + sb * 2 * KB + k * 1024 + l * 16);
                    }
#pragma unroll
                    for (int mt = 0; mt < PMT; mt++) sc[mt][sb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[mt][k], sc[mt][sb], 0, 0, 0);
                }
            }
            f32x4_t vs[2];
#pragma unroll
            for (int sb = 0; sb < 2; sb++) {
                f32x4_t f = {qscale, qscale, qscale, qscale};
                if constexpr (F8) {
                    f *= *reinterpret_cast<const f32x4_t*>(sc_at + sb * 128 + g4 * 16);
                    vs[sb] = *reinterpret_cast<const f32x4_t*>(sc_at + sb * 128 + 64 + g4 * 16);
                }
#pragma unroll
                for (int mt = 0; mt < PMT; mt++) {
                    sc[mt][sb] *= f;
                    // c tanh(z) = c (1 - 2 / (e^{2z} + 1)), absolutely accurate to ~2^-23 c
                    if (a.softcap > 0.f)
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            sc[mt][sb][i] = capk * (1.f - 2.f * __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(sc[mt][sb][i] * (2.f * LOG2E)) + 1.f));
                }
            }
            if (!whole) {
#pragma unroll
                for (int mt = 0; mt < PMT; mt++)
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const uint32_t at2 = (uint32_t)(t0 + 16 * (j >> 2) + 4 * g4 + (j & 3) - vlo[mt]);
                        if (at2 >= ((ok2 >> (j >> 2)) & 1 ? vn[mt] : 0u)) sc[mt][j >> 2][j & 3] = -__builtin_inff();
                    }
            }
            // ---- softmax: the exponentials' base follows a row's maximum only when
            // some row's has risen by more than 2^8
            float top[PMT];
            bool rise = false;
#pragma unroll
            for (int mt = 0; mt < PMT; mt++) {
                float t = -__builtin_inff();
#pragma unroll
                for (int sb = 0; sb < 2; sb++)
                    t = fmaxf(t, fmaxf(fmaxf(sc[mt][sb][0], sc[mt][sb][1]), fmaxf(sc[mt][sb][2], sc[mt][sb][3])));
                t = fmaxf(t, tr_partner<16>(t));
                top[mt] = fmaxf(t, tr_partner<32>(t));
                rise |= top[mt] > m[mt] + 8.f;
            }
            if (__any(rise)) {
#pragma unroll
                for (int mt = 0; mt < PMT; mt++) {
                    const float mn = fmaxf(m[mt], top[mt]);
                    const float f = __builtin_amdgcn_exp2f(m[mt] - (mn == -__builtin_inff() ? 0.f : mn));
                    sum[mt] *= f;
#pragma unroll
                    for (int h = 0; h < NH; h++)
#pragma unroll
                        for (int e = 0; e < E; e++) acc[mt][h][e] *= f;
                    m[mt] = mn;
                }
            }
            uint32_t p[PMT][4];             // pairs of positions' probabilities, bf16
#pragma unroll
            for (int mt = 0; mt < PMT; mt++) {
                const float b = m[mt] == -__builtin_inff() ? 0.f : m[mt];       // a row that has seen nothing yet
#pragma unroll
                for (int sb = 0; sb < 2; sb++) {
                    f32x4_t e, v;
#pragma unroll
                    for (int i = 0; i < 4; i++) e[i] = __builtin_amdgcn_exp2f(sc[mt][sb][i] - b);
                    v = e;
                    // e4m3 values: the weight is p v_scale, rounded; the sum takes it over v_scale
                    if constexpr (F8)
#pragma unroll
                        for (int i = 0; i < 4; i++) v[i] = e[i] == 0.f ? 0.f : e[i] * vs[sb][i];
                    p[mt][2 * sb] = pk_bf16(v[0], v[1]);
                    p[mt][2 * sb + 1] = pk_bf16(v[2], v[3]);
                    if constexpr (F8) {
                        const f32x4_t u = {bf16lo_to_f32(p[mt][2 * sb]), bf16hi_to_f32(p[mt][2 * sb]),
                                           bf16lo_to_f32(p[mt][2 * sb + 1]), bf16hi_to_f32(p[mt][2 * sb + 1])};
#pragma unroll
                        for (int i = 0; i < 4; i++) sum[mt][i] += u[i] == 0.f ? e[i] : u[i] * __builtin_amdgcn_rcpf(vs[sb][i]);
                    }
                }
            }
            auto weights = [&](int mt) { return __builtin_bit_cast(bf16x8_t, u32x4_a{p[mt][0], p[mt][1], p[mt][2], p[mt][3]}); };
            if constexpr (!F8) {            // the sum of the rounded weights: a row of ones
                const u32x4_a one = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
                for (int mt = 0; mt < PMT; mt++)
                    sum[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, one), weights(mt), sum[mt], 0, 0, 0);
            }
            // ---- O^T += V^T P^T
#pragma unroll
            for (int h = 0; h < NH; h++) {
                uint32_t v[8][EW];
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const unsigned char* from = st + (j >> 2) * 2 * KB + KB + ((4 * (j & 3) + g4) * D + h * 16 * E + r16 * E) * ES;
                    if constexpr (EW == 4) {
                        const u32x4_a x = *reinterpret_cast<const u32x4_a*>(from);
#pragma unroll
                        for (int q = 0; q < 4; q++) v[j][q % EW] = x[q];
                    } else if constexpr (EW == 2) {
                        const u32x2_a x = *reinterpret_cast<const u32x2_a*>(from);
                        v[j][0] = x[0];
                        v[j][1 % EW] = x[1];
                    } else {
                        v[j][0] = *reinterpret_cast<const uint32_t*>(from);
                    }
                }
                // values that no row of the wave sees become 0, and so do infinite and NaN
                // ones for now (0 * inf is NaN: they must not meet the zero probability
                // of a row that does not see them); add_strange() adds those
                if (!whole) {
                    const uint32_t span = (uint32_t)max(min(w_hi + 1, t_hi) - w_lo, 0);
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const uint32_t at2 = (uint32_t)(t0 + 16 * (j >> 2) + 4 * g4 + (j & 3) - w_lo);
                        const uint32_t in = at2 < ((ok2 >> (j >> 2)) & 1 ? span : 0u) ? 0xFFFFFFFFu : 0u;
#pragma unroll
                        for (int q = 0; q < EW; q++) {
                            const uint32_t y = v[j][q] & in;
                            // the top bit of each element whose exponent is all ones (e4m3: that is 0x7F), then all its bits
                            const uint32_t b = F8 ? ((y & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u : ((y & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
                            strange |= b;
                            v[j][q] = y & ~((b - (b >> (F8 ? 7 : 15))) | b);
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < EW; q++) {
                    u32x4_a f[PER];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const uint32_t x = v[2 * j][q], y = v[2 * j + 1][q];
                        if constexpr (F8) {
                            const uint32_t lo = __builtin_amdgcn_perm(y, x, 0x05010400);   // x0 y0 x1 y1
                            const uint32_t hh = __builtin_amdgcn_perm(y, x, 0x07030602);   // x2 y2 x3 y3
                            f[0][j] = fp8x2_bf16<false>(lo);
                            f[1][j] = fp8x2_bf16<true>(lo);
                            f[PER - 2][j] = fp8x2_bf16<false>(hh);
                            f[PER - 1][j] = fp8x2_bf16<true>(hh);
                        } else {
                            f[0][j] = __builtin_amdgcn_perm(y, x, 0x05040100);
                            f[1][j] = __builtin_amdgcn_perm(y, x, 0x07060302);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < PER; e++)
#pragma unroll
                        for (int mt = 0; mt < PMT; mt++)
                            acc[mt][h][PER * q + e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(bf16x8_t, f[e]), weights(mt), acc[mt][h][PER * q + e], 0, 0, 0);
                }
            }
        };

        // ---- the stages: stage k has landed everywhere once each wave has waited for
        // its own loads and met the barrier; stage k - 1 is read by then and takes the
        // loads of stage k + 2
        for (int k = 0; k < n; k++) {
            if (k + 1 < n) wait_loads<SG::DMA>();
            else wait_loads<0>();
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            const int ok_k = ok[0];
            ok[0] = ok[1];
            if (k + 2 < n) ok[1] = issue(k + 2);
            const unsigned char* st = smem + k % SG::ST * SG::BYTES;
#pragma unroll 1
            for (int hf = 0; hf < SG::HALVES; hf++) {
                const int t0 = t_lo + k * SG::POS + 32 * hf;
                if (t0 > w_hi || t0 + 32 <= w_lo) continue;          // no row of the wave sees it
                half(st + hf * 4 * KB, st + SG::SCALES + hf * 256, t0, (ok_k >> (2 * hf)) & 3);
            }
        }

        // the infinite and NaN values left out above, of elements d + {0, 1, 2, 3} E and
        // the positions that a row at position p sees (every probability is > 0)
        auto add_strange = [&](f32x4_t& o, int p, int d) {
            for (int pos = max(t_lo, a.window > 0 ? p - a.window + 1 : 0); pos < min(t_hi, p + 1); pos++) {
                const int t0 = pos & ~31, e = trow[min(pos >> ps, a.W - 1)];
                if (e < 0 || e >= a.kv.num_pages) continue;
                if (t0 >= full_lo && t0 + 32 <= full_hi) {           // in the products, unless the tile lacks a page
                    const int e0 = trow[min(t0 >> ps, a.W - 1)], e1 = trow[min((t0 + 16) >> ps, a.W - 1)];
                    if (e0 >= 0 && e0 < a.kv.num_pages && e1 >= 0 && e1 < a.kv.num_pages) continue;
                }
                const int64_t at2 = ((((int64_t)e * nkv + head) << ps) + (pos & pmask)) * D + d;
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    if constexpr (F8) {
                        if ((((const uint8_t*)a.kv.v)[at2 + c * E] & 0x7F) == 0x7F) o[c] = __builtin_nanf("");
                    } else {
                        const uint16_t v = ((const uint16_t*)a.kv.v)[at2 + c * E];
                        if ((v & 0x7F80) == 0x7F80) o[c] += bf16_to_f32(v);
                    }
                }
            }
        };

        // ---- a unit that lies in this share alone is done; of others the piece that
        // begins with the share is partial 2 b, one that begins inside it 2 b + 1
        const bool direct = st1 - st0 == cost;
        const int64_t pidx = 2 * (int64_t)blockIdx.x + (piece_at == share_lo ? 0 : 1);
        const bool any_strange = __any(strange != 0);
#pragma unroll
        for (int mt = 0; mt < PMT; mt++) {
            const int x = x0 + mt * 16 + r16;
            float L = sum[mt][0];
            if constexpr (F8) {             // this lane's positions
                L = (sum[mt][0] + sum[mt][1]) + (sum[mt][2] + sum[mt][3]);
                L += tr_partner<16>(L);
                L += tr_partner<32>(L);
            }
            if (x >= nrows) continue;
            const int i = ((r_in + x) * a.G16) >> 16;
            if (any_strange) {
#pragma unroll
                for (int h = 0; h < NH; h++)
#pragma unroll
                    for (int e = 0; e < E; e++) add_strange(acc[mt][h][e], rq.first + i0 + i, 16 * E * h + 4 * E * g4 + e);
            }
            // O^T rows 4 g4 + i of MFMA (h, e) are d = 16 E h + E (4 g4 + i) + e
            if (direct) {
                const float inv = L == 0.f ? 0.f : __builtin_amdgcn_rcpf(L);     // (a row that sees nothing: 0)
                uint16_t* dst = a.out + ((int64_t)(rq.row0 + i0 + i) * a.n_heads + head * G + r_in + x - i * G) * D + 4 * E * g4;
#pragma unroll
                for (int h = 0; h < NH; h++)
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        uint32_t o[E / 2];
#pragma unroll
                        for (int e = 0; e < E; e += 2) o[e / 2] = pk_bf16(acc[mt][h][e][c] * inv, acc[mt][h][e + 1][c] * inv);
                        if constexpr (E == 8)
                            *reinterpret_cast<u32x4_a*>(dst + 16 * E * h + E * c) = u32x4_a{o[0], o[1], o[E / 2 - 2], o[E / 2 - 1]};
                        else
                            *reinterpret_cast<u32x2_a*>(dst + 16 * E * h + E * c) = u32x2_a{o[0], o[1]};
                    }
            } else {                        // in the order (h, e, 4 g4 + i)
                float* pd = a.part + (pidx * RB + x) * D + 4 * g4;
#pragma unroll
                for (int h = 0; h < NH; h++)
#pragma unroll
                    for (int e = 0; e < E; e++) *reinterpret_cast<f32x4_t*>(pd + (h * E + e) * 16) = acc[mt][h][e];
                if (g4 == 0) a.ml[pidx * RB + x] = make_float2(m[mt], L);
            }
        }
    }
}

template <int D, int F8>
hipError_t launch_prompt(AttnArgs a, hipStream_t st) {
    using SG = Stage<D, F8>;
    auto kern = k_prompt_attn<D, F8>;
    const size_t lds = (size_t)SG::BYTES * SG::ST + ((size_t)a.S * 4 + 15) / 16 * 16;
    static LdsLimit lim;
    hipError_t e = lim.ensure((const void*)kern, 156 * 1024);
    if (e != hipSuccess) return e;
    a.shares = PROMPT_SHARES;
    hipLaunchKernelGGL(kern, dim3(a.shares), dim3(PROMPT_THREADS), lds, st, a);
    if (a.whole) return hipGetLastError();
    if ((int64_t)a.T * a.n_heads <= 32 * PROMPT_ROWS)
        hipLaunchKernelGGL((k_attn_join<D, PROMPT_ROWS, TICK, true, D, 4>), dim3(a.T, a.n_heads), dim3(4 * WAVE), 0, st, a);
    else
        hipLaunchKernelGGL((k_attn_join<D, PROMPT_ROWS, TICK, true, D, 1>), dim3((a.T + join_rows(true, 1) - 1) / join_rows(true, 1), (a.n_heads + 3) / 4), dim3(AT_THREADS), 0, st, a);
    return hipGetLastError();
}

}  // namespace

PromptShape prompt_attn_shape() { return {PROMPT_ROWS, PROMPT_SHARES}; }

hipError_t launch_prompt_attn(const AttnArgs& a, hipStream_t st) {
    const bool f8 = a.kv.k_scale != nullptr;
    switch (a.kv.head_dim) {
        case 64: return f8 ? launch_prompt<64, 1>(a, st) : launch_prompt<64, 0>(a, st);
        case 128: return f8 ? launch_prompt<128, 1>(a, st) : launch_prompt<128, 0>(a, st);
        case 256: return f8 ? launch_prompt<256, 1>(a, st) : launch_prompt<256, 0>(a, st);
    }
    return hipErrorInvalidValue;
}
