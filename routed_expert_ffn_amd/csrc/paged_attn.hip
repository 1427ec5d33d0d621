// paged_attn.hip -- attention of a request's new rows over its paged cache,
// split over the cache's length and joined (gfx950).
//
// Row i (query token) of request s at position p = kv_len - n + i, head h:
//   s_j = scale q.k_j (capped: c tanh(s_j / c)),  out = sum_j e^{s_j - m} v_j / sum_j e^{s_j - m},  j <= p (and j > p - window)
//
// The G query heads of a key-value head and the request's new rows together
// are the "rows" r = i G + g of one product, so the cache is read once for all
// of them: 16 MT rows per item.  A wave takes 32 positions at a time:
//   S^T[position][row] = K Q^T      MFMA 16x16x32 bf16, two sub-tiles of 16 positions
//   O^T[d][row]       += V^T P^T    MFMA 16x16x32 bf16, k = the 32 positions
// In S^T a lane holds row l & 15 and positions 4 (l >> 4) + i of each sub-tile;
// with the k index of the second product running over the positions in that
// same order, P goes from the first product's result into the second's operand
// without leaving the lane.  Both operands come straight from memory into
// registers, with no LDS in between: the key pages are laid out in 16-byte
// chunks side by side, so 16 lanes read 16 positions' chunk contiguously, and of
// a value row lane l & 15 takes 8 consecutive elements (E below), the 16 lanes
// a whole row; MFMA m of the second product then takes element E r + m as its
// row r, and one byte permute per register pairs up two positions' elements.
// One pass with a running maximum and sum per row, both in registers; the
// waves of a block take the tiles in turn and are joined through LDS, the
// splits of a request by k_attn_join.
//
// Bound by HBM at few rows (each cached byte is used for 16 rows at a time):
// see launch_paged_attn for how the work is split.
#include "attn.h"
#include "common.h"
#include "device.h"
#include "stream.h"

namespace {

constexpr int NW = 4;                       // waves per block
constexpr int AT_THREADS = NW * WAVE;
constexpr int TILE = 32;                    // positions per wave step
constexpr float LOG2E = 1.44269504088896341f;

typedef uint32_t u32x2_a __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_a __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_a __attribute__((ext_vector_type(2)));

MOE_DEV uint32_t pk_bf16(float lo, float hi) {
    const bf16x2_a v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}
// two e4m3 of word w (its low or high half) -> packed bf16 (exact)
template <bool HI>
MOE_DEV uint32_t fp8x2_bf16(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}

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
    int target;                             // items the splitting aims at (grid blocks)
    int4* meta;                             // [S] (first partial, splits, 0, 0)
    float* part;                            // [partial][rows][D] unnormalised sums
    float2* ml;                             // [partial][rows] (maximum, sum)
};

// What a block needs of a request: its row range, positions and split.
struct Request {
    int row0, n, first;                     // first batch row, rows, position of its first row
    int len;                                // positions that the table can hold
    int range;                              // positions that any of its rows may see
    int groups;                             // items per key-value head and split
};
MOE_DEV Request request_of(const AttnArgs& a, int s, int rows_per_item) {
    Request r;
    const int b = min(max(a.q_offsets[s], 0), a.T), e = min(max(a.q_offsets[s + 1], 0), a.T);
    const int L = max(a.kv_len[s], 0);
    r.row0 = b;
    r.n = max(e - b, 0);
    r.first = L - r.n;
    r.len = (int)min((int64_t)L, (int64_t)a.W << a.kv.page_shift);
    const int lo = a.window > 0 ? max(r.first - a.window + 1, 0) : 0;
    r.range = max(r.len - lo, 0);
    const int G = a.n_heads / a.kv.n_kv_heads;
    r.groups = (int)(((int64_t)r.n * G + rows_per_item - 1) / rows_per_item);
    return r;
}

template <int D, int F8>
struct Tile {                               // one wave's 32 positions
    static constexpr int KV = F8 ? D / 64 : D / 32;       // 16-byte key chunks per lane and sub-tile
    static constexpr int E = D == 64 ? 4 : 8;             // value elements per lane and load
    static constexpr int NH = D / (16 * E);               // loads per position
    static constexpr int EW = F8 ? E / 4 : E / 2;         // their 32-bit words
    u32x4_a k[2][KV];
    uint32_t v[8][NH][EW];
    f32x4_t ks[2], vs[2];
};

template <int D, int F8, int MT>
__global__ __launch_bounds__(AT_THREADS) void k_paged_attn(const AttnArgs a) {
    using TL = Tile<D, F8>;
    constexpr int E = TL::E, NH = TL::NH, EW = TL::EW, KV = TL::KV;
    constexpr int RB = 16 * MT;             // rows per item
    constexpr bool QREG = D * MT <= 256;    // q fragments in registers (up to 32 of them), else from LDS at each use
    constexpr int DP = D + 4;               // padded row of the join area
    constexpr int QP = D + 8;               // padded q row, bf16
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    // [S + 1] first item of each request, [S] first partial; then the q rows /
    // join area; the scan's scratch
    int* istart = (int*)smem;
    int* pstart = istart + a.S + 1;
    unsigned char* area = smem + ((size_t)(2 * a.S + 1) * 4 + 15) / 16 * 16;
    uint16_t* qs = (uint16_t*)area;                              // [RB][QP]
    float* ja = (float*)area;                                    // [NW][16][DP]
    float2* jml = (float2*)(area + sizeof(float) * NW * 16 * DP);  // [NW][16]
    __shared__ int64_t sc64[NW];
    __shared__ int sc32[2][NW];
    __shared__ int strange;                 // the item met infinite or NaN values in a tile seen in part

    const int tid = threadIdx.x, l = lane_id(), w = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int G = a.n_heads / a.kv.n_kv_heads, nkv = a.kv.n_kv_heads;

    // ---- the split, from the lengths: U = positions to go over, summed over
    // row groups and heads; C positions per item so that about `target` items
    // result, a multiple of the block's 128 positions
    int64_t U = 0;
    int RG = 0;
    for (int s = tid; s < a.S; s += AT_THREADS) {
        const Request r = request_of(a, s, RB);
        U += (int64_t)r.groups * nkv * r.range;
        RG += r.groups * nkv;
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        U += __shfl_xor(U, d, WAVE);
        RG += __shfl_xor(RG, d, WAVE);
    }
    if (l == 0) { sc64[w] = U; sc32[0][w] = RG; }
    __syncthreads();
    U = 0; RG = 0;
#pragma unroll
    for (int i = 0; i < NW; i++) { U += sc64[i]; RG += sc32[0][i]; }
    const int64_t room = RG < a.target / 2 ? a.target - RG : a.target;
    const int64_t C0 = (U + room - 1) / room;
    const int64_t C = max((C0 + TILE * NW - 1) / (TILE * NW), (int64_t)1) * (TILE * NW);
    // first item and first partial of every request: running sums over the
    // requests, 256 at a time
    int ibase = 0, pbase = 0;
    for (int s0 = 0; s0 < a.S; s0 += AT_THREADS) {
        const int s = s0 + tid;
        int it = 0, pt = 0, nsplit = 0;
        if (s < a.S) {
            const Request r = request_of(a, s, RB);
            nsplit = max((int)(((int64_t)r.range + C - 1) / C), 1);
            it = r.groups * nkv * nsplit;
            pt = nsplit > 1 ? it : 0;
        }
        const int ii = wave_incl_scan(it), pi = wave_incl_scan(pt);
        __syncthreads();                    // the scratch's last readers are done
        if (l == WAVE - 1) { sc32[0][w] = ii; sc32[1][w] = pi; }
        __syncthreads();
        int ib = ibase, pb = pbase;
#pragma unroll
        for (int i = 0; i < NW; i++) {
            if (i < w) { ib += sc32[0][i]; pb += sc32[1][i]; }
            ibase += sc32[0][i];
            pbase += sc32[1][i];
        }
        if (s < a.S) {
            istart[s] = ib + ii - it;
            pstart[s] = pb + pi - pt;
            if (blockIdx.x == 0) a.meta[s] = make_int4(pb + pi - pt, nsplit, 0, 0);
        }
    }
    if (tid == 0) istart[a.S] = ibase;
    __syncthreads();
    const int items = istart[a.S];

    const int r16 = l & 15, g4 = l >> 4;
    const float qscale = a.softcap > 0.f ? a.scale / a.softcap : a.scale * LOG2E;
    const float capk = a.softcap * LOG2E;
    const int ps = a.kv.page_shift, pmask = (1 << ps) - 1;

    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        int s = 0, hi = a.S;
        while (hi - s > 1) {
            const int mid = (s + hi) >> 1;
            if (istart[mid] <= item) s = mid;
            else hi = mid;
        }
        const Request rq = request_of(a, s, RB);
        const int nsplit = max((int)(((int64_t)rq.range + C - 1) / C), 1);
        // item = (row group, kv head, split), split fastest
        int x = item - istart[s];
        const int split = x % nsplit;
        x /= nsplit;
        const int head = x % nkv, grp = x / nkv;
        const int row0 = grp * RB, nrows = min(RB, rq.n * G - row0);
        const int i0 = row0 / G, i1 = (row0 + nrows - 1) / G;
        // positions [lo, hi) that some row of the item sees, and this split's part
        const int p_lo = rq.first + i0, p_hi = rq.first + i1;       // positions of its first and last row
        const int see_lo = a.window > 0 ? max(p_lo - a.window + 1, 0) : 0;
        const int see_hi = min(p_hi + 1, rq.len);
        const int a0 = see_lo & ~(TILE - 1);
        const int total = max(see_hi - a0, 0);
        const int per = (int)(((int64_t)total + (int64_t)nsplit * TILE * NW - 1) / ((int64_t)nsplit * TILE * NW)) * (TILE * NW);
        const int t_lo = (int)min((int64_t)a0 + (int64_t)split * per, (int64_t)see_hi);
        const int t_hi = (int)min((int64_t)t_lo + per, (int64_t)see_hi);
        // every row sees [full_lo, full_hi) whole
        const int full_lo = a.window > 0 ? max(p_hi - a.window + 1, 0) : 0;
        const int full_hi = min(p_lo + 1, rq.len);

        // ---- the item's q rows: row r = query token i0.., head of the group
        __syncthreads();                    // the last item's join area is read
        if (tid == 0) strange = 0;
        for (int c = tid; c < RB * (D / 8); c += AT_THREADS) {
            const int rr = c / (D / 8), cc = c - rr * (D / 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (rr < nrows) {
                const int row = row0 + rr, i = row / G, g = row - i * G;
                v = *reinterpret_cast<const uint4*>(a.q + (int64_t)(rq.row0 + i) * a.q_stride +
                                                    (int64_t)(head * G + g) * D + cc * 8);
            }
            *reinterpret_cast<uint4*>(qs + rr * QP + cc * 8) = v;
        }
        __syncthreads();
        // q fragments: bf16 keys: step k, lane group g4 holds chunk 4 k + g4; e4m3:
        // chunk 4 (k / 2) + g4 of 16 elements, half k & 1
        auto q_frag = [&](int mt, int k) __attribute__((always_inline)) {
            const int d = F8 ? 16 * (4 * (k >> 1) + g4) + 8 * (k & 1) : 32 * k + 8 * g4;
            return *reinterpret_cast<const bf16x8_t*>(qs + (mt * 16 + r16) * QP + d);
        };
        bf16x8_t qf[QREG ? MT : 1][QREG ? D / 32 : 1];
        if constexpr (QREG) {
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int k = 0; k < D / 32; k++) qf[mt][k] = q_frag(mt, k);
        }
        // this lane's row in each row tile: the positions it sees, [vlo, vhi]
        int vlo[MT], vhi[MT];
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            const int row = row0 + mt * 16 + r16, i = row / G;
            const bool real = mt * 16 + r16 < nrows;
            const int p = rq.first + i;
            vhi[mt] = real ? min(p, rq.len - 1) : -1;
            vlo[mt] = a.window > 0 ? max(p - a.window + 1, 0) : 0;
        }

        f32x4_t acc[MT][NH][E];
        float m[MT], sum[MT];
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            m[mt] = -__builtin_inff();
            sum[mt] = 0.f;
#pragma unroll
            for (int h = 0; h < NH; h++)
#pragma unroll
                for (int e = 0; e < E; e++) acc[mt][h][e] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }

        const int32_t* trow = a.table + (int64_t)s * a.W;
        auto load = [&](TL& t, int t0, int (&page)[2]) __attribute__((always_inline)) {
#pragma unroll
            for (int sb = 0; sb < 2; sb++) {
                const int pos = t0 + 16 * sb;
                // sub-tiles past the table repeat its last page and are masked
                const int e = trow[min(pos >> ps, a.W - 1)];
                page[sb] = (e >= 0 && e < a.kv.num_pages) ? e : -1;
                const int64_t ph = (int64_t)max(page[sb], 0) * nkv + head;
                const int off = pos & pmask;
                if constexpr (F8) {
                    const uint8_t* kb = (const uint8_t*)a.kv.k + ((ph * (D / 16)) << (ps + 4)) + off * 16;
#pragma unroll
                    for (int c = 0; c < KV; c++)
                        t.k[sb][c] = *reinterpret_cast<const u32x4_a*>(kb + (((4 * c + g4) << ps) + r16) * 16);
                    const uint8_t* vb = (const uint8_t*)a.kv.v + ((ph << ps) + off) * D;
#pragma unroll
                    for (int j = 0; j < 4; j++)
#pragma unroll
                        for (int h = 0; h < NH; h++) {
                            const uint8_t* src = vb + (4 * g4 + j) * D + h * 16 * E + r16 * E;
                            if constexpr (EW == 2) {
                                const u32x2_a q = *reinterpret_cast<const u32x2_a*>(src);
                                t.v[4 * sb + j][h][0] = q[0];
                                t.v[4 * sb + j][h][EW - 1] = q[1];
                            } else {
                                t.v[4 * sb + j][h][0] = *reinterpret_cast<const uint32_t*>(src);
                            }
                        }
                    t.ks[sb] = *reinterpret_cast<const f32x4_t*>(a.kv.k_scale + (ph << ps) + off + 4 * g4);
                    t.vs[sb] = *reinterpret_cast<const f32x4_t*>(a.kv.v_scale + (ph << ps) + off + 4 * g4);
                } else {
                    const uint16_t* kb = (const uint16_t*)a.kv.k + ((ph * (D / 8)) << (ps + 3)) + off * 8;
#pragma unroll
                    for (int c = 0; c < KV; c++)
                        t.k[sb][c] = *reinterpret_cast<const u32x4_a*>(kb + (((4 * c + g4) << ps) + r16) * 8);
                    const uint16_t* vb = (const uint16_t*)a.kv.v + ((ph << ps) + off) * D;
#pragma unroll
                    for (int j = 0; j < 4; j++)
#pragma unroll
                        for (int h = 0; h < NH; h++) {
                            const uint16_t* src = vb + (4 * g4 + j) * D + h * 16 * E + r16 * E;
                            if constexpr (EW == 4) {
                                const u32x4_a q = *reinterpret_cast<const u32x4_a*>(src);
#pragma unroll
                                for (int i = 0; i < EW; i++) t.v[4 * sb + j][h][i] = q[i % 4];
                            } else {
                                const u32x2_a q = *reinterpret_cast<const u32x2_a*>(src);
#pragma unroll
                                for (int i = 0; i < EW; i++) t.v[4 * sb + j][h][i] = q[i % 2];
                            }
                        }
                }
            }
        };
        // S^T of one row tile: [sub-tile][i], in units of log2 (uncapped) or of the cap
        auto scores = [&](const TL& t, int mt, f32x4_t (&sc)[2]) __attribute__((always_inline)) {
#pragma unroll
            for (int sb = 0; sb < 2; sb++) {
                f32x4_t c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < D / 32; k++) {
                    bf16x8_t kf;
                    if constexpr (F8) {
                        const uint32_t w0 = t.k[sb][k >> 1][2 * (k & 1)], w1 = t.k[sb][k >> 1][2 * (k & 1) + 1];
                        const u32x4_a q = {fp8x2_bf16<false>(w0), fp8x2_bf16<true>(w0), fp8x2_bf16<false>(w1),
                                           fp8x2_bf16<true>(w1)};
                        kf = __builtin_bit_cast(bf16x8_t, q);
                    } else {
                        kf = __builtin_bit_cast(bf16x8_t, t.k[sb][k]);
                    }
                    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, QREG ? qf[QREG ? mt : 0][QREG ? k : 0] : q_frag(mt, k), c, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    float v = c[i];
                    if constexpr (F8) v *= t.ks[sb][i];
                    v *= qscale;
                    // c tanh(z) = c (1 - 2 / (e^{2z} + 1)), absolutely accurate to ~2^-23 c
                    if (a.softcap > 0.f) v = capk * (1.f - 2.f * __builtin_amdgcn_rcpf(exp2f(v * (2.f * LOG2E)) + 1.f));
                    sc[sb][i] = v;
                }
            }
        };
        // O^T += V^T P^T, the P fragments given
        auto values = [&](const TL& t, const u32x4_a (&p)[MT]) __attribute__((always_inline)) {
#pragma unroll
            for (int h = 0; h < NH; h++) {
                if constexpr (F8) {
#pragma unroll
                    for (int q = 0; q < EW; q++) {          // 4 elements of each position per word
                        u32x4_a f[4];
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const uint32_t x = t.v[2 * j][h][q], y = t.v[2 * j + 1][h][q];
                            const uint32_t lo = __builtin_amdgcn_perm(y, x, 0x05010400);   // x0 y0 x1 y1
                            const uint32_t hh = __builtin_amdgcn_perm(y, x, 0x07030602);   // x2 y2 x3 y3
                            f[0][j] = fp8x2_bf16<false>(lo);
                            f[1][j] = fp8x2_bf16<true>(lo);
                            f[2][j] = fp8x2_bf16<false>(hh);
                            f[3][j] = fp8x2_bf16<true>(hh);
                        }
#pragma unroll
                        for (int e = 0; e < 4; e++)
#pragma unroll
                            for (int mt = 0; mt < MT; mt++)
                                acc[mt][h][4 * q + e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    __builtin_bit_cast(bf16x8_t, f[e]), __builtin_bit_cast(bf16x8_t, p[mt]),
                                    acc[mt][h][4 * q + e], 0, 0, 0);
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < EW; q++) {          // 2 elements of each position per word
                        u32x4_a f[2];
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const uint32_t x = t.v[2 * j][h][q], y = t.v[2 * j + 1][h][q];
                            f[0][j] = __builtin_amdgcn_perm(y, x, 0x05040100);
                            f[1][j] = __builtin_amdgcn_perm(y, x, 0x07060302);
                        }
#pragma unroll
                        for (int e = 0; e < 2; e++)
#pragma unroll
                            for (int mt = 0; mt < MT; mt++)
                                acc[mt][h][2 * q + e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    __builtin_bit_cast(bf16x8_t, f[e]), __builtin_bit_cast(bf16x8_t, p[mt]),
                                    acc[mt][h][2 * q + e], 0, 0, 0);
                    }
                }
            }
        };
        // running maximum and sum of one row tile; sc -> probabilities
        auto soften = [&](f32x4_t (&sc)[2], int mt) __attribute__((always_inline)) {
            float top = fmaxf(fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[0][2], sc[0][3])),
                              fmaxf(fmaxf(sc[1][0], sc[1][1]), fmaxf(sc[1][2], sc[1][3])));
            top = fmaxf(top, tr_partner<16>(top));
            top = fmaxf(top, tr_partner<32>(top));
            const float mn = fmaxf(m[mt], top);
            const float base = mn == -__builtin_inff() ? 0.f : mn;       // a row that has seen nothing yet
            if (__any(mn > m[mt])) {
                const float f = exp2f(m[mt] - base);
                sum[mt] *= f;
#pragma unroll
                for (int h = 0; h < NH; h++)
#pragma unroll
                    for (int e = 0; e < E; e++) acc[mt][h][e] *= f;
                m[mt] = mn;
            }
#pragma unroll
            for (int sb = 0; sb < 2; sb++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    sc[sb][i] = exp2f(sc[sb][i] - base);
                    sum[mt] += sc[sb][i];
                }
        };
        auto pack_p = [&](const TL& t, const f32x4_t (&sc)[2]) __attribute__((always_inline)) -> u32x4_a {
            u32x4_a p;
#pragma unroll
            for (int sb = 0; sb < 2; sb++) {
                f32x4_t v = sc[sb];
                if constexpr (F8)
#pragma unroll
                    for (int i = 0; i < 4; i++) v[i] = v[i] == 0.f ? 0.f : v[i] * t.vs[sb][i];
                p[2 * sb] = pk_bf16(v[0], v[1]);
                p[2 * sb + 1] = pk_bf16(v[2], v[3]);
            }
            return p;
        };

        // every row sees all of the tile's positions
        auto whole_tile = [&](int t0) {
            if (t0 < full_lo || t0 + TILE > full_hi) return false;
            const int e0 = trow[min(t0 >> ps, a.W - 1)], e1 = trow[min((t0 + 16) >> ps, a.W - 1)];
            return e0 >= 0 && e0 < a.kv.num_pages && e1 >= 0 && e1 < a.kv.num_pages;
        };
        for (int t0 = t_lo + w * TILE; t0 < t_hi; t0 += NW * TILE) {
            TL t;
            int page[2];
            load(t, t0, page);
            const bool whole = t0 >= full_lo && t0 + TILE <= full_hi && page[0] >= 0 && page[1] >= 0;   // = whole_tile(t0)
            // tiles that some row sees in part: which of this lane's positions are
            // there at all; values that no row sees become 0
            bool odd = false;               // an infinite or NaN value among those that are there
            uint32_t there = 0xFFu;
            if (!whole) {
                there = 0;
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const int pos = t0 + 16 * (j >> 2) + 4 * g4 + (j & 3);
                    const bool in = page[j >> 2] >= 0 && pos >= see_lo && pos < see_hi;
                    there |= (in ? 1u : 0u) << j;
#pragma unroll
                    for (int h = 0; h < NH; h++)
#pragma unroll
                        for (int q = 0; q < EW; q++) {
                            const uint32_t v = in ? t.v[j][h][q] : 0u;
                            t.v[j][h][q] = v;
                            if constexpr (F8) odd |= (((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;   // a byte 0x7F
                            else odd |= (v & 0x7F80u) == 0x7F80u || (v & 0x7F800000u) == 0x7F800000u;
                        }
                }
                // 0 * inf is NaN: an infinite or NaN value must not meet the zero
                // probability of a row that does not see it.  Such values become 0
                // here and are added to the rows that see them when the item ends.
                if (__any(odd)) {
                    strange = 1;
#pragma unroll
                    for (int j = 0; j < 8; j++)
#pragma unroll
                        for (int h = 0; h < NH; h++)
#pragma unroll
                            for (int q = 0; q < EW; q++) {
                                const uint32_t v = t.v[j][h][q];
                                uint32_t keep = 0;
                                if constexpr (F8) {
#pragma unroll
                                    for (int b = 0; b < 4; b++)
                                        keep |= ((v >> (8 * b)) & 0x7Fu) == 0x7Fu ? 0u : 0xFFu << (8 * b);
                                } else {
                                    keep = ((v & 0x7F80u) == 0x7F80u ? 0u : 0xFFFFu) |
                                           ((v & 0x7F800000u) == 0x7F800000u ? 0u : 0xFFFF0000u);
                                }
                                t.v[j][h][q] = v & keep;
                            }
                }
            }
            u32x4_a p[MT];
#pragma unroll
            for (int mt = 0; mt < MT; mt++) {
                f32x4_t sc[2];
                scores(t, mt, sc);
                if (!whole) {
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const int pos = t0 + 16 * (j >> 2) + 4 * g4 + (j & 3);
                        if (!((there >> j) & 1) || pos < vlo[mt] || pos > vhi[mt]) sc[j >> 2][j & 3] = -__builtin_inff();
                    }
                }
                soften(sc, mt);
                p[mt] = pack_p(t, sc);
            }
            values(t, p);
        }

        // the infinite and NaN values left out above, of elements d .. d + 3 and the
        // positions that a row at position p sees (every probability is > 0)
        auto add_strange = [&](f32x4_t& o, int p, int d) {
            for (int t0 = t_lo; t0 < t_hi; t0 += TILE) {
                if (whole_tile(t0)) continue;
                for (int pos = max(t0, a.window > 0 ? p - a.window + 1 : 0); pos < min(t0 + TILE, min(p + 1, see_hi)); pos++) {
                    const int e = trow[min(pos >> ps, a.W - 1)];
                    if (e < 0 || e >= a.kv.num_pages) continue;
                    const int64_t at = ((((int64_t)e * nkv + head) << ps) + (pos & pmask)) * D + d;
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        if constexpr (F8) {
                            if ((((const uint8_t*)a.kv.v)[at + c] & 0x7F) == 0x7F) o[c] = __builtin_nanf("");
                        } else {
                            const uint16_t v = ((const uint16_t*)a.kv.v)[at + c];
                            if ((v & 0x7F80) == 0x7F80) o[c] += bf16_to_f32(v);
                        }
                    }
                }
            }
        };

        // ---- join the block's waves, one row tile at a time
        const bool direct = nsplit == 1;
        const int64_t pidx = direct ? 0 : (int64_t)pstart[s] + (item - istart[s]);
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            float sm = sum[mt];
            sm += tr_partner<16>(sm);
            sm += tr_partner<32>(sm);
            __syncthreads();                // q rows, or the row tile before, are read
            if (g4 == 0) jml[w * 16 + r16] = make_float2(m[mt], sm);
            __syncthreads();
            float M = jml[r16].x;
#pragma unroll
            for (int i = 1; i < NW; i++) M = fmaxf(M, jml[i * 16 + r16].x);
            const float base = M == -__builtin_inff() ? 0.f : M;
            const float f = exp2f(m[mt] - base);
            // lane: row r16; O^T rows 4 g4 + i of MFMA e are d = 16 E h + E (4 g4 + i) + e
#pragma unroll
            for (int h = 0; h < NH; h++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    float* dst = ja + (w * 16 + r16) * DP + 16 * E * h + E * (4 * g4 + i);
#pragma unroll
                    for (int e = 0; e < E; e += 4)
                        *reinterpret_cast<f32x4_t*>(dst + e) =
                            f32x4_t{acc[mt][h][e][i] * f, acc[mt][h][e + 1][i] * f, acc[mt][h][e + 2][i] * f,
                                    acc[mt][h][e + 3][i] * f};
                }
            __syncthreads();
            // 16 threads per row, D / 16 elements each, 4 at a time
            const int rr = tid >> 4, part = tid & 15, row = mt * 16 + rr;
            if (row < nrows) {
                float Mr = jml[rr].x, L = 0.f;
#pragma unroll
                for (int i = 1; i < NW; i++) Mr = fmaxf(Mr, jml[i * 16 + rr].x);
                const float br = Mr == -__builtin_inff() ? 0.f : Mr;
#pragma unroll
                for (int i = 0; i < NW; i++) {
                    const float2 x2 = jml[i * 16 + rr];
                    L += x2.y * exp2f(x2.x - br);
                }
                const float inv = L == 0.f ? 0.f : 1.0f / L;
                const int grow = row0 + row, i = grow / G, g = grow - i * G;
                uint16_t* dst = a.out + ((int64_t)(rq.row0 + i) * a.n_heads + head * G + g) * D;
                float* pd = a.part + (pidx * RB + row) * D;
#pragma unroll
                for (int c = 0; c < D / 64; c++) {
                    const int d = c * 64 + part * 4;
                    f32x4_t o = *reinterpret_cast<const f32x4_t*>(ja + rr * DP + d);
#pragma unroll
                    for (int i2 = 1; i2 < NW; i2++) o += *reinterpret_cast<const f32x4_t*>(ja + (i2 * 16 + rr) * DP + d);
                    if (strange) add_strange(o, rq.first + i, d);
                    if (direct) {
                        // (a row that sees nothing: no sum, 0)
                        const u32x2_a q = {pk_bf16(o[0] * inv, o[1] * inv), pk_bf16(o[2] * inv, o[3] * inv)};
                        *reinterpret_cast<u32x2_a*>(dst + d) = q;
                    } else {
                        *reinterpret_cast<f32x4_t*>(pd + d) = o;
                    }
                }
                if (!direct && part == 0) a.ml[pidx * RB + row] = make_float2(Mr, L);
            }
        }
    }
}

// out = sum_c 2^{m_c - M} acc_c / sum_c 2^{m_c - M} sum_c over a request's splits,
// in split order.  One wave per (row of the batch, head): D / 64 elements a lane.
template <int D>
__global__ __launch_bounds__(AT_THREADS) void k_attn_join(const AttnArgs a, int rows_per_item) {
    constexpr int EL = D / 64;
    const int64_t id = (int64_t)blockIdx.x * NW + threadIdx.x / WAVE;
    const int t = (int)(id / a.n_heads), hq = (int)(id - (int64_t)t * a.n_heads), l = lane_id();
    if (t >= a.T) return;
    int s = 0, hi = a.S;
    while (hi - s > 1) {
        const int mid = (s + hi) >> 1;
        if (a.q_offsets[mid] <= t) s = mid;
        else hi = mid;
    }
    const int4 me = a.meta[s];
    const int nsplit = me.y;
    const int b = max(a.q_offsets[s], 0);
    if (nsplit <= 1 || t < b || t >= a.q_offsets[s + 1]) return;
    const int nkv = a.kv.n_kv_heads, G = a.n_heads / nkv;
    const int head = hq / G, row = (t - b) * G + (hq - head * G);
    const int grp = row / rows_per_item, rr = row - grp * rows_per_item;
    const int64_t p0 = (int64_t)me.x + ((int64_t)grp * nkv + head) * nsplit;
    float M = -__builtin_inff();
    for (int c = l; c < nsplit; c += WAVE) M = fmaxf(M, a.ml[(p0 + c) * rows_per_item + rr].x);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) M = fmaxf(M, wave_xor(M, d));
    const float base = M == -__builtin_inff() ? 0.f : M;
    float L = 0.f, o[EL];
#pragma unroll
    for (int e = 0; e < EL; e++) o[e] = 0.f;
    for (int c = 0; c < nsplit; c++) {
        const float2 x = a.ml[(p0 + c) * rows_per_item + rr];
        const float f = exp2f(x.x - base);
        L += x.y * f;
        const float* src = a.part + ((p0 + c) * rows_per_item + rr) * D + l * EL;
#pragma unroll
        for (int e = 0; e < EL; e++) o[e] += src[e] * f;
    }
    const float inv = L == 0.f ? 0.f : 1.0f / L;
    uint16_t* dst = a.out + ((int64_t)t * a.n_heads + hq) * D + l * EL;
#pragma unroll
    for (int e = 0; e < EL; e++) dst[e] = f32_to_bf16_rne(o[e] * inv);
}

// Rows per item: as many row tiles as a request has rows on average, so that
// its cache is read once; more than 64 rows (16 at head_dim 256, where the
// accumulators take MT x 64 registers) go over it again.
int row_tiles(int T, int n_heads, int n_kv_heads, int head_dim, int S) {
    const int64_t rows = ((int64_t)T * (n_heads / n_kv_heads) + S - 1) / S;
    const int most = head_dim == 256 ? 1 : 4;
    const int mt = (int)((rows + 15) / 16 < most ? (rows + 15) / 16 : most);
    return mt < 1 ? 1 : mt;
}

constexpr int TARGET_ITEMS = 512;           // two blocks on each of 256 CUs

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

struct AttnWs {
    size_t ml, part, total;
};
AttnWs attn_ws(int T, int n_heads, int n_kv_heads, int head_dim, int S) {
    const int rb = 16 * row_tiles(T, n_heads, n_kv_heads, head_dim, S);
    // a request with two splits or more has ceil(range / C) <= 2 range / C of
    // them per row group and head, and the ranges sum to at most target * C
    const size_t parts = 2 * (size_t)TARGET_ITEMS;
    AttnWs w;
    w.ml = up256((size_t)S * sizeof(int4));
    w.part = w.ml + up256(parts * rb * sizeof(float2));
    w.total = w.part + up256(parts * rb * head_dim * sizeof(float));
    return w;
}

template <int D, int F8, int MT>
hipError_t launch_attn(const AttnArgs& a, hipStream_t st) {
    auto kern = k_paged_attn<D, F8, MT>;
    const size_t head = ((size_t)(2 * a.S + 1) * 4 + 15) / 16 * 16;
    const size_t join = sizeof(float) * NW * 16 * (D + 4) + sizeof(float2) * NW * 16, qrows = (size_t)16 * MT * (D + 8) * 2;
    const size_t lds = head + (join > qrows ? join : qrows);
    static LdsLimit lim;
    hipError_t e = lim.ensure((const void*)kern, 128 * 1024);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3(a.target), dim3(AT_THREADS), lds, st, a);
    const int64_t waves = (int64_t)a.T * a.n_heads;
    hipLaunchKernelGGL((k_attn_join<D>), dim3((unsigned)((waves + NW - 1) / NW)), dim3(AT_THREADS), 0, st, a, 16 * MT);
    return hipGetLastError();
}

template <int D, int F8>
hipError_t launch_mt(const AttnArgs& a, int mt, hipStream_t st) {
    switch (mt) {
        case 1: return launch_attn<D, F8, 1>(a, st);
        default:
            if constexpr (D < 256) {
                if (mt == 2) return launch_attn<D, F8, 2>(a, st);
                if (mt == 3) return launch_attn<D, F8, 3>(a, st);
                return launch_attn<D, F8, 4>(a, st);
            }
    }
    return hipErrorInvalidValue;
}

}  // namespace

size_t paged_attn_workspace_bytes(int T, int n_heads, int n_kv_heads, int head_dim, int S) {
    return attn_ws(T, n_heads, n_kv_heads, head_dim, S).total;
}

hipError_t launch_paged_attn(const uint16_t* q, int64_t q_stride, int T, int n_heads, const KvView& cache,
                             const int32_t* table, int W, const int32_t* q_offsets, const int32_t* kv_len, int S,
                             float scale, float softcap, int window, uint16_t* out, void* ws, hipStream_t st) {
    if (T == 0) return hipSuccess;
    const AttnWs L = attn_ws(T, n_heads, cache.n_kv_heads, cache.head_dim, S);
    char* wb = (char*)ws;
    AttnArgs a{q,     q_stride, T,       n_heads, cache, table,        W,          q_offsets,           kv_len,
               S,     scale,    softcap, window,  out,   TARGET_ITEMS, (int4*)wb, (float*)(wb + L.part), (float2*)(wb + L.ml)};
    const int mt = row_tiles(T, n_heads, cache.n_kv_heads, cache.head_dim, S);
    const bool f8 = cache.k_scale != nullptr;
    switch (cache.head_dim) {
        case 64: return f8 ? launch_mt<64, 1>(a, mt, st) : launch_mt<64, 0>(a, mt, st);
        case 128: return f8 ? launch_mt<128, 1>(a, mt, st) : launch_mt<128, 0>(a, mt, st);
        case 256: return f8 ? launch_mt<256, 1>(a, mt, st) : launch_mt<256, 0>(a, mt, st);
    }
    return hipErrorInvalidValue;
}
