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
// waves of a block take the tiles in turn and are joined through LDS.
//
// The work, for a balanced load whatever the lengths: a unit is (request, row
// group, key-value head), its length in steps of 32 NW positions; all units'
// steps in a row, with a constant for each unit, are cut into equal shares, one
// per block.  A block walks the pieces of units in its share; a unit that lies in
// several shares leaves a partial result in each, which k_attn_join adds up in
// the order of the shares.
//
// Bound by HBM at few rows: each cached byte is used for 16 MT rows at a time.  One row over
// 262,144 positions (16 heads of 256 on 2, 537 MB): 86 us, 6.2 TB/s, and 6 us for the join; 64 requests
// of one row and up to 8192 positions, e4m3 (166 MB), 37 and 5 us, 4.5 TB/s.  5 rows over 4096 positions, 13 and 5 us for 8.5 MB, are
// latency: a block's 16 positions per wave pass q, the first tile, one softmax, the
// join through LDS and a partial result of 40 rows.
#include "attn_split.h"
#include "device.h"

namespace {

constexpr int NW = 4;                       // waves per block
static_assert(NW * WAVE == AT_THREADS);

// One wave's NSUB sub-tiles of 16 positions.
template <int D, int F8, int NSUB, int DS>
struct Tile {
    static constexpr int KV = F8 ? D / 64 : D / 32;       // 16-byte key chunks per lane and sub-tile
    static constexpr int E = D == 64 ? 4 : 8;             // value elements per lane and load
    static constexpr int NH = D / (16 * E);               // loads per position
    static constexpr int EW = F8 ? E / 4 : E / 2;         // their 32-bit words
    u32x4_a k[NSUB][KV];
    uint32_t v[4 * NSUB][NH / DS][EW];
    f32x4_t ks[NSUB], vs[NSUB];
};

// Buffer loads: a wave-uniform base, a byte offset per lane; `bytes` 0 makes
// every load return 0 without touching memory.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
MOE_DEV rsrc_t buffer_of(const void* base, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00027000);
}
template <int AUX>
MOE_DEV u32x4_a buf128(rsrc_t r, int off) { return __builtin_bit_cast(u32x4_a, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, AUX)); }
template <int AUX>
MOE_DEV u32x2_a buf64(rsrc_t r, int off) { return __builtin_bit_cast(u32x2_a, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, AUX)); }
template <int AUX>
MOE_DEV uint32_t buf32(rsrc_t r, int off) { return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, AUX); }

// blocks per CU, by registers
constexpr int blocks_per_cu(int D, int MT) { return MT == 1 || D == 64 || (D == 128 && MT == 2) || (D == 256 && MT == 2) ? 2 : 1; }
constexpr int shares_of(int D, int MT) { return 256 * blocks_per_cu(D, MT); }

// A kernel's shape: row tiles, sub-tiles per wave step, blocks per CU.
template <int D, int F8, int MT>
struct Shape {
    // Head parts: at head_dim 256 with more than one row tile two waves share
    // their positions (and compute their scores twice), each summing the values of
    // half of the head: half the accumulators, and half the planes to join.
    static constexpr int DS = D == 256 && MT > 1 ? 2 : 1;
    // sub-tiles per wave step: 16 KB of cache in flight per wave (8 KB of e4m3), by registers
    static constexpr int NSUB = D == 256 && (MT == 2 || (MT == 1 && !F8)) ? 1 : 2;
    static constexpr int STEP = 16 * NSUB * NW / DS;    // positions per block step
    static constexpr bool QREG = D * MT <= 128;     // q fragments in registers (up to 16 of them), else LDS at each use
};

template <int D, int F8, int MT>
__global__ __launch_bounds__(AT_THREADS, (blocks_per_cu(D, MT))) void k_paged_attn(const AttnArgs a) {
    constexpr int NSUB = Shape<D, F8, MT>::NSUB;
    constexpr bool QREG = Shape<D, F8, MT>::QREG;
    constexpr int DS = Shape<D, F8, MT>::DS, PW = NW / DS, STEP = Shape<D, F8, MT>::STEP;
    using TL = Tile<D, F8, NSUB, DS>;
    constexpr int E = TL::E, NH = TL::NH / DS, EW = TL::EW, KV = TL::KV;
    constexpr int TILE = 16 * NSUB;         // positions per wave step
    constexpr int RB = 16 * MT;             // rows per unit
    constexpr int NT = MT == 1 ? 2 : 0;     // the cache is read once: non-temporal
    constexpr int DP = D + 4;               // padded row of the join area
    constexpr int QP = D + 8;               // padded q row, bf16
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    // more than 64 requests: [S] first steps; then the q rows / join area
    const bool lanes = a.S <= WAVE;
    int* base = (int*)smem;
    unsigned char* area = smem + (lanes ? 0 : ((size_t)a.S * 4 + 15) / 16 * 16);
    uint16_t* qs = (uint16_t*)area;                              // [RB][QP]
    float* ja = (float*)area;                                    // [PW][RB][DP]
    float2* jml = (float2*)(area + sizeof(float) * PW * RB * DP);  // [PW][RB]
    __shared__ int sc32[NW];
    __shared__ int strange;                 // the piece met infinite or NaN values in a tile seen in part

    const int tid = threadIdx.x, l = lane_id(), w = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int wp = w % PW, wd = w / PW;     // the wave's positions and head part
    const int G = a.G, nkv = a.kv.n_kv_heads;

    // ---- first step of every request.  Up to 64 requests: lane s holds request
    // s, in every wave by itself.  More: running sums through LDS, 256 at a time.
    Request mine;
    int my_base = 0, total;
    if (lanes) {
        mine = request_of<RB, STEP, false>(a, min(l, a.S - 1));
        if (l >= a.S) mine.units = 0;
        const int c = mine.units * mine.steps, incl = wave_incl_scan(c);
        total = __builtin_amdgcn_readlane(incl, WAVE - 1);
        my_base = incl - c;
        if (blockIdx.x == 0 && w == 0 && l < a.S) a.base[l] = my_base;
    } else {
        total = 0;
        for (int s0 = 0; s0 < a.S; s0 += AT_THREADS) {
            const int s = s0 + tid;
            int c = 0;
            if (s < a.S) {
                const Request r = request_of<RB, STEP, false>(a, s);
                c = r.units * r.steps;
            }
            const int incl = wave_incl_scan(c);
            __syncthreads();                // the scratch's last readers are done
            if (l == WAVE - 1) sc32[w] = incl;
            __syncthreads();
            int b = total;
#pragma unroll
            for (int i = 0; i < NW; i++) {
                if (i < w) b += sc32[i];
                total += sc32[i];
            }
            if (s < a.S) {
                base[s] = b + incl - c;
                if (blockIdx.x == 0) a.base[s] = b + incl - c;
            }
        }
        __syncthreads();
        total = __builtin_amdgcn_readfirstlane(total);
    }
    const int share = max((int)(((uint32_t)total + a.shares - 1) / a.shares), 1);
    if (blockIdx.x == 0 && tid == 0) a.share[0] = share;
    const int share_lo = min((int64_t)blockIdx.x * share, (int64_t)total);
    const int share_hi = min((int64_t)share_lo + share, (int64_t)total);

    const int r16 = l & 15, g4 = l >> 4;
    const float qscale = a.softcap > 0.f ? a.scale / a.softcap : a.scale * LOG2E;
    const float capk = a.softcap * LOG2E;
    const int ps = a.kv.page_shift, pmask = (1 << ps) - 1;

    for (int at = share_lo; at < share_hi;) {
        int s;
        Request rq;
        int s_base;
        if (lanes) {
            s = __popcll(__ballot(l < a.S && my_base <= at)) - 1;      // (empty requests share a base with their successor)
            rq.row0 = __builtin_amdgcn_readlane(mine.row0, s);
            rq.n = __builtin_amdgcn_readlane(mine.n, s);
            rq.first = __builtin_amdgcn_readlane(mine.first, s);
            rq.len = __builtin_amdgcn_readlane(mine.len, s);
            rq.units = __builtin_amdgcn_readlane(mine.units, s);
            rq.steps = __builtin_amdgcn_readlane(mine.steps, s);
            s_base = __builtin_amdgcn_readlane(my_base, s);
        } else {
            s = 0;
            int hi = a.S;
            while (hi - s > 1) {
                const int mid = (s + hi) >> 1;
                if (base[mid] <= at) s = mid;
                else hi = mid;
            }
            s = __builtin_amdgcn_readfirstlane(s);
            rq = request_of<RB, STEP, false>(a, s);
            s_base = base[s];
        }
        // (the same in every lane, and kept in scalar registers: buffer descriptors
        // made from vector registers cost a loop around each load)
        s = uniform(s);
        s_base = uniform(s_base);
        rq.row0 = uniform(rq.row0);
        rq.n = uniform(rq.n);
        rq.first = uniform(rq.first);
        rq.len = uniform(rq.len);
        rq.units = uniform(rq.units);
        rq.steps = uniform(rq.steps);
        // the piece: steps [st0, st1) of unit (row group, head)
        const int unit = uniform((int)((uint32_t)(at - s_base) / (uint32_t)rq.steps));
        if ((uint32_t)unit >= (uint32_t)rq.units) return;    // (offsets that do not ascend, their steps past int32: no row is read)
        const int st0 = at - s_base - unit * rq.steps;
        if (a.whole && st0 > 0) {           // the share before has it
            at += rq.steps - st0;
            continue;
        }
        const int st1 = a.whole ? rq.steps : min(rq.steps, st0 + (share_hi - at));
        const int piece_at = at;
        at += st1 - st0;
        const int grp = uniform((int)((uint32_t)unit / (uint32_t)nkv)), head = unit - grp * nkv;
        const int row0 = grp * RB, nrows = min(RB, rq.n * G - row0);
        const int i0 = (int)((uint32_t)row0 / (uint32_t)G), r_in = row0 - i0 * G;   // row0 = token i0, its head r_in
        const int i1 = i0 + (((r_in + nrows - 1) * a.G16) >> 16);
        // positions [see_lo, see_hi) that some row of the unit sees; the piece's
        // steps are its share of them (units of a request have equally many
        // steps, though the first rows of a long prompt see less)
        const int p_lo = rq.first + i0, p_hi = rq.first + i1;       // positions of its first and last row
        const int see_lo = a.window > 0 ? max(p_lo - a.window + 1, 0) : 0;
        const int see_hi = max(min(p_hi + 1, rq.len), 0);
        const int a0 = see_lo & ~(TILE - 1);
        const int real_steps = (max(see_hi - a0, 0) + STEP - 1) / STEP;
        const float stretch = (float)real_steps / (float)rq.steps;
        auto step_at = [&](int st) {        // monotone in st, whole at the end: neighbouring pieces meet
            return st == rq.steps || real_steps == rq.steps ? min(st, real_steps) : min((int)((float)st * stretch), real_steps);
        };
        const int t_lo = uniform((int)min((int64_t)a0 + (int64_t)step_at(st0) * STEP, (int64_t)see_hi));
        const int t_hi = uniform(st1 == rq.steps ? see_hi : (int)min((int64_t)a0 + (int64_t)step_at(st1) * STEP, (int64_t)see_hi));
        // every row sees [full_lo, full_hi) whole
        const int full_lo = a.window > 0 ? max(p_hi - a.window + 1, 0) : 0;
        const int full_hi = min(p_lo + 1, rq.len);

        const table_ptr trow = (table_ptr)(uintptr_t)(a.table + (int64_t)s * a.W);
        // pages of a tile's sub-tiles; -1: none (outside the cache, or past the piece)
        struct Pages { int p[NSUB]; };
        auto pages_of = [&](int t0) __attribute__((always_inline)) {
            Pages e;
#pragma unroll
            for (int sb = 0; sb < NSUB; sb++) {
                const int v = trow[min((t0 + 16 * sb) >> ps, a.W - 1)];
                e.p[sb] = uniform((v >= 0 && v < a.kv.num_pages && t0 < t_hi) ? v : -1);
            }
            return e;
        };
        constexpr int ES = F8 ? 1 : 2, X = 16 / ES;          // element bytes, elements per key chunk
        auto load_k = [&](TL& t, int t0, const Pages& pg) __attribute__((always_inline)) {
#pragma unroll
            for (int sb = 0; sb < NSUB; sb++) {
                const int64_t ph = (int64_t)max(pg.p[sb], 0) * nkv + head;
                const int off = (t0 + 16 * sb) & pmask;
                const rsrc_t r = buffer_of((const char*)a.kv.k + (((ph * (D / X)) << ps) + off) * 16,
                                           pg.p[sb] < 0 ? 0 : ((D / X) << ps) * 16 - off * 16);
#pragma unroll
                for (int c = 0; c < KV; c++) t.k[sb][c] = buf128<NT>(r, (((4 * c + g4) << ps) + r16) * 16);
                if constexpr (F8)
                    t.ks[sb] = __builtin_bit_cast(f32x4_t, buf128<NT>(buffer_of(a.kv.k_scale + (ph << ps) + off, pg.p[sb] < 0 ? 0 : 64), g4 * 16));
            }
        };
        auto load_v = [&](TL& t, int t0, const Pages& pg) __attribute__((always_inline)) {
#pragma unroll
            for (int sb = 0; sb < NSUB; sb++) {
                const int64_t ph = (int64_t)max(pg.p[sb], 0) * nkv + head;
                const int off = (t0 + 16 * sb) & pmask;
                const rsrc_t r = buffer_of((const char*)a.kv.v + (((ph << ps) + off) * D + wd * (D / DS)) * ES,
                                           pg.p[sb] < 0 ? 0 : (16 * D - wd * (D / DS)) * ES);
#pragma unroll
                for (int j = 0; j < 4; j++)
#pragma unroll
                    for (int h = 0; h < NH; h++) {
                        const int at = (4 * g4 * D + r16 * E + j * D + h * 16 * E) * ES;
                        uint32_t* v = t.v[4 * sb + j][h];
                        if constexpr (EW == 4) {
                            const u32x4_a q = buf128<NT>(r, at);
#pragma unroll
                            for (int i = 0; i < 4; i++) v[i % EW] = q[i];
                        } else if constexpr (EW == 2) {
                            const u32x2_a q = buf64<NT>(r, at);
                            v[0] = q[0];
                            v[1 % EW] = q[1];
                        } else {
                            v[0] = buf32<NT>(r, at);
                        }
                    }
                if constexpr (F8)
                    t.vs[sb] = __builtin_bit_cast(f32x4_t, buf128<NT>(buffer_of(a.kv.v_scale + (ph << ps) + off, pg.p[sb] < 0 ? 0 : 64), g4 * 16));
            }
        };

        // ---- the unit's q rows (row r = query token i0.., head of the group), as
        // the fragments of the first product: bf16 keys: step k, lane group g4
        // holds chunk 4 k + g4; e4m3: chunk 4 (k / 2) + g4 of 16 elements, half k & 1
        auto q_dim = [&](int k) __attribute__((always_inline)) {
            return F8 ? 16 * (4 * (k >> 1) + g4) + 8 * (k & 1) : 32 * k + 8 * g4;
        };
        auto q_row = [&](int rr) __attribute__((always_inline)) -> const uint16_t* {
            const int x = r_in + min(rr, nrows - 1);            // (rows past the unit's repeat its last, unused)
            const int i = (x * a.G16) >> 16, g = x - i * G;
            return a.q + (int64_t)(rq.row0 + i0 + i) * a.q_stride + (int64_t)(head * G + g) * D;
        };
        // the loads go out before the first tile's: they are waited for first
        constexpr int QC = RB * (D / 8), QN = QREG ? 1 : (QC + AT_THREADS - 1) / AT_THREADS;
        bf16x8_t qf[QREG ? MT : 1][QREG ? D / 32 : 1];
        u32x4_a qv[QN];
        if constexpr (QREG) {
#pragma unroll
            for (int mt = 0; mt < MT; mt++) {
                const uint16_t* src = q_row(mt * 16 + r16);
#pragma unroll
                for (int k = 0; k < D / 32; k++) qf[mt][k] = *reinterpret_cast<const bf16x8_t*>(src + q_dim(k));
            }
        } else {
#pragma unroll
            for (int n = 0; n < QN; n++) {
                const int c = min(n * AT_THREADS + tid, QC - 1);
                qv[n] = *reinterpret_cast<const u32x4_a*>(q_row(c / (D / 8)) + c % (D / 8) * 8);
            }
        }
        TL t;
        const int t_first = t_lo + wp * TILE;
        Pages pg = pages_of(t_first), pg_next = pages_of(t_first + STEP);
        load_k(t, t_first, pg);
        load_v(t, t_first, pg);
        lds_barrier();                      // the last piece's join area is read
        if (tid == 0) strange = 0;
        if constexpr (!QREG) {
#pragma unroll
            for (int n = 0; n < QN; n++) {
                const int c = min(n * AT_THREADS + tid, QC - 1);        // (the last chunk again, the same value)
                *reinterpret_cast<u32x4_a*>(qs + c / (D / 8) * QP + c % (D / 8) * 8) = qv[n];
            }
        }
        lds_barrier();
        auto q_frag = [&](int mt, int k) __attribute__((always_inline)) {
            if constexpr (QREG) return qf[mt][k];
            else return *reinterpret_cast<const bf16x8_t*>(qs + (mt * 16 + r16) * QP + q_dim(k));
        };
        // this lane's row in each row tile: the positions it sees, [vlo, vhi]
        int vlo[MT], vhi[MT];
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            const int p = rq.first + i0 + (((r_in + mt * 16 + r16) * a.G16) >> 16);
            vhi[mt] = mt * 16 + r16 < nrows ? min(p, rq.len - 1) : -1;
            vlo[mt] = a.window > 0 ? max(p - a.window + 1, 0) : 0;
        }

        f32x4_t acc[MT][NH][E];
        // running sums of the weights: bf16 values, a row of ones of the second
        // product (the whole sum in every lane); e4m3, this lane's positions
        float m[MT];
        f32x4_t sum[MT];
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            m[mt] = -__builtin_inff();
            sum[mt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < NH; h++)
#pragma unroll
                for (int e = 0; e < E; e++) acc[mt][h][e] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }

        // S^T of one row tile: [sub-tile][i], in units of log2
        auto scores = [&](const TL& t, int mt, f32x4_t (&sc)[NSUB]) __attribute__((always_inline)) {
#pragma unroll
            for (int sb = 0; sb < NSUB; sb++) {
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
                    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q_frag(mt, k), c, 0, 0, 0);
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
        // O^T += V^T P^T over sub-tiles 2 pr and 2 pr + 1 (NSUB 1: the one there is)
        constexpr int JP = NSUB == 1 ? 2 : 4;             // pairs of positions per product
        auto mma = [&](const uint32_t (&f)[JP], const uint32_t (&p)[JP], f32x4_t c) __attribute__((always_inline)) {
            if constexpr (NSUB == 1) {
                return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4_a, f),
                                                                 __builtin_bit_cast(s16x4_a, p), c, 0, 0, 0);
            } else {
                return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f),
                                                               __builtin_bit_cast(bf16x8_t, p), c, 0, 0, 0);
            }
        };
        auto values = [&](const TL& t, const uint32_t (&p)[MT][2 * NSUB]) __attribute__((always_inline)) {
            constexpr int PER = F8 ? 4 : 2;               // elements per word
            if constexpr (!F8) {
                uint32_t one[JP];
#pragma unroll
                for (int j = 0; j < JP; j++) one[j] = 0x3F803F80u;
#pragma unroll
                for (int mt = 0; mt < MT; mt++) {
                    uint32_t pp[JP];
#pragma unroll
                    for (int j = 0; j < JP; j++) pp[j] = p[mt][j];
                    sum[mt] = mma(one, pp, sum[mt]);
                }
            }
#pragma unroll
            for (int pr = 0; pr < 2 * NSUB / JP; pr++)
#pragma unroll
                for (int h = 0; h < NH; h++)
#pragma unroll
                    for (int q = 0; q < EW; q++) {
                        uint32_t f[PER][JP];
#pragma unroll
                        for (int j = 0; j < JP; j++) {
                            const uint32_t x = t.v[2 * (pr * JP + j)][h][q], y = t.v[2 * (pr * JP + j) + 1][h][q];
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
                        for (int mt = 0; mt < MT; mt++) {
                            uint32_t pp[JP];
#pragma unroll
                            for (int j = 0; j < JP; j++) pp[j] = p[mt][pr * JP + j];
#pragma unroll
                            for (int e = 0; e < PER; e++)
                                acc[mt][h][PER * q + e] = mma(f[e], pp, acc[mt][h][PER * q + e]);
                        }
                    }
        };
        // running maxima; scores -> probabilities.  The row tiles go together (one
        // branch, independent chains).
        auto soften = [&](f32x4_t (&sc)[MT][NSUB]) __attribute__((always_inline)) {
            float top[MT];
            bool rise = false;
#pragma unroll
            for (int mt = 0; mt < MT; mt++) {
                float t = -__builtin_inff();
#pragma unroll
                for (int sb = 0; sb < NSUB; sb++)
                    t = fmaxf(t, fmaxf(fmaxf(sc[mt][sb][0], sc[mt][sb][1]), fmaxf(sc[mt][sb][2], sc[mt][sb][3])));
                t = fmaxf(t, tr_partner<16>(t));
                top[mt] = fmaxf(t, tr_partner<32>(t));
                rise |= top[mt] > m[mt] + 8.f;
            }
            // The base of the exponentials follows a row's maximum only when some row's
            // has risen by more than 2^8: until then its probabilities grow to 256 at
            // most, as exact as below 1, and nothing is scaled.
            if (__any(rise)) {
                bool seen = false;
#pragma unroll
                for (int mt = 0; mt < MT; mt++) seen |= m[mt] > -__builtin_inff();
                const bool scale = __any(seen);              // (nothing to scale before the first tile that a row sees)
#pragma unroll
                for (int mt = 0; mt < MT; mt++) {
                    const float mn = fmaxf(m[mt], top[mt]);
                    if (scale) {
                        const float f = __builtin_amdgcn_exp2f(m[mt] - (mn == -__builtin_inff() ? 0.f : mn));
                        if constexpr (F8) sum[mt][0] *= f;
                        else sum[mt] *= f;
#pragma unroll
                        for (int h = 0; h < NH; h++)
#pragma unroll
                            for (int e = 0; e < E; e++) acc[mt][h][e] *= f;
                    }
                    m[mt] = mn;
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; mt++) {
                const float base = m[mt] == -__builtin_inff() ? 0.f : m[mt];     // a row that has seen nothing yet
#pragma unroll
                for (int sb = 0; sb < NSUB; sb++)
#pragma unroll
                    for (int i = 0; i < 4; i++) sc[mt][sb][i] = __builtin_amdgcn_exp2f(sc[mt][sb][i] - base);
            }
        };
        // the second product's operand, and the running sum of the weights as that
        // product sees them: the sum of the rounded probabilities, so that their
        // rounding (half a step of bf16) cancels where few positions dominate.
        // e4m3 values: the weight is p v_scale, rounded; the sum takes it over v_scale.
        auto pack_p = [&](const TL& t, const f32x4_t (&sc)[NSUB], int mt, uint32_t (&p)[2 * NSUB])
                          __attribute__((always_inline)) {
#pragma unroll
            for (int sb = 0; sb < NSUB; sb++) {
                f32x4_t v = sc[sb];
                if constexpr (F8)
#pragma unroll
                    for (int i = 0; i < 4; i++) v[i] = v[i] == 0.f ? 0.f : v[i] * t.vs[sb][i];
                p[2 * sb] = pk_bf16(v[0], v[1]);
                p[2 * sb + 1] = pk_bf16(v[2], v[3]);
                if constexpr (F8) {
                    f32x4_t u = {bf16lo_to_f32(p[2 * sb]), bf16hi_to_f32(p[2 * sb]), bf16lo_to_f32(p[2 * sb + 1]),
                                 bf16hi_to_f32(p[2 * sb + 1])};
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        u[i] = u[i] == 0.f ? sc[sb][i] : u[i] * __builtin_amdgcn_rcpf(t.vs[sb][i]);
                    sum[mt][0] += (u[0] + u[1]) + (u[2] + u[3]);
                }
            }
        };
        // position of this lane's j-th value of the tile
        auto pos_of = [&](int t0, int j) __attribute__((always_inline)) { return t0 + 16 * (j >> 2) + 4 * g4 + (j & 3); };

        // The tile's registers are refilled as they are used up: the next tile's
        // keys load under this one's softmax and second product, its values under
        // the next one's scores, and its pages are looked up a tile ahead.  (Past
        // the last tile the loads return at once.)
        for (int t0 = t_first; t0 < t_hi; t0 += STEP) {
            bool pages = true;
#pragma unroll
            for (int sb = 0; sb < NSUB; sb++) pages = pages && pg.p[sb] >= 0;
            const bool whole = pages && t0 >= full_lo && t0 + TILE <= full_hi;      // = whole_tile(t0)
            // tiles that some row sees in part: which of this lane's positions are
            // there at all; values that no row sees become 0
            uint32_t there = 0xFFFFFFFFu;
            if (!whole) {
                bool odd = false;           // an infinite or NaN value among those that are there
                there = 0;
#pragma unroll
                for (int j = 0; j < 4 * NSUB; j++) {
                    const int pos = pos_of(t0, j);
                    const bool in = pg.p[j >> 2] >= 0 && pos >= see_lo && pos < see_hi;
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
                // here and are added to the rows that see them when the piece ends.
                if (__any(odd)) {
                    strange = 1;
#pragma unroll
                    for (int j = 0; j < 4 * NSUB; j++)
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
            f32x4_t sc[MT][NSUB];
            if constexpr (!QREG) asm volatile("" ::: "memory");   // the q fragments are read again for every tile
#pragma unroll
            for (int mt = 0; mt < MT; mt++) scores(t, mt, sc[mt]);
            load_k(t, t0 + STEP, pg_next);
            if (!whole) {
#pragma unroll
                for (int mt = 0; mt < MT; mt++)
#pragma unroll
                    for (int j = 0; j < 4 * NSUB; j++) {
                        const int pos = pos_of(t0, j);
                        if (!((there >> j) & 1) || pos < vlo[mt] || pos > vhi[mt]) sc[mt][j >> 2][j & 3] = -__builtin_inff();
                    }
            }
            soften(sc);
            uint32_t p[MT][2 * NSUB];
#pragma unroll
            for (int mt = 0; mt < MT; mt++) pack_p(t, sc[mt], mt, p[mt]);
            values(t, p);
            load_v(t, t0 + STEP, pg_next);
            pg = pg_next;
            pg_next = pages_of(t0 + 2 * STEP);
        }

        // every row sees all of the tile's positions
        auto whole_tile = [&](int t0) {
            if (t0 < full_lo || t0 + TILE > full_hi) return false;
            for (int pos = t0; pos < t0 + TILE; pos += 16) {
                const int e = trow[min(pos >> ps, a.W - 1)];
                if (e < 0 || e >= a.kv.num_pages) return false;
            }
            return true;
        };
        // the infinite and NaN values left out above, of elements d + {0, 1, 2, 3} sd
        // and the positions that a row at position p sees (every probability is > 0)
        auto add_strange = [&](f32x4_t& o, int p, int d, int sd) {
            for (int t0 = t_lo; t0 < t_hi; t0 += TILE) {
                if (whole_tile(t0)) continue;
                for (int pos = max(t0, a.window > 0 ? p - a.window + 1 : 0); pos < min(t0 + TILE, min(p + 1, see_hi)); pos++) {
                    const int e = trow[min(pos >> ps, a.W - 1)];
                    if (e < 0 || e >= a.kv.num_pages) continue;
                    const int64_t at = ((((int64_t)e * nkv + head) << ps) + (pos & pmask)) * D + d;
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        if constexpr (F8) {
                            if ((((const uint8_t*)a.kv.v)[at + c * sd] & 0x7F) == 0x7F) o[c] = __builtin_nanf("");
                        } else {
                            const uint16_t v = ((const uint16_t*)a.kv.v)[at + c * sd];
                            if ((v & 0x7F80) == 0x7F80) o[c] += bf16_to_f32(v);
                        }
                    }
                }
            }
        };

        // ---- join the block's waves through LDS.  A unit that lies in this share
        // alone is done; of others the piece that begins with the share is partial
        // 2 b, one that begins inside it 2 b + 1.  (What runs once per piece is kept
        // in loops: its code is paid for in instruction fetches, about 60 ns per 64
        // bytes.)
        const bool direct = st1 - st0 == rq.steps;
        const int64_t pidx = 2 * (int64_t)blockIdx.x + (piece_at == share_lo ? 0 : 1);
        if (!QREG) lds_barrier();           // the q rows are read
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            float sm = sum[mt][0];
            if constexpr (F8) {
                sm += tr_partner<16>(sm);
                sm += tr_partner<32>(sm);
            }
            if (g4 == 0 && wd == 0) jml[wp * RB + mt * 16 + r16] = make_float2(m[mt], sm);
            // O^T rows 4 g4 + i of MFMA (h, e) are d = 16 E h + E (4 g4 + i) + e: kept
            // in that order, (h, e, 4 g4 + i), here and in the partial results
#pragma unroll
            for (int h = 0; h < NH; h++)
#pragma unroll
                for (int e = 0; e < E; e++)
                    *reinterpret_cast<f32x4_t*>(ja + (wp * RB + mt * 16 + r16) * DP + ((wd * NH + h) * E + e) * 16 + 4 * g4) =
                        acc[mt][h][e];
        }
        lds_barrier();
        // 16 threads per row, D / 16 elements each, 4 at a time
        const int rr = tid >> 4, part = tid & 15;
        if (strange) {
            for (int row = rr; row < nrows; row += 16) {
                int top = 0;                // a wave whose sums enter unscaled
                for (int i = 1; i < PW; i++) top = jml[i * RB + row].x > jml[top * RB + row].x ? i : top;
                const int p = rq.first + i0 + (((r_in + row) * a.G16) >> 16);
                for (int c = part; c < D / 4; c += 16) {
                    f32x4_t* o = reinterpret_cast<f32x4_t*>(ja + (top * RB + row) * DP + c * 4);
                    f32x4_t v = *o;
                    add_strange(v, p, dim_of<D>(c), E);
                    *o = v;
                }
            }
        }
#pragma unroll 1
        for (int row = rr; row < nrows; row += 16) {
            float2 x[PW];
#pragma unroll
            for (int i = 0; i < PW; i++) x[i] = jml[i * RB + row];
            f32x4_t o[D / 64];
#pragma unroll
            for (int c = 0; c < D / 64; c++) o[c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            float Mr = x[0].x, L = 0.f;
#pragma unroll
            for (int i = 1; i < PW; i++) Mr = fmaxf(Mr, x[i].x);
            const float br = Mr == -__builtin_inff() ? 0.f : Mr;
#pragma unroll
            for (int i = 0; i < PW; i++) {
                const float f = __builtin_amdgcn_exp2f(x[i].x - br);
                L += x[i].y * f;
#pragma unroll
                for (int c = 0; c < D / 64; c++)
                    o[c] += *reinterpret_cast<const f32x4_t*>(ja + (i * RB + row) * DP + (c * 16 + part) * 4) * f;
            }
            if (direct) {
                const float inv = L == 0.f ? 0.f : __builtin_amdgcn_rcpf(L);     // (a row that sees nothing: 0)
                const int x0 = r_in + row, i = (x0 * a.G16) >> 16, g = x0 - i * G;
                uint16_t* dst = a.out + ((int64_t)(rq.row0 + i0 + i) * a.n_heads + head * G + g) * D;
#pragma unroll
                for (int c = 0; c < D / 64; c++)
#pragma unroll
                    for (int q = 0; q < 4; q++) dst[dim_of<D>(c * 16 + part) + E * q] = (uint16_t)pk_bf16(o[c][q] * inv, 0.f);
            } else {
                float* pd = a.part + (pidx * RB + row) * D;
#pragma unroll
                for (int c = 0; c < D / 64; c++) *reinterpret_cast<f32x4_t*>(pd + (c * 16 + part) * 4) = o[c];
                if (part == 0) a.ml[pidx * RB + row] = make_float2(Mr, L);
            }
        }
    }
}

// Row tiles per unit: as many as a request has rows on average, so that its
// cache is read once; more than 64 rows (48 at head_dim 256, where the
// accumulators take MT x 64 registers) go over it again.
int row_tiles(int T, int n_heads, int n_kv_heads, int head_dim, int S) {
    const int64_t rows = ((int64_t)T * (n_heads / n_kv_heads) + S - 1) / S;
    const int most = head_dim == 256 ? 3 : 4;
    const int mt = (int)((rows + 15) / 16 < most ? (rows + 15) / 16 : most);
    return mt < 1 ? 1 : mt;
}

// Many rows per request: prompt_attn.hip's kernel reads the cache once for 256
// rows, where this one goes over it again for every 64, but its blocks take longer to
// fill and leave more to join.  It is taken from 2^25 scores on (rows x positions of
// the table or window; the requests' own lengths are on the device), if the
// requests have more than 128 rows on average.  Both sides, this one's time first, on
// requests of r rows x positions, 2 key-value heads: D 128, 8 of 256 x 16,384 115 us against 82,
// of 1024 x 2048 63 against 58 and below the bound 8 of 512 x 2048 49 against 53; D 256, 1024 x 16,384 126
// against 113, 8 of 512 x 2048 79 against 90; D 64, 1024 x 16,384 47 against 42, 8 of 512 x 2048 37
// against 43; at 128 rows, D 256, 8 x 16,384 145 against 170.
bool many_rows(int T, int n_heads, int n_kv_heads, int S) { return (int64_t)T * (n_heads / n_kv_heads) > (int64_t)128 * S; }
bool take_prompt(const AttnArgs& a) {
    const int64_t table = (int64_t)a.W << a.kv.page_shift, seen = (int64_t)a.window + a.T / a.S;
    return many_rows(a.T, a.n_heads, a.kv.n_kv_heads, a.S) &&
           (int64_t)a.T * a.n_heads * (a.window > 0 && seen < table ? seen : table) >= 1 << 25;
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

struct AttnWs {
    size_t ml, part, total;
};
AttnWs attn_ws(int T, int n_heads, int n_kv_heads, int head_dim, int S) {
    const int mt = row_tiles(T, n_heads, n_kv_heads, head_dim, S);
    const PromptShape ps = prompt_attn_shape();
    const size_t few = (size_t)shares_of(head_dim, mt) * 16 * mt, many = (size_t)ps.shares * ps.rows;
    const size_t rows = 2 * (many_rows(T, n_heads, n_kv_heads, S) && many > few ? many : few);
    AttnWs w;
    w.ml = up256(((size_t)S + 1) * sizeof(int));
    w.part = w.ml + up256(rows * sizeof(float2));
    w.total = w.part + up256(rows * head_dim * sizeof(float));
    return w;
}

template <int D, int F8, int MT>
hipError_t launch_attn(AttnArgs a, hipStream_t st) {
    using SH = Shape<D, F8, MT>;
    auto kern = k_paged_attn<D, F8, MT>;
    const size_t head = a.S <= WAVE ? 0 : ((size_t)a.S * 4 + 15) / 16 * 16;
    const size_t join = (sizeof(float) * (D + 4) + sizeof(float2)) * 16 * MT * (NW / SH::DS);
    const size_t qrows = SH::QREG ? 0 : (size_t)16 * MT * (D + 8) * 2;
    const size_t lds = head + (join > qrows ? join : qrows);
    static LdsLimit lim;
    hipError_t e = lim.ensure((const void*)kern, 156 * 1024);
    if (e != hipSuccess) return e;
    a.shares = shares_of(D, MT);
    hipLaunchKernelGGL(kern, dim3(a.shares), dim3(AT_THREADS), lds, st, a);
    if (a.whole) return hipGetLastError();
    const int64_t chunks = (int64_t)a.T * a.n_heads * (D / 64);
    auto launch_join = [&](auto kern, dim3 grid, int threads) { hipLaunchKernelGGL(kern, grid, dim3(threads), 0, st, a); };
    if (chunks <= 128) launch_join(k_attn_join<D, 16 * MT, SH::STEP, false, 64, 16>, dim3(a.T, a.n_heads * (D / 64)), 16 * WAVE);
    else if (chunks <= 1024) launch_join(k_attn_join<D, 16 * MT, SH::STEP, false, 64, 4>, dim3(a.T, a.n_heads * (D / 64)), 4 * WAVE);
    else launch_join(k_attn_join<D, 16 * MT, SH::STEP, false, D, 1>, dim3(a.T, (a.n_heads + NW - 1) / NW), AT_THREADS);
    return hipGetLastError();
}

template <int D, int F8>
hipError_t launch_mt(const AttnArgs& a, int mt, hipStream_t st) {
    switch (mt) {
        case 1: return launch_attn<D, F8, 1>(a, st);
        case 2: return launch_attn<D, F8, 2>(a, st);
        case 3: return launch_attn<D, F8, 3>(a, st);
        default:
            if constexpr (D < 256) return launch_attn<D, F8, 4>(a, st);
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
    AttnArgs a{};
    a.q = q; a.q_stride = q_stride; a.T = T; a.n_heads = n_heads; a.kv = cache;
    a.table = table; a.W = W; a.q_offsets = q_offsets; a.kv_len = kv_len; a.S = S;
    a.scale = scale; a.softcap = softcap; a.out = out;
    a.window = window >= 1 << 30 ? 0 : window;     // positions stay below 2^30: no window
    // contexts of up to 512 positions are at most a few steps long: no splitting,
    // and no second launch (one to eight such requests: 14 -> 8 us a call)
    a.whole = (int64_t)W << cache.page_shift <= 512;
    a.share = (int*)wb; a.base = (int*)wb + 1;
    a.G = n_heads / cache.n_kv_heads; a.G16 = (65536 + a.G - 1) / a.G;
    a.ml = (float2*)(wb + L.ml); a.part = (float*)(wb + L.part);
    if (take_prompt(a)) return launch_prompt_attn(a, st);
    const int mt = row_tiles(T, n_heads, cache.n_kv_heads, cache.head_dim, S);
    const bool f8 = cache.k_scale != nullptr;
    switch (cache.head_dim) {
        case 64: return f8 ? launch_mt<64, 1>(a, mt, st) : launch_mt<64, 0>(a, mt, st);
        case 128: return f8 ? launch_mt<128, 1>(a, mt, st) : launch_mt<128, 0>(a, mt, st);
        case 256: return f8 ? launch_mt<256, 1>(a, mt, st) : launch_mt<256, 0>(a, mt, st);
    }
    return hipErrorInvalidValue;
}
