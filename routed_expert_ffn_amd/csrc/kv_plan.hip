// kv_plan.hip -- page tables, slots and positions of one step, from the
// requests' lengths (gfx950).
//
// With m_s the admissible new tokens of request s: q_offsets = min(T, exclusive
// sum of m), n_s its differences, take_s the pages that n_s tokens add, and the
// pages handed out in request order at the exclusive sum of take.  Two scans
// over S <= 4096 requests, then one independent lookup per row and per new page.
//
// Latency-bound (a step of 64 requests reads and writes 4 KB), so it is one
// launch: every block redoes both scans in LDS (each thread owns EPT
// consecutive requests) and then takes its share of rows and pages, finding a
// row's request by binary search.  64 requests of 5 tokens 3.8 us of kernel time, 1024
// ragged ones 5.6 us (a call, 6.5 and 6.7, is the host's launch): two scans of 6 lane
// moves, two barriers and two dependent loads for a row.  One scan kernel and a second
// launch for the rows would pay another launch, 2 us and more, to save each block the scans.
#include "attn.h"
#include "common.h"

namespace {

constexpr int PLAN_THREADS = 256;

// exclusive sum over the block of one value per thread; total in every thread
template <typename V>
MOE_DEV V block_excl_scan(V v, V* wave_tot, V& total) {
    const int l = lane_id(), w = threadIdx.x / WAVE;
    V incl = v;
#pragma unroll
    for (int d = 1; d < WAVE; d <<= 1) {
        const V o = __shfl_up(incl, d, WAVE);
        if (l >= d) incl += o;
    }
    if (l == WAVE - 1) wave_tot[w] = incl;
    __syncthreads();
    V base = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < PLAN_THREADS / WAVE; i++) {
        const V t = wave_tot[i];
        if (i < w) base += t;
        total += t;
    }
    return base + incl - v;
}

// the largest s < S with start[s] <= i (empty requests share a start with their successor)
MOE_DEV int owner(const int* start, int S, int i) {
    int lo = 0, hi = S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <int EPT>
__global__ __launch_bounds__(PLAN_THREADS) void k_kv_plan(const int32_t* __restrict__ cached_len,
                                                          const int32_t* __restrict__ new_len, int S,
                                                          const int32_t* __restrict__ free_pages, int n_free,
                                                          int page_shift, int T, int32_t* __restrict__ table, int W,
                                                          int32_t* __restrict__ q_offsets, int32_t* __restrict__ kv_len,
                                                          int32_t* __restrict__ positions, int32_t* __restrict__ slots,
                                                          int32_t* __restrict__ counts) {
    __shared__ int64_t tot64[PLAN_THREADS / WAVE];
    __shared__ int tot32[PLAN_THREADS / WAVE];
    __shared__ int qo[PLAN_THREADS * EPT + 1], first[PLAN_THREADS * EPT], cached[PLAN_THREADS * EPT];
    const int s0 = threadIdx.x * EPT;
    const int64_t cap = (int64_t)W << page_shift;
    const int ps1 = (1 << page_shift) - 1;
    int c[EPT];
    int64_t m[EPT], sum = 0;
#pragma unroll
    for (int i = 0; i < EPT; i++) {
        const int s = min(s0 + i, S - 1);
        c[i] = (int)min((int64_t)max(cached_len[s], 0), cap);
        m[i] = s0 + i < S ? min((int64_t)max(new_len[s], 0), cap - c[i]) : 0;
        sum += m[i];
    }
    int64_t all;
    int64_t at = block_excl_scan(sum, tot64, all);
    int n[EPT], o[EPT], take[EPT], tsum = 0;
#pragma unroll
    for (int i = 0; i < EPT; i++) {
        o[i] = (int)min(at, (int64_t)T);
        at += m[i];
        n[i] = (int)min(at, (int64_t)T) - o[i];
        take[i] = (int)((((int64_t)c[i] + n[i] + ps1) >> page_shift) - (((int64_t)c[i] + ps1) >> page_shift));
        tsum += take[i];
    }
    int pages;
    int pf = block_excl_scan(tsum, tot32, pages);
    const int rows = (int)min(all, (int64_t)T);
#pragma unroll
    for (int i = 0; i < EPT; i++) {
        if (s0 + i < S) {
            qo[s0 + i] = o[i];
            first[s0 + i] = pf;
            cached[s0 + i] = c[i];
            if (blockIdx.x == 0) {
                q_offsets[s0 + i] = o[i];
                kv_len[s0 + i] = c[i] + n[i];
            }
        }
        pf += take[i];
    }
    if (threadIdx.x == 0) {
        qo[S] = rows;
        if (blockIdx.x == 0) {
            q_offsets[S] = rows;
            counts[0] = rows;
            counts[1] = pages;
        }
    }
    __syncthreads();
    const int gid = blockIdx.x * PLAN_THREADS + threadIdx.x, step = gridDim.x * PLAN_THREADS;
    for (int t = gid; t < T; t += step) {
        int pos = 0, slot = -1;
        if (t < rows) {
            const int s = owner(qo, S, t);
            pos = cached[s] + (t - qo[s]);
            const int idx = pos >> page_shift, have = (int)(((int64_t)cached[s] + ps1) >> page_shift);
            int page = -1;
            if (idx < have) {
                page = table[(int64_t)s * W + idx];            // a page that is there: no block writes it
            } else {
                const int f = first[s] + (idx - have);
                if (f < n_free) page = free_pages[f];
            }
            // (an entry too large for an int32 slot is no page of any cache)
            if (page >= 0 && page <= (0x7fffffff >> page_shift)) slot = (page << page_shift) | (pos & ps1);
        }
        positions[t] = pos;
        slots[t] = slot;
    }
    for (int j = gid; j < pages; j += step) {
        const int s = owner(first, S, j);
        const int have = (int)(((int64_t)cached[s] + ps1) >> page_shift);
        table[(int64_t)s * W + have + (j - first[s])] = j < n_free ? free_pages[j] : -1;
    }
}

}  // namespace

hipError_t launch_kv_plan(const int32_t* cached_len, const int32_t* new_len, int S, const int32_t* free_pages,
                          int n_free, int page_shift, int T, int32_t* table, int W, int32_t* q_offsets,
                          int32_t* kv_len, int32_t* positions, int32_t* slots, int32_t* counts, hipStream_t st) {
    // one row per thread up to 128 blocks; the pages (at most T + S) follow in the same threads
    const int64_t n = T > S ? T : S;
    const int grid = (int)(n <= PLAN_THREADS ? 1 : n >= 128 * PLAN_THREADS ? 128 : (n + PLAN_THREADS - 1) / PLAN_THREADS);
    const int ept = (S + PLAN_THREADS - 1) / PLAN_THREADS;
    auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3(grid), dim3(PLAN_THREADS), 0, st, cached_len, new_len, S, free_pages, n_free,
                           page_shift, T, table, W, q_offsets, kv_len, positions, slots, counts);
    };
    if (ept <= 1) go(k_kv_plan<1>);
    else if (ept <= 4) go(k_kv_plan<4>);
    else go(k_kv_plan<16>);
    return hipGetLastError();
}
