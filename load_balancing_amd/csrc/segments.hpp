// segments.hpp -- the plan's segments as row tiles, for the grouped products.
//
// Segment s < E: home expert s (rows home_row_off[s] .. + keep[s] of rank
// s div L); s >= E: replica s - E.  Tiles of BM rows never cross a segment, so
// every tile multiplies by one expert's weights.  n_rep is known only on the
// device: every workgroup scans the segments' tile counts into LDS.
#pragma once

#include "moonep_internal.hpp"

namespace moonep {

struct SegTables {
    const int32_t *plan;
    PlanLayout pl;
    const int32_t *wslot;
    int32_t R, E, L, C, nslots;

    // A word of the tables at a uniform address: a scalar load, which does not
    // wait for the vector loads in flight.  The tables are not written by the
    // kernels that read them.
    __device__ static __forceinline__ int32_t word(const int32_t *p)
    {
        return *(const __attribute__((address_space(4))) int32_t *)(uintptr_t)p;
    }

    __device__ __forceinline__ int32_t n_rep() const
    {
        const int32_t n = plan[pl.header + MOONEP_PLAN_H_N_REP];
        return n < 0 ? 0 : (n < pl.cap ? n : pl.cap);
    }

    // Rows of segment s.  A bad table entry makes an empty segment, so every
    // access through it stays in bounds.
    __device__ __forceinline__ int32_t rows(int32_t s) const
    {
        if (s < E) {
            const int32_t off = plan[pl.home_row_off + s], n = plan[pl.keep + s];
            return (off >= 0 && n >= 0 && off <= C - n) ? n : 0;
        }
        const int32_t j = s - E;
        const int32_t h = plan[pl.rep_host + j], e = plan[pl.rep_expert + j];
        const int32_t off = plan[pl.rep_row_off + j], n = plan[pl.rep_count + j];
        return (h >= 0 && h < R && e >= 0 && e < E && off >= 0 && n >= 0 && off <= C - n) ? n : 0;
    }

    // First buffer row of a segment that has rows.  s is uniform.
    __device__ __forceinline__ int64_t first_row(int32_t s) const
    {
        s = __builtin_amdgcn_readfirstlane(s);
        if (s < E)
            return (int64_t)(s / L) * C + word(plan + pl.home_row_off + s);
        return (int64_t)word(plan + pl.rep_host + s - E) * C + word(plan + pl.rep_row_off + s - E);
    }

    // First buffer row of a segment that has rows, its row count, and its weight
    // row: of the pool if *pooled, else of the home weights.  s is uniform.
    __device__ __forceinline__ int64_t segment(int32_t s, int32_t *n, int64_t *weight_row,
                                               bool *pooled) const
    {
        s = __builtin_amdgcn_readfirstlane(s);
        *pooled = false;
        if (s < E) {
            *weight_row = s;
            *n = word(plan + pl.keep + s);
            return (int64_t)(s / L) * C + word(plan + pl.home_row_off + s);
        }
        const int32_t j = s - E, ws = word(wslot + j);
        *pooled = ws >= 0 && ws < nslots;
        *weight_row = *pooled ? ws : word(plan + pl.rep_expert + j);
        *n = word(plan + pl.rep_count + j);
        return (int64_t)word(plan + pl.rep_host + j) * C + word(plan + pl.rep_row_off + j);
    }
};

inline SegTables seg_tables(const moonep_shape &s, const int32_t *plan, const int32_t *wslot, int32_t B)
{
    SegTables t{};
    t.plan = plan;
    t.pl = plan_layout(s.E, s.R);
    t.wslot = wslot;
    t.R = s.R;
    t.E = s.E;
    t.L = s.E / s.R;
    t.C = s.S * s.K;
    t.nslots = s.R * B;
    return t;
}

// Exclusive scan of one int per thread over a block of NW waves.
template <int NW>
__device__ __forceinline__ int block_scan_excl(int v, int *tmp, int *total)
{
    const int lane = lane_id(), wid = (int)threadIdx.x >> 6;
    int incl = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d, 64);
        if (lane >= d)
            incl += o;
    }
    if (lane == 63)
        tmp[wid] = incl;
    __syncthreads();
    int base = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const int t = tmp[w];
        base += w < wid ? t : 0;
        sum += t;
    }
    __syncthreads();
    *total = sum;
    return base + incl - v;
}

// First tile of every segment into seg_start [nseg + 1] (LDS); returns the
// number of tiles.  tmp: NW ints of LDS.
template <int BM, int NW>
__device__ __forceinline__ int32_t scan_tiles(const SegTables &t, int32_t nseg, int32_t *seg_start,
                                              int *tmp)
{
    const int32_t per = (nseg + NW * 64 - 1) / (NW * 64);
    const int32_t s0 = (int32_t)threadIdx.x * per;
    int32_t mine = 0;
    for (int32_t s = s0; s < s0 + per && s < nseg; ++s)
        mine += (t.rows(s) + BM - 1) / BM;
    int32_t total = 0;
    int32_t run = block_scan_excl<NW>(mine, tmp, &total);
    for (int32_t s = s0; s < s0 + per && s < nseg; ++s) {
        seg_start[s] = run;
        run += (t.rows(s) + BM - 1) / BM;
    }
    if (threadIdx.x == 0)
        seg_start[nseg] = total;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(total);  // the same in every lane
}

// Segment that holds tile t: the last s with seg_start[s] <= t, for nseg <=
// 4096 and every lane of the wave active (uniform).  Two rounds of 64
// comparisons at once: every step-th segment, then the step after the last of
// those.
__device__ __forceinline__ int32_t find_segment(const int32_t *seg_start, int32_t nseg, int32_t t)
{
    const int lane = lane_id();
    const int32_t step = (nseg + 63) / 64;
    const int32_t c = lane * step;
    const int32_t s0 = (__popcll(ballot(c < nseg && seg_start[c < nseg ? c : 0] <= t)) - 1) * step;
    const int32_t d = s0 + lane;
    return s0 + __popcll(ballot(lane < step && d < nseg && seg_start[d < nseg ? d : 0] <= t)) - 1;
}

// Position of workgroup b among all of them when each XCD (workgroup b runs on
// XCD b % 8) takes a run of consecutive items per round of P items.
__device__ __forceinline__ int xcd_slot(int b, int P)
{
    const int xcd = b % 8;
    int slot = b / 8;
    for (int x = 0; x < xcd; ++x)
        slot += (P - x + 7) / 8;
    return slot;
}

// Item -> (row tile, column block): groups of GM row tiles, the row tile
// running fastest inside a group (fewer in the last one).
template <int GM, class Item>
__device__ __forceinline__ void item_of(Item it, int32_t tiles, int32_t nbn, int32_t *t, int32_t *nb)
{
    const Item gi = it / ((Item)GM * nbn);
    const int32_t within = (int32_t)(it - gi * ((Item)GM * nbn));
    const int32_t gleft = tiles - (int32_t)gi * GM;
    const int32_t gm = gleft < GM ? gleft : GM;
    *t = (int32_t)gi * GM + within % gm;
    *nb = within / gm;
}

}  // namespace moonep
