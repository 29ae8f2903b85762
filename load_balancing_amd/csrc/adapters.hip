// adapters.hip -- low-rank adapters of many requests at once, beside a
// projection that all rows share, and their gradients.
//
// Row r with adapter m = ids[r] (none if m is outside [0, n)), matrices A_m
// [rank, in] and B_m [out, rank], scale s_m:
//   u[r]  = x[r] A_m^T                       y[r]  = base[r] + s_m u[r] B_m^T
//   du[r] = s_m dy[r] B_m                    dx[r] = base[r] + du[r] A_m
//   dA_m  = sum of du[r]^T x[r]              dB_m  = sum of s_m dy[r]^T u[r]
//
// All of it is bound by memory: 4 rank operations or fewer for each element of
// x, dy, base and y, which are read or written once (dy twice in the backward).
// Three kernels, each in the two orders of its matrix:
//   shrink  rows [D] against a matrix, to rank values in fp32 (u, du);
//   expand  rank values against a matrix, added to base rows (y, dx);
//   wgrad   rank values against rows [D], summed over an adapter's rows.
// They use the 16 x 16 x 32 bf16 matrix instruction with operands loaded
// straight into registers, without LDS: the rows of a 16-position tile are the
// instruction's columns, so that every lane holds one row's results, and a tile
// whose rows have several adapters is run once for each of them, each lane
// keeping the results of its own row's adapter (what another adapter's matrix
// holds, NaN or infinity, cannot reach it).  Positions are taken in `order`,
// where rows of one adapter stand together, or as they are.
//
// Lane layout of the instruction (m, n: 16; k: 32): operand A lane l holds row
// m = l % 16, k = 8 (l / 16) .. + 7; operand B lane l column n = l % 16, same k;
// the result's lane l holds column l % 16, rows 4 (l / 16) .. + 3.  The 16 rows
// of tile t of T stand for indexes m T + t, so that a lane's results over T
// tiles are 4 T consecutive indexes.
//
// Rounding: u and du stay in fp32.  Where they enter a product they are split
// into bf16 parts whose products the instruction sums in fp32: two parts (16
// bits) in expand, whose result is rounded to bf16; three (24 bits, all of it)
// in wgrad, whose result is fp32.
#include "segments.hpp"

namespace moonep {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

namespace {

constexpr int kAdBlock = 256;  // four waves
constexpr int kMostSplits = 16;
constexpr int kMostChunks = 64;
constexpr int32_t kSplitRows = 2048;  // up to here a tile's contraction is split

union Frag {
    uint16_t h[8];
    uint32_t w[4];
    bf16x8 v;
};

template <int N>
struct Halves {  // N bf16 values loaded as one
    uint16_t h[N];
};
template <int N>
__device__ __forceinline__ Halves<N> load_halves(const uint16_t *p)
{
    Halves<N> v;
    __builtin_memcpy(&v, __builtin_assume_aligned(p, 2 * N), 2 * N);
    return v;
}

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Rows in the order they are worked on, and their adapters.
struct AdRows {
    const int32_t *ids, *order;
    int32_t rows, n;

    __device__ __forceinline__ int32_t row(int64_t p) const
    {
        if (p >= rows)
            return -1;
        const int32_t r = order ? order[p] : (int32_t)p;
        return (uint32_t)r < (uint32_t)rows ? r : -1;
    }
    __device__ __forceinline__ int32_t id(int32_t r) const
    {
        if (r < 0)
            return -1;
        const int32_t i = ids[r];
        return (uint32_t)i < (uint32_t)n ? i : -1;
    }
};

// The matrices of the bank that one kernel multiplies by.
struct AdMats {
    const uint16_t *first;  // adapter 0's
    int64_t stride;
    int32_t rank, D;  // rank x D (contiguous D), or D x rank (contiguous rank)
};

// ---------------------------------------------------------------------------
// shrink
// ---------------------------------------------------------------------------

struct ShrinkArgs {
    AdRows r;
    AdMats w;
    const uint16_t *x;
    const float *scale;  // per adapter, or NULL for 1
    float *out;          // [splits][rows][rank]
};

// T tiles of 16 of the rank; kNN: the matrix is [D][rank]; RT row tiles a wave.
// kSplit: the four waves share a row tile, each a part of the contraction, of
// which blockIdx.y is one of gridDim.y parts; their sums are joined in LDS.
template <int T, bool kNN, int RT, bool kSplit>
__global__ __launch_bounds__(kAdBlock) void shrink_kernel(ShrinkArgs a)
{
    constexpr int U = T * (kNN ? 2 : 1) + RT <= 4 ? 4 : (T <= 4 ? 2 : 1);  // steps in flight
    const int lane = lane_id(), wave = (int)threadIdx.x >> 6;
    const int m = lane & 15, g = lane >> 4;
    const int32_t D = a.w.D, rank = a.w.rank;
    const int64_t p0 = kSplit ? (int64_t)blockIdx.x * 16 : ((int64_t)blockIdx.x * 4 + wave) * 16 * RT;
    const int32_t steps = (D + 31) / 32;
    int32_t k0 = 0, k1 = steps;
    if (kSplit) {
        const int32_t parts = (int32_t)gridDim.y * 4, part = (int32_t)blockIdx.y * 4 + wave;
        k0 = (int32_t)((int64_t)steps * part / parts);
        k1 = (int32_t)((int64_t)steps * (part + 1) / parts);
    } else if (p0 >= a.r.rows) {
        return;
    }
    const int32_t full = k1 < D / 32 ? k1 : D / 32;  // steps before this have all 32

    int32_t row[RT], id[RT];
    const uint16_t *xp[RT];
    uint64_t todo[RT];
    f32x4 res[RT][T];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        row[i] = a.r.row(p0 + i * 16 + m);
        id[i] = a.r.id(row[i]);
        xp[i] = a.x + (int64_t)(row[i] < 0 ? 0 : row[i]) * D + g * 8;
        todo[i] = ballot(id[i] >= 0);
#pragma unroll
        for (int t = 0; t < T; ++t)
            res[i][t] = f32x4{0, 0, 0, 0};
    }
    const int32_t r0 = m * T < rank ? m * T : 0;  // lanes past the rank repeat index 0: not stored

    for (;;) {
        int32_t cur = -1;
#pragma unroll
        for (int i = 0; i < RT; ++i)
            if (cur < 0 && todo[i])
                cur = __builtin_amdgcn_readlane(id[i], __builtin_ctzll(todo[i]));
        if (cur < 0)
            break;
        const uint16_t *w = a.w.first + cur * a.w.stride;
        w += kNN ? (int64_t)g * 8 * rank + r0 : (int64_t)r0 * D + g * 8;
        auto load_w = [&](int32_t k, bool in, Frag (&f)[T]) {
            if constexpr (kNN) {
                Halves<T> v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = load_halves<T>(w + (int64_t)((in ? k * 32 : 0) + j) * rank);
#pragma unroll
                for (int t = 0; t < T; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        f[t].w[j] = (uint32_t)v[2 * j].h[t] | (uint32_t)v[2 * j + 1].h[t] << 16;
            } else {
#pragma unroll
                for (int t = 0; t < T; ++t)
                    f[t].v = *(const bf16x8 *)(w + (int64_t)t * D + (in ? k * 32 : 0));
            }
        };
        f32x4 acc[RT][T];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int t = 0; t < T; ++t)
                acc[i][t] = f32x4{0, 0, 0, 0};
        int32_t k = k0;
        for (; k + U <= full; k += U) {
            Frag x[U][RT], f[U][T];
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    x[u][i].v = *(const bf16x8 *)(xp[i] + (k + u) * 32);
                load_w(k + u, true, f[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int t = 0; t < T; ++t)
                        acc[i][t] = mfma16(f[u][t].v, x[u][i].v, acc[i][t]);
        }
        for (; k < k1; ++k) {
            // the last step may end inside: chunks past D are zeros in both operands
            const bool in = k * 32 + g * 8 < D;
            Frag x[RT], f[T];
#pragma unroll
            for (int i = 0; i < RT; ++i)
                x[i].v = *(const bf16x8 *)(in ? xp[i] + k * 32 : xp[i] - g * 8);
            if (in) {
                load_w(k, true, f);
            } else {
#pragma unroll
                for (int t = 0; t < T; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        f[t].w[j] = 0;
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[i].w[j] = 0;
            }
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int t = 0; t < T; ++t)
                    acc[i][t] = mfma16(f[t].v, x[i].v, acc[i][t]);
        }
        const float s = a.scale ? a.scale[cur] : 1.0f;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const bool mine = id[i] == cur;
            todo[i] &= ~ballot(mine);
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    res[i][t][j] = mine ? acc[i][t][j] * s : res[i][t][j];
        }
    }

    float *out = a.out + (kSplit ? (int64_t)blockIdx.y * a.r.rows * rank : 0);
    if constexpr (kSplit) {
        __shared__ f32x4 join[4][T][64];
#pragma unroll
        for (int t = 0; t < T; ++t)
            join[wave][t][lane] = res[0][t];
        __syncthreads();
        if (wave)
            return;
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int v = 1; v < 4; ++v)
                res[0][t] += join[v][t][lane];
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        if (row[i] < 0)
            continue;
        float v[4 * T];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int t = 0; t < T; ++t)
                v[j * T + t] = res[i][t][j];
        float *o = out + (int64_t)row[i] * rank + g * 4 * T;
#pragma unroll
        for (int q = 0; q < T; ++q)
            if (g * 4 * T + q * 4 < rank)
                *(f32x4 *)(o + q * 4) = f32x4{v[q * 4], v[q * 4 + 1], v[q * 4 + 2], v[q * 4 + 3]};
    }
}

// ---------------------------------------------------------------------------
// expand
// ---------------------------------------------------------------------------

struct ExpandArgs {
    AdRows r;
    AdMats w;
    const float *u;      // [parts][rows][rank]
    float *u_out;        // their sum, or NULL
    const float *scale;  // per adapter, or NULL for 1
    const uint16_t *base;
    uint16_t *y;
    int32_t parts, tiles;  // row tiles a workgroup
};

// The contraction is over 2 rank: both bf16 parts of u in turn, 8 of a part in
// one 8-value chunk, KS steps of four chunks; chunks past it are zeros.  A wave
// has 16 CT columns, column m CT + t in row m of tile t, and walks row tiles.
template <int KS, int CT, bool kNN>
__global__ __launch_bounds__(kAdBlock) void expand_kernel(ExpandArgs a)
{
    const int lane = lane_id(), wave = (int)threadIdx.x >> 6;
    const int m = lane & 15, g = lane >> 4;
    const int32_t D = a.w.D, rank = a.w.rank, rc = rank / 8;
    const int32_t c0 = ((int32_t)blockIdx.x * 4 + wave) * 16 * CT;
    if (c0 >= D)
        return;
    const int32_t wc = c0 + m * CT < D ? c0 + m * CT : 0;  // lanes past D repeat column 0: not stored
    const int32_t oc = c0 + g * 4 * CT;                    // this lane's output columns
    int chunk[KS];
    bool low[KS], in[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const int c = s * 4 + g;
        in[s] = c < 2 * rc;
        low[s] = c >= rc;
        chunk[s] = in[s] ? (low[s] ? c - rc : c) * 8 : 0;
    }

    Frag wf[KS][CT];
    int32_t have = -1;
    const int64_t first = (int64_t)blockIdx.y * a.tiles * 16;
    for (int32_t tile = 0; tile < a.tiles; ++tile) {
        const int64_t p0 = first + tile * 16;
        if (p0 >= a.r.rows)
            break;
        const int32_t row = a.r.row(p0 + m), id = a.r.id(row);
        const bool mine_io = row >= 0 && (id >= 0 || a.y != a.base);
        u32x4 b[CT / 2];
#pragma unroll
        for (int q = 0; q < CT / 2; ++q)
            b[q] = mine_io && oc + q * 8 < D ? *(const u32x4 *)(a.base + (int64_t)row * D + oc + q * 8)
                                             : u32x4{0, 0, 0, 0};
        Frag uf[KS];
        const float s = a.scale ? (id >= 0 ? a.scale[id] : 0.0f) : 1.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            f32x4 v0 = {0, 0, 0, 0}, v1 = {0, 0, 0, 0};
            if (row >= 0 && in[k]) {
                const float *u = a.u + (int64_t)row * rank + chunk[k];
                v0 = *(const f32x4 *)u;
                v1 = *(const f32x4 *)(u + 4);
                for (int32_t q = 1; q < a.parts; ++q) {
                    u += (int64_t)a.r.rows * rank;
                    v0 += *(const f32x4 *)u;
                    v1 += *(const f32x4 *)(u + 4);
                }
                if (a.u_out && c0 == 0 && !low[k]) {
                    float *o = a.u_out + (int64_t)row * rank + chunk[k];
                    *(f32x4 *)o = v0;
                    *(f32x4 *)(o + 4) = v1;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e0 = (j < 2 ? v0[2 * j] : v1[2 * j - 4]) * s;
                const float e1 = (j < 2 ? v0[2 * j + 1] : v1[2 * j - 3]) * s;
                const uint32_t hi = pack_bf16(e0, e1);
                const float h0 = bf16_lo(hi), h1 = bf16_hi(hi);
                // of an infinity the second part is 0
                const float l0 = __builtin_isfinite(h0) ? e0 - h0 : 0.0f;
                const float l1 = __builtin_isfinite(h1) ? e1 - h1 : 0.0f;
                uf[k].w[j] = low[k] ? pack_bf16(l0, l1) : hi;
            }
        }
        f32x4 res[CT];
#pragma unroll
        for (int t = 0; t < CT; ++t)
            res[t] = f32x4{0, 0, 0, 0};
        uint64_t todo = ballot(id >= 0);
        while (todo) {
            const int32_t cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
            if (cur != have) {
                have = cur;
                const uint16_t *w = a.w.first + cur * a.w.stride;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    if constexpr (kNN) {
                        Halves<CT> v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            v[j] = load_halves<CT>(w + (int64_t)(chunk[k] + j) * D + wc);
#pragma unroll
                        for (int t = 0; t < CT; ++t)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                wf[k][t].w[j] = (uint32_t)v[2 * j].h[t] | (uint32_t)v[2 * j + 1].h[t] << 16;
                    } else {
#pragma unroll
                        for (int t = 0; t < CT; ++t)
                            wf[k][t].v = *(const bf16x8 *)(w + (int64_t)(wc + t) * rank + chunk[k]);
                    }
                    if (!in[k]) {
#pragma unroll
                        for (int t = 0; t < CT; ++t)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                wf[k][t].w[j] = 0;
                    }
                }
            }
            const bool mine = id == cur;
            todo &= ~ballot(mine);
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                f32x4 acc = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    acc = mfma16(wf[k][t].v, uf[k].v, acc);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    res[t][j] = mine ? acc[j] : res[t][j];
            }
        }
        if (mine_io) {
            float v[4 * CT];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int t = 0; t < CT; ++t)
                    v[j * CT + t] = res[t][j];
#pragma unroll
            for (int q = 0; q < CT / 2; ++q) {
                if (oc + q * 8 >= D)
                    continue;
                u32x4 o;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[j] = pack_bf16(bf16_lo(b[q][j]) + v[q * 8 + 2 * j], bf16_hi(b[q][j]) + v[q * 8 + 2 * j + 1]);
                // a row without an adapter is copied bit for bit
                *(u32x4 *)(a.y + (int64_t)row * D + oc + q * 8) = id >= 0 ? o : b[q];
            }
        }
    }
}

// ---------------------------------------------------------------------------
// wgrad
// ---------------------------------------------------------------------------

struct WgradArgs {
    AdRows r;  // order: the plan's
    const int32_t *off, *keep;
    int32_t rank, in_dim, out_dim, chunk, nchunks, blocks_a, accumulate;
    int64_t stride, a_off, b_off;
    const float *du, *u, *scale;
    const uint16_t *x, *dy;
    float *part;  // [nchunks + n][rank * (in_dim + out_dim)]
    float *d_bank;
};

// Rows of adapter e: positions [off, off + keep) of the plan, none if the table
// is not one.
__device__ __forceinline__ int32_t adapter_rows(const int32_t *off, const int32_t *keep, int32_t e,
                                                int32_t rows, int32_t *first)
{
    const int32_t o = off[e], n = keep[e];
    *first = o;
    return o >= 0 && n >= 0 && o <= rows - n ? n : 0;
}

// The three bf16 parts of a value pair, packed.
__device__ __forceinline__ void split3(float a, float b, uint32_t *p0, uint32_t *p1, uint32_t *p2)
{
    const uint32_t hi = pack_bf16(a, b);
    const float h0 = bf16_lo(hi), h1 = bf16_hi(hi);
    const float r0 = __builtin_isfinite(h0) ? a - h0 : 0.0f;
    const float r1 = __builtin_isfinite(h1) ? b - h1 : 0.0f;
    const uint32_t mid = pack_bf16(r0, r1);
    *p0 = hi;
    *p1 = mid;
    *p2 = pack_bf16(r0 - bf16_lo(mid), r1 - bf16_hi(mid));
}

// T tiles of 16 of the rank against 16 CT columns a wave.  blockIdx.x: columns
// of x (dA), then of dy (dB); blockIdx.y: a chunk of positions.  The sums of an
// adapter whose rows lie in one chunk go to their place, those of a longer one
// to a slot of the workspace: chunk + adapter, which no two pieces share, since
// from one piece to the next the chunk or the adapter grows and neither falls.
template <int T, int CT>
__global__ __launch_bounds__(kAdBlock) void wgrad_kernel(WgradArgs a)
{
    const int lane = lane_id(), wave = (int)threadIdx.x >> 6;
    const int n = lane & 15, g = lane >> 4;
    const bool is_a = (int32_t)blockIdx.x < a.blocks_a;
    const int32_t D = is_a ? a.in_dim : a.out_dim, rank = a.rank, rows = a.r.rows;
    const int32_t c0 = (((int32_t)blockIdx.x - (is_a ? 0 : a.blocks_a)) * 4 + wave) * 16 * CT;
    if (c0 >= D)
        return;
    const int32_t col = c0 + n * CT;
    const uint16_t *qp = (is_a ? a.x : a.dy) + (col < D ? col : 0);
    const int32_t r0 = n * T < rank ? n * T : 0;
    const float *pp = (is_a ? a.du : a.u) + r0;
    const int64_t window = (int64_t)rank * (a.in_dim + a.out_dim);
    int32_t p = (int32_t)blockIdx.y * a.chunk;
    const int32_t p_end = rows - p < a.chunk ? rows : p + a.chunk;

    while (p < p_end) {
        int32_t row = a.r.order[p];
        if ((uint32_t)row >= (uint32_t)rows)
            return;
        const int32_t e = __builtin_amdgcn_readfirstlane(a.r.ids[row]);
        if ((uint32_t)e >= (uint32_t)a.r.n)
            return;  // the rows without an adapter come last
        int32_t first;
        const int32_t cnt = adapter_rows(a.off, a.keep, e, rows, &first);
        if (p < first || p >= first + cnt)
            return;  // not this order's plan
        const int32_t end = first + cnt < p_end ? first + cnt : p_end;
        const float s = is_a ? 1.0f : a.scale[e];

        f32x4 acc[T][CT];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int c = 0; c < CT; ++c)
                acc[t][c] = f32x4{0, 0, 0, 0};

        auto step = [&](int32_t at, bool whole) {
            Halves<CT> q[8];
            float v[8][T];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int32_t pos = at + g * 8 + j;
                const bool in = whole || pos < end;
                int32_t r = a.r.order[in ? pos : at];
                r = (uint32_t)r < (uint32_t)rows ? r : 0;
                q[j] = load_halves<CT>(qp + (int64_t)r * D);
                __builtin_memcpy(v[j], __builtin_assume_aligned(pp + (int64_t)r * rank, T < 4 ? 4 * T : 16), 4 * T);
                if (!in) {
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        q[j].h[c] = 0;
#pragma unroll
                    for (int t = 0; t < T; ++t)
                        v[j][t] = 0.0f;
                }
            }
            Frag qf[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    qf[c].w[j] = (uint32_t)q[2 * j].h[c] | (uint32_t)q[2 * j + 1].h[c] << 16;
#pragma unroll
            for (int t = 0; t < T; ++t) {
                Frag f0, f1, f2;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    split3(v[2 * j][t] * s, v[2 * j + 1][t] * s, &f0.w[j], &f1.w[j], &f2.w[j]);
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    acc[t][c] = mfma16(f0.v, qf[c].v, acc[t][c]);
                    acc[t][c] = mfma16(f1.v, qf[c].v, acc[t][c]);
                    acc[t][c] = mfma16(f2.v, qf[c].v, acc[t][c]);
                }
            }
        };
        int32_t at = p;
        for (; at + 32 <= end; at += 32)
            step(at, true);
        if (at < end)
            step(at, false);

        const int32_t ch = (int32_t)blockIdx.y;
        const bool direct = first / a.chunk == (first + cnt - 1) / a.chunk;
        const bool add = direct && a.accumulate;
        float *o = direct ? a.d_bank + e * a.stride + (is_a ? a.a_off : a.b_off)
                          : a.part + (ch + e) * window + (is_a ? 0 : (int64_t)rank * a.in_dim);
        if (col < D) {
            if (is_a) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int t = 0; t < T; ++t) {
                        const int32_t r = (g * 4 + i) * T + t;
                        if (r >= rank)
                            continue;
                        float *z = o + (int64_t)r * D + col;
#pragma unroll
                        for (int c = 0; c < CT; c += 4) {
                            f32x4 val = {acc[t][c][i], acc[t][c + 1][i], acc[t][c + 2][i], acc[t][c + 3][i]};
                            if (add)
                                val += *(const f32x4 *)(z + c);
                            *(f32x4 *)(z + c) = val;
                        }
                    }
            } else {
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    float v[4 * T];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int t = 0; t < T; ++t)
                            v[i * T + t] = acc[t][c][i];
                    float *z = o + (int64_t)(col + c) * rank + g * 4 * T;
#pragma unroll
                    for (int q = 0; q < T; ++q) {
                        if (g * 4 * T + q * 4 >= rank)
                            continue;
                        f32x4 val = {v[q * 4], v[q * 4 + 1], v[q * 4 + 2], v[q * 4 + 3]};
                        if (add)
                            val += *(const f32x4 *)(z + q * 4);
                        *(f32x4 *)(z + q * 4) = val;
                    }
                }
            }
        }
        p = end;
    }
}

// Adapters without rows get zeros, and the pieces of those in several chunks
// are summed, in the order of the chunks.
__global__ __launch_bounds__(kAdBlock) void wgrad_join_kernel(WgradArgs a)
{
    const int32_t e = (int32_t)blockIdx.y;
    int32_t first;
    const int32_t cnt = adapter_rows(a.off, a.keep, e, a.r.rows, &first);
    const int32_t ch0 = cnt ? first / a.chunk : 0, ch1 = cnt ? (first + cnt - 1) / a.chunk : 0;
    if (cnt ? ch0 == ch1 : a.accumulate)
        return;
    const int64_t na = (int64_t)a.rank * a.in_dim, window = na + (int64_t)a.rank * a.out_dim;
    for (int64_t i = ((int64_t)blockIdx.x * kAdBlock + threadIdx.x) * 4; i < window;
         i += (int64_t)gridDim.x * kAdBlock * 4) {
        float *o = a.d_bank + e * a.stride + (i < na ? a.a_off + i : a.b_off + i - na);
        f32x4 v = {0, 0, 0, 0};
        if (cnt) {
            const float *src = a.part + (ch0 + e) * window + i;
            for (int32_t c = ch0; c <= ch1; ++c, src += window)
                v += *(const f32x4 *)src;
            if (a.accumulate)
                v += *(const f32x4 *)o;
        }
        *(f32x4 *)o = v;
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

int status() { return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_ERR_HIP; }

int split_count(int32_t rows, int32_t D)
{
    if (rows > kSplitRows)
        return 1;
    const int32_t tiles = (rows + 15) / 16, steps = (D + 31) / 32;
    int32_t s = 512 / tiles;
    s = s < kMostSplits ? s : kMostSplits;
    s = s < (steps + 3) / 4 ? s : (steps + 3) / 4;
    return s < 1 ? 1 : s;
}

template <int T, bool kNN>
void shrink_as(const ShrinkArgs &a, int splits, hipStream_t st)
{
    const int32_t rows = a.r.rows;
    if (rows <= kSplitRows)
        hipLaunchKernelGGL((shrink_kernel<T, kNN, 1, true>), dim3((rows + 15) / 16, splits),
                           dim3(kAdBlock), 0, st, a);
    else
        hipLaunchKernelGGL((shrink_kernel<T, kNN, 2, false>), dim3((rows + 127) / 128),
                           dim3(kAdBlock), 0, st, a);
}

template <bool kNN>
void shrink(const ShrinkArgs &a, int splits, hipStream_t st)
{
    if (a.w.rank <= 16)
        shrink_as<1, kNN>(a, splits, st);
    else if (a.w.rank <= 32)
        shrink_as<2, kNN>(a, splits, st);
    else if (a.w.rank <= 64)
        shrink_as<4, kNN>(a, splits, st);
    else
        shrink_as<8, kNN>(a, splits, st);
}

template <int KS, int CT, bool kNN>
void expand_as(ExpandArgs a, hipStream_t st)
{
    const int64_t tiles = ((int64_t)a.r.rows + 15) / 16, blocks = (a.w.D + 64 * CT - 1) / (64 * CT);
    int64_t per = tiles * blocks / 1024;
    per = per < 1 ? 1 : (per > 16 ? 16 : per);
    while ((tiles + per - 1) / per > 65535)
        per *= 2;
    a.tiles = (int32_t)per;
    hipLaunchKernelGGL((expand_kernel<KS, CT, kNN>), dim3((unsigned)blocks, (unsigned)((tiles + per - 1) / per)),
                       dim3(kAdBlock), 0, st, a);
}

template <bool kNN>
void expand(const ExpandArgs &a, hipStream_t st)
{
    if (a.w.rank <= 16)
        expand_as<1, 4, kNN>(a, st);
    else if (a.w.rank <= 32)
        expand_as<2, 4, kNN>(a, st);
    else if (a.w.rank <= 64)
        expand_as<4, 4, kNN>(a, st);
    else
        expand_as<8, 2, kNN>(a, st);
}

template <int T, int CT>
void wgrad_as(WgradArgs a, hipStream_t st)
{
    a.blocks_a = (a.in_dim + 64 * CT - 1) / (64 * CT);
    const int32_t blocks = a.blocks_a + (a.out_dim + 64 * CT - 1) / (64 * CT);
    hipLaunchKernelGGL((wgrad_kernel<T, CT>), dim3(blocks, a.nchunks), dim3(kAdBlock), 0, st, a);
}

}  // namespace

size_t adapter_workspace(int64_t rows, const moonep_adapters &ad)
{
    return (size_t)rows * ad.rank * 4 * kMostSplits + 65536;
}

size_t adapter_bwd_workspace(int64_t rows, const moonep_adapters &ad)
{
    return (size_t)rows * ad.rank * 4 * (kMostSplits + 1) +
           (size_t)(kMostChunks + ad.n) * ad.rank * ((size_t)ad.in_dim + ad.out_dim) * 4 + 65536;
}

int launch_adapter(int32_t rows, const moonep_adapters &ad, const int32_t *ids, const int32_t *order,
                   const uint16_t *x, const uint16_t *bank, const float *scale, const uint16_t *base,
                   float *u, uint16_t *y, void *ws, hipStream_t st)
{
    if (rows == 0)
        return MOONEP_OK;
    const AdRows r{ids, order, rows, ad.n};
    const int splits = split_count(rows, ad.in_dim);
    float *to = splits > 1 ? (float *)ws : u;
    shrink<false>(ShrinkArgs{r, {bank + ad.a_offset, ad.stride, ad.rank, ad.in_dim}, x, nullptr, to},
                  splits, st);
    expand<false>(ExpandArgs{r, {bank + ad.b_offset, ad.stride, ad.rank, ad.out_dim}, to,
                             splits > 1 ? u : nullptr, scale, base, y, splits, 0}, st);
    return status();
}

int launch_adapter_bwd(int32_t rows, int32_t E, const moonep_adapters &ad, const int32_t *ids,
                       const int32_t *order, const int32_t *plan, const uint16_t *x, const float *u,
                       const uint16_t *dy, const uint16_t *bank, const float *scale,
                       const uint16_t *dx_base, uint16_t *dx, int accumulate, float *d_bank, void *ws,
                       hipStream_t st)
{
    if (rows == 0 && (!d_bank || accumulate))
        return MOONEP_OK;
    const AdRows r{ids, order, rows, ad.n};
    const size_t plane = (size_t)rows * ad.rank;
    float *du = (float *)ws, *parts = du + plane;
    if (rows) {
        // with one part, or nobody to join them, du is written at once
        const int splits = dx ? split_count(rows, ad.out_dim) : 1;
        float *to = splits > 1 ? parts : du;
        shrink<true>(ShrinkArgs{r, {bank + ad.b_offset, ad.stride, ad.rank, ad.out_dim}, dy, scale, to},
                     splits, st);
        if (dx)
            expand<true>(ExpandArgs{r, {bank + ad.a_offset, ad.stride, ad.rank, ad.in_dim}, to,
                                    splits > 1 ? du : nullptr, nullptr, dx_base, dx, splits, 0}, st);
    }
    if (d_bank) {
        const PlanLayout pl = plan_layout(E, 1);
        WgradArgs a{};
        a.r = r;
        a.off = plan + pl.home_row_off;
        a.keep = plan + pl.keep;
        a.rank = ad.rank;
        a.in_dim = ad.in_dim;
        a.out_dim = ad.out_dim;
        a.stride = ad.stride;
        a.a_off = ad.a_offset;
        a.b_off = ad.b_offset;
        a.accumulate = accumulate;
        a.du = du;
        a.u = u;
        a.scale = scale;
        a.x = x;
        a.dy = dy;
        a.part = (float *)(((uintptr_t)(parts + kMostSplits * plane) + 255) & ~(uintptr_t)255);
        a.d_bank = d_bank;
        // chunks of at least 128 positions, 64 at most, for about 1024 workgroups
        const int32_t blocks = (ad.in_dim + ad.out_dim + 255) / 256;
        int32_t chunks = 1024 / blocks;
        chunks = chunks < 1 ? 1 : (chunks > kMostChunks ? kMostChunks : chunks);
        int64_t chunk = ((int64_t)rows + chunks - 1) / chunks;
        chunk = (chunk + 31) / 32 * 32;
        chunk = chunk < 128 ? 128 : chunk;
        a.chunk = (int32_t)chunk;
        a.nchunks = (int32_t)(((int64_t)rows + chunk - 1) / chunk);
        if (rows) {
            if (ad.rank <= 16)
                wgrad_as<1, 4>(a, st);
            else if (ad.rank <= 32)
                wgrad_as<2, 4>(a, st);
            else if (ad.rank <= 64)
                wgrad_as<4, 4>(a, st);
            else
                wgrad_as<8, 4>(a, st);
        }
        const int64_t window = (int64_t)ad.rank * ((int64_t)ad.in_dim + ad.out_dim);
        const int64_t nb = (window + kAdBlock * 4 - 1) / (kAdBlock * 4);
        hipLaunchKernelGGL(wgrad_join_kernel, dim3((unsigned)(nb < 128 ? nb : 128), ad.n), dim3(kAdBlock),
                           0, st, a);
    }
    return status();
}

}  // namespace moonep
