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
// Three products, on the 16 x 16 x 32 bf16 matrix instruction, each with its
// matrix in either order:
//   shrink  rows [D] against a matrix, to rank values in fp32 (u, du);
//   expand  rank values against a matrix, added to base rows (y, dx);
//   wgrad   rank values against rows [D], summed over an adapter's rows.
// Rows are worked on in tiles of 16 or 64 positions, in `order`, where rows of one
// adapter stand together, or as they are.  A tile whose rows have several
// adapters is run once for each, every row keeping the results of its own (what
// another adapter's matrix holds, NaN or infinity, cannot reach it).
//
// Lane layout of the instruction (m, n: 16; k: 32): operand A lane l holds row
// m = l % 16, k = 8 (l / 16) .. + 7; operand B lane l column n = l % 16, same k;
// the result's lane l holds column l % 16, rows 4 (l / 16) .. + 3.  Loaded from rows
// as they are, an operand's neighbouring lanes are in different rows, and the
// vector-memory path serves one 64-byte piece after the other: such kernels ran at
// half the bandwidth.  So whatever is read for every row comes in runs: rows of x
// through LDS, base and y with 16 lanes along a row, and the rank values laid out by
// their producer in the order of the lanes that take them (`parts`, `turned`).
//
// Rounding: u and du stay in fp32.  Where they enter a product they are split
// into bf16 parts whose products the instruction sums in fp32: two parts (16
// bits) in expand, whose result is rounded to bf16; three (24 bits, all of it)
// in wgrad, whose result is fp32.
#include "segments.hpp"

namespace moonep {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

namespace {

constexpr int kAdBlock = 256;  // four waves
constexpr int kMostSplits = 14, kMostSplitsBwd = 8;
constexpr int kMostChunks = 64;
constexpr int32_t kFewRows = 256;  // up to here a tile's adapters are spread over waves

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
    const float *scale;     // per adapter: of the results, or of `parts` alone
    float *out;             // [splits][rows][rank]
    uint16_t *parts;        // or NULL: scale * result, see Parts
};

// Two bf16 parts of a pair of values, packed: 16 bits of each.  The second part
// of an infinity is 0.
__device__ __forceinline__ void split2(float a, float b, uint32_t *hi, uint32_t *lo)
{
    const uint32_t h = pack_bf16(a, b);
    const float h0 = bf16_lo(h), h1 = bf16_hi(h);
    *hi = h;
    *lo = pack_bf16(__builtin_isfinite(h0) ? a - h0 : 0.0f, __builtin_isfinite(h1) ? b - h1 : 0.0f);
}

// The two bf16 parts of rank values in the order in which expand's lanes take them:
// for each 16 positions, steps() steps of 64 lanes x 8 values.  Lane 16 g + m of step
// s holds chunk c = 4 s + g of position m: values 8 (c % per) .. + 7 of part c / per.
// Chunks past the rank are not written, nor used.
struct Parts {
    int32_t per;  // chunks of a part: whole steps, or half of one
    __host__ __device__ explicit Parts(int32_t rank) : per(rank <= 16 ? 2 : rank <= 32 ? 4 : rank <= 64 ? 8 : 16) {}
    __host__ __device__ int32_t steps() const { return per / 2; }
    // Elements before chunk c of a position.
    __device__ int64_t at(int64_t pos, int32_t c) const
    {
        return ((pos / 16 * (per * 2) + c) * 16 + pos % 16) * 8;
    }
    // Values c .. c + 3 of a position (c % 4 == 0).
    __device__ __forceinline__ void put(uint16_t *parts, int64_t pos, int32_t c, f32x4 v) const
    {
        u32x2 hi, lo;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t h, l;
            split2(v[2 * j], v[2 * j + 1], &h, &l);
            hi[j] = h;
            lo[j] = l;
        }
        *(u32x2 *)(parts + at(pos, c / 8) + c % 8) = hi;
        *(u32x2 *)(parts + at(pos, per + c / 8) + c % 8) = lo;
    }
};

__device__ __align__(16) const uint32_t kZeros[4] = {0, 0, 0, 0};

__device__ __forceinline__ void dma16(const void *src, char *dst)
{
    __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N >= 0 && N <= 63, "vmcnt");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

// A workgroup barrier that waits for this wave's LDS operations only.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// N fragments whose 8 values of k are rows of LDS: 16 lanes read 4 rows x 16
// columns, 8 bytes each, and lane d gets column d; `lo` for the first four rows and
// `hi` for the others.  With its wait inside: see gemm_bwd.hip.
template <int N>
__device__ __forceinline__ void tr_frags(const uint32_t (&lo)[N], const uint32_t (&hi)[N], Frag (&f)[N])
{
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    static_assert(N == 1 || N == 2 || N == 4, "fragments a read");
    s16x4 r[2 * N];
    if constexpr (N == 1)
        asm volatile("ds_read_b64_tr_b16 %0, %2\n\t"
                     "ds_read_b64_tr_b16 %1, %3\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(r[0]), "=&v"(r[1])
                     : "v"(lo[0]), "v"(hi[0])
                     : "memory");
    else if constexpr (N == 2)
        asm volatile("ds_read_b64_tr_b16 %0, %4\n\t"
                     "ds_read_b64_tr_b16 %1, %5\n\t"
                     "ds_read_b64_tr_b16 %2, %6\n\t"
                     "ds_read_b64_tr_b16 %3, %7\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])
                     : "v"(lo[0]), "v"(hi[0]), "v"(lo[1]), "v"(hi[1])
                     : "memory");
    else
        asm volatile("ds_read_b64_tr_b16 %0, %8\n\t"
                     "ds_read_b64_tr_b16 %1, %9\n\t"
                     "ds_read_b64_tr_b16 %2, %10\n\t"
                     "ds_read_b64_tr_b16 %3, %11\n\t"
                     "ds_read_b64_tr_b16 %4, %12\n\t"
                     "ds_read_b64_tr_b16 %5, %13\n\t"
                     "ds_read_b64_tr_b16 %6, %14\n\t"
                     "ds_read_b64_tr_b16 %7, %15\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]),
                       "=&v"(r[6]), "=&v"(r[7])
                     : "v"(lo[0]), "v"(hi[0]), "v"(lo[1]), "v"(hi[1]), "v"(lo[2]), "v"(hi[2]), "v"(lo[3]),
                       "v"(hi[3])
                     : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i].v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(r[2 * i], r[2 * i + 1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// Many rows: 64 positions a workgroup, 16 a wave, rows and matrix through a ring of
// LDS stages of 64 values of the contraction, filled by LDS-DMA.  blockIdx.y is one
// of gridDim.y parts of the contraction.  The matrix's stage is [16 T][64], or
// with kNN what memory has: 64 rows of rank.
template <int T, bool kNN>
struct ShrinkCfg {
    static constexpr int kRows = 64, kStageX = kRows * 128, kStageW = T * 2048;
    static constexpr int kStageBytes = kStageX + kStageW;
    static constexpr int kWInstr = T < 4 ? 1 : T / 2;  // loads of a wave for the matrix's stage
    static constexpr int kPerStage = 2 + kWInstr;
    static constexpr int kStages = T == 8 ? 3 : 4;
    static constexpr int kLds = kStages * kStageBytes;
    // 16-byte chunk c of row r of a stage of 128-byte rows sits at c ^ swz(r)
    __device__ static constexpr int swz(int r) { return (r / 2) % 8; }
};

template <int T, bool kNN>
__global__ __launch_bounds__(kAdBlock) void shrink_kernel(ShrinkArgs a)
{
    using G = ShrinkCfg<T, kNN>;
    extern __shared__ __align__(16) char ring[];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int m = lane & 15, g = lane >> 4;
    const int32_t D = a.w.D, rank = a.w.rank;
    const int64_t p0 = (int64_t)blockIdx.x * G::kRows;
    const int32_t steps = (D + 63) / 64;
    const int32_t k0 = (int32_t)((int64_t)steps * blockIdx.y / gridDim.y);
    const int32_t nk = (int32_t)((int64_t)steps * (blockIdx.y + 1) / gridDim.y) - k0;

    // this lane's chunk of two rows, of its wave's two loads of a stage of rows
    const uint16_t *xp[2];
    int xc[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const int r = (v * 4 + wave) * 8 + lane / 8;
        const int32_t row = a.r.row(p0 + r);
        xc[v] = (lane % 8) ^ G::swz(r);
        xp[v] = a.x + (int64_t)(row < 0 ? 0 : row) * D + xc[v] * 8;
    }
    uint64_t todo = ballot(a.r.id(a.r.row(p0 + lane)) >= 0);  // the same in every wave
    const int32_t id_all = a.r.id(a.r.row(p0 + lane));
    const int64_t pos = p0 + wave * 16 + m;
    const int32_t row = a.r.row(pos), id = a.r.id(row);
    f32x4 res[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
        res[t] = f32x4{0, 0, 0, 0};

    while (todo) {
        const int32_t cur = __builtin_amdgcn_readlane(id_all, __builtin_ctzll(todo));
        todo &= ~ballot(id_all == cur);
        const uint16_t *w = a.w.first + cur * a.w.stride;
        const int32_t kn = kNN ? rank / 8 : 2 * T;  // KiB of the matrix's stage
        const uint16_t *wp[G::kWInstr];
        int wk[G::kWInstr];  // the value of the contraction that this lane's chunk begins at, in a stage
#pragma unroll
        for (int v = 0; v < G::kWInstr; ++v) {
            const int at = (v * 4 + wave) % kn * 64 + lane;  // waves without a load of their own repeat one
            if (kNN) {
                wk[v] = at * 8 / rank;
                wp[v] = w + at * 8;
            } else {
                const int r = at / 8;
                wk[v] = ((at % 8) ^ G::swz(r)) * 8;
                wp[v] = w + (int64_t)(r < rank ? r : 0) * D + wk[v];
            }
        }
        auto issue = [&](int32_t kt, int st) {
            char *to = ring + st * G::kStageBytes;
            const int32_t k = (k0 + kt) * 64;
#pragma unroll
            for (int v = 0; v < 2; ++v)
                dma16(k + xc[v] * 8 < D ? (const void *)(xp[v] + k) : kZeros, to + (v * 4 + wave) * 1024);
#pragma unroll
            for (int v = 0; v < G::kWInstr; ++v)
                dma16(k + wk[v] < D ? (const void *)(wp[v] + (kNN ? (int64_t)k * rank : k)) : kZeros,
                      to + G::kStageX + (v * 4 + wave) % kn * 1024);
        };
        f32x4 acc[T];
#pragma unroll
        for (int t = 0; t < T; ++t)
            acc[t] = f32x4{0, 0, 0, 0};
        lds_barrier();  // the adapter before is done with the ring
#pragma unroll
        for (int st = 0; st + 1 < G::kStages; ++st)
            if (st < nk)
                issue(st, st);
        const bool mine = ballot(id == cur) != 0;
        int now = 0;
        for (int32_t kt = 0; kt < nk; ++kt) {
            if (kt + G::kStages - 2 < nk)
                wait_vm<(G::kStages - 2) * G::kPerStage>();
            else
                wait_vm<0>();
            lds_barrier();  // the stage is visible to all, the one before is free
            if (kt + G::kStages - 1 < nk)
                issue(kt + G::kStages - 1, now ? now - 1 : G::kStages - 1);
            const char *x = ring + now * G::kStageBytes, *ws = x + G::kStageX;
            now = now + 1 == G::kStages ? 0 : now + 1;
            if (!mine)
                continue;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                Frag xf, wf[T];
                xf.v = *(const bf16x8 *)(x + (wave * 16 + m) * 128 + (((ks * 4 + g) ^ G::swz(m)) << 4));
                if constexpr (kNN) {
                    const uint32_t at = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char *)ws +
                                        (ks * 32 + g * 8 + (m >> 2)) * rank * 2 + (m & 3) * 8;
                    constexpr int N = T < 4 ? T : 4;
#pragma unroll
                    for (int t = 0; t < T; t += N) {
                        uint32_t lo[N], hi[N];
                        Frag f[N];
#pragma unroll
                        for (int q = 0; q < N; ++q) {
                            lo[q] = at + (t + q) * 32;
                            hi[q] = lo[q] + 8 * rank;
                        }
                        tr_frags<N>(lo, hi, f);
#pragma unroll
                        for (int q = 0; q < N; ++q)
                            wf[t + q] = f[q];
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < T; ++t)
                        wf[t].v = *(const bf16x8 *)(ws + (t * 16 + m) * 128 + (((ks * 4 + g) ^ G::swz(m)) << 4));
                }
#pragma unroll
                for (int t = 0; t < T; ++t)
                    acc[t] = mfma16(wf[t].v, xf.v, acc[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                res[t][j] = id == cur ? acc[t][j] : res[t][j];
    }
    if (row < 0)
        return;
    const float s = id >= 0 && a.scale ? a.scale[id] : 1.0f;
    const Parts parts(rank);
    float *o = a.out + ((int64_t)blockIdx.y * a.r.rows + row) * rank;
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int32_t c = t * 16 + g * 4;
        if (c >= rank)
            continue;
        *(f32x4 *)(o + c) = a.parts ? res[t] : res[t] * s;
        if (a.parts)
            parts.put(a.parts, pos, c, res[t] * s);
    }
}

// Few rows: 16 positions a workgroup, operands straight into registers.  The four
// waves share the rows, each with a part of the contraction, of which blockIdx.y
// is one of gridDim.y parts; their sums are joined in LDS.  Of a tile's
// adapters, workgroup blockIdx.z has every gridDim.z-th, and their rows.  The 16
// rows of the instruction's tile t are indexes m T + t of the rank, so that a
// lane's results are 4 T consecutive ones.
template <int T, bool kNN>
__global__ __launch_bounds__(kAdBlock) void shrink_few_kernel(ShrinkArgs a)
{
    constexpr int RT = 1;
    constexpr int U = T <= 4 ? 4 : 2;  // steps in flight
    const int lane = lane_id(), wave = (int)threadIdx.x >> 6;
    const int m = lane & 15, g = lane >> 4;
    const int32_t D = a.w.D, rank = a.w.rank;
    const int64_t p0 = (int64_t)blockIdx.x * 16 * RT;
    const int32_t steps = (D + 31) / 32;
    const int32_t cuts = (int32_t)gridDim.y * 4, cut = (int32_t)blockIdx.y * 4 + wave;
    const int32_t k0 = (int32_t)((int64_t)steps * cut / cuts);
    const int32_t k1 = (int32_t)((int64_t)steps * (cut + 1) / cuts);
    const int32_t full = k1 < D / 32 ? k1 : D / 32;  // steps before this have all 32

    int32_t row[RT], id[RT];
    const uint16_t *xp[RT];
    uint64_t todo[RT], store[RT];
    f32x4 res[RT][T];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        row[i] = a.r.row(p0 + i * 16 + m);
        id[i] = a.r.id(row[i]);
        xp[i] = a.x + (int64_t)(row[i] < 0 ? 0 : row[i]) * D + g * 8;
        todo[i] = ballot(id[i] >= 0);
        store[i] = blockIdx.z == 0 ? ballot(row[i] >= 0 && id[i] < 0) : 0;
#pragma unroll
        for (int t = 0; t < T; ++t)
            res[i][t] = f32x4{0, 0, 0, 0};
    }
    const int32_t r0 = m * T < rank ? m * T : 0;  // lanes past the rank repeat index 0: not stored

    for (uint32_t turn = 0;; turn = turn + 1 == gridDim.z ? 0 : turn + 1) {
        int32_t cur = -1;
#pragma unroll
        for (int i = 0; i < RT; ++i)
            if (cur < 0 && todo[i])
                cur = __builtin_amdgcn_readlane(id[i], __builtin_ctzll(todo[i]));
        if (cur < 0)
            break;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const uint64_t mine = ballot(id[i] == cur);
            todo[i] &= ~mine;
            store[i] |= turn == blockIdx.z ? mine : 0;
        }
        if (turn != blockIdx.z)
            continue;
        const uint16_t *w = a.w.first + cur * a.w.stride;
        w += kNN ? (int64_t)g * 8 * rank + r0 : (int64_t)r0 * D + g * 8;
        auto load_w = [&](int32_t k, Frag (&f)[T]) {
            if constexpr (kNN) {
                Halves<T> v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = load_halves<T>(w + (int64_t)(k * 32 + j) * rank);
#pragma unroll
                for (int t = 0; t < T; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        f[t].w[j] = (uint32_t)v[2 * j].h[t] | (uint32_t)v[2 * j + 1].h[t] << 16;
            } else {
#pragma unroll
                for (int t = 0; t < T; ++t)
                    f[t].v = *(const bf16x8 *)(w + (int64_t)t * D + k * 32);
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
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    x[u][i].v = *(const bf16x8 *)(xp[i] + (k + u) * 32);
#pragma unroll
            for (int u = 0; u < U; ++u)
                load_w(k + u, f[u]);
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
            Frag x[RT], f[T];
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[i].w[j] = 0;
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f[t].w[j] = 0;
            if (k * 32 + g * 8 < D) {
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    x[i].v = *(const bf16x8 *)(xp[i] + k * 32);
                load_w(k, f);
            }
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int t = 0; t < T; ++t)
                    acc[i][t] = mfma16(f[t].v, x[i].v, acc[i][t]);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    res[i][t][j] = id[i] == cur ? acc[i][t][j] : res[i][t][j];
    }

    // Row tile i is joined and written by wave i % 4.
    __shared__ f32x4 join[RT][4][T][64];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int t = 0; t < T; ++t)
            join[i][wave][t][lane] = res[i][t];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        if ((i & 3) != wave || !(store[i] >> lane & 1))
            continue;
        const float s = id[i] >= 0 && a.scale ? a.scale[id[i]] : 1.0f;
        float v[4 * T];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            f32x4 sum = join[i][0][t][lane];
#pragma unroll
            for (int q = 1; q < 4; ++q)
                sum += join[i][q][t][lane];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j * T + t] = sum[j] * s;
        }
        float *o = a.out + ((int64_t)blockIdx.y * a.r.rows + row[i]) * rank + g * 4 * T;
#pragma unroll
        for (int q = 0; q < T; ++q)
            if (g * 4 * T + q * 4 < rank)
                *(f32x4 *)(o + q * 4) = f32x4{v[q * 4], v[q * 4 + 1], v[q * 4 + 2], v[q * 4 + 3]};
    }
}

// ---------------------------------------------------------------------------
// prepare: partial sums joined and cut into the parts that the products take
// ---------------------------------------------------------------------------

constexpr int kStep = 32;  // positions of one step of wgrad's contraction

struct PrepArgs {
    AdRows r;
    const float *scale;
    int32_t rank, tiles, splits;
    const float *sums;   // [splits][rows][rank]
    float *total;        // [rows][rank]: their sum, or NULL
    uint16_t *parts;     // of scale_parts ? scale * sum : sum, or NULL
    int32_t scale_parts;
    const float *u;      // [rows][rank]
    // For wgrad, or NULL: all bits of the sums, and of scale * u, as wgrad's lanes take
    // them: for each 32 positions and each of three bf16 parts, `tiles` tiles of 64
    // lanes x 8 values; lane 16 g + m of tile t holds index 16 t + m of the rank at
    // positions 8 g .. + 7.  Zeros for positions without an adapter; indexes past the
    // rank are not used.
    uint16_t *t_sum, *t_u;
};

// The three bf16 parts of a value, all 24 bits; the later ones of an infinity are 0.
__device__ __forceinline__ void split3(float a, uint16_t *p0, uint16_t *p1, uint16_t *p2)
{
    const uint32_t hi = pack_bf16(a, 0.0f);
    const float h = bf16_lo(hi);
    const float r = __builtin_isfinite(h) ? a - h : 0.0f;
    const uint32_t mid = pack_bf16(r, 0.0f);
    *p0 = (uint16_t)hi;
    *p1 = (uint16_t)mid;
    *p2 = (uint16_t)pack_bf16(r - bf16_lo(mid), 0.0f);
}

// One workgroup: 32 positions, 8 threads each.
__global__ __launch_bounds__(kAdBlock) void adapter_prep_kernel(PrepArgs a)
{
    extern __shared__ __align__(16) uint16_t turned[];  // both arrays' step, as it leaves
    const int p = (int)threadIdx.x & 31, part = (int)threadIdx.x >> 5;
    const int32_t rank = a.rank, plane = a.tiles * 512;  // elements of one bf16 part of a step
    const int64_t pos = (int64_t)blockIdx.x * kStep + p;
    const int32_t row = a.r.row(pos), id = a.r.id(row);
    const float s = id >= 0 ? a.scale[id] : 0.0f, by = a.scale_parts ? s : 1.0f;
    const Parts parts(rank);
    for (int32_t c = part * 4; c < rank; c += 32) {
        f32x4 v = {0, 0, 0, 0}, w = {0, 0, 0, 0};
        if (id >= 0) {
            const float *q = a.sums + (int64_t)row * rank + c;
            v = *(const f32x4 *)q;
            for (int32_t i = 1; i < a.splits; ++i)
                v += *(const f32x4 *)(q + i * ((int64_t)a.r.rows * rank));
            if (a.t_u)
                w = *(const f32x4 *)(a.u + (int64_t)row * rank + c) * s;
        }
        if (row >= 0 && a.total)
            *(f32x4 *)(a.total + (int64_t)row * rank + c) = v;
        if (row >= 0 && a.parts)
            parts.put(a.parts, pos, c, v * by);
        if (a.t_u) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int32_t r = c + j;
                uint16_t *t = turned + (r / 16 * 64 + p / 8 * 16 + r % 16) * 8 + p % 8;
                split3(v[j], t, t + plane, t + 2 * plane);
                t += 3 * plane;
                split3(w[j], t, t + plane, t + 2 * plane);
            }
        }
    }
    if (!a.t_u)
        return;
    __syncthreads();
    const int32_t words = 3 * plane / 8;
    for (int32_t i = (int)threadIdx.x; i < 2 * words; i += kAdBlock) {
        u32x4 *to = (u32x4 *)(i < words ? a.t_sum : a.t_u) + (int64_t)blockIdx.x * words;
        to[i < words ? i : i - words] = ((const u32x4 *)turned)[i];
    }
}

// ---------------------------------------------------------------------------
// expand
// ---------------------------------------------------------------------------

struct ExpandArgs {
    AdRows r;
    AdMats w;
    const uint16_t *parts;  // what is multiplied
    const uint16_t *base;
    uint16_t *y;
    int32_t tiles;          // row tiles a workgroup
    // few rows: the parts are not made yet
    const float *sums;      // [splits][rows][rank]
    float *total;           // their sum
    const float *scale;
    int32_t splits;
};

template <int CT>
struct Piece;  // CT bf16 values of a row
template <>
struct Piece<8> {
    typedef u32x4 type;
};
template <>
struct Piece<4> {
    typedef u32x2 type;
};

// The contraction is over both parts, PS steps each (kHalf: both in one step).
// Positions are the instruction's rows and columns its columns: a wave has 16 CT,
// column n CT + t in column n of tile t, so that a lane's results are CT
// consecutive columns of positions 4 g .. + 3, and 16 lanes write a run of a row.
template <int PS, bool kHalf, int CT, bool kNN>
struct Expand {
    static constexpr int kSteps = kHalf ? 1 : 2 * PS;
    typedef typename Piece<CT>::type piece;
    int32_t D, rank, c0, col, wc;
    int chunk[PS];  // values of the rank this lane has in step s of a part
    bool in[PS];

    __device__ __forceinline__ Expand(const AdMats &w, int32_t column)
    {
        const int n = lane_id() & 15, g = lane_id() >> 4;
        D = w.D;
        rank = w.rank;
        c0 = column;
        col = c0 + n * CT;
        wc = col < D ? col : 0;  // lanes past D repeat column 0: not stored
#pragma unroll
        for (int s = 0; s < PS; ++s) {
            const int c = (s * 4 + (kHalf ? g & 1 : g)) * 8;
            in[s] = c < rank;
            chunk[s] = in[s] ? c : 0;
        }
    }
    __device__ __forceinline__ void load_w(const uint16_t *w, Frag (&f)[PS][CT]) const
    {
#pragma unroll
        for (int k = 0; k < PS; ++k) {
            if constexpr (kNN) {
                Halves<CT> v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = load_halves<CT>(w + (int64_t)(chunk[k] + j) * D + wc);
#pragma unroll
                for (int t = 0; t < CT; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        f[k][t].w[j] = (uint32_t)v[2 * j].h[t] | (uint32_t)v[2 * j + 1].h[t] << 16;
            } else {
#pragma unroll
                for (int t = 0; t < CT; ++t)
                    f[k][t].v = *(const bf16x8 *)(w + (int64_t)(wc + t) * rank + chunk[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < PS; ++k)
#pragma unroll
            for (int t = 0; t < CT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f[k][t].w[j] = in[k] ? f[k][t].w[j] : 0;
    }
    // The tile's parts; positions past the last row read what is there, and are not stored.
    __device__ __forceinline__ void load_parts(const uint16_t *parts, int64_t tile, Frag (&f)[kSteps]) const
    {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                f[s].w[j] = 0;
            if (in[kHalf ? 0 : s % PS])
                f[s].v = *(const bf16x8 *)(parts + ((tile * kSteps + s) * 64 + lane_id()) * 8);
        }
    }
    __device__ __forceinline__ void load_base(const uint16_t *base, const int32_t (&row)[4],
                                              const bool (&wanted)[4], piece (&b)[4]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b[i] = piece{};
            if (wanted[i] && col < D)
                b[i] = *(const piece *)(base + (int64_t)row[i] * D + col);
        }
    }
    __device__ __forceinline__ void product(const Frag (&w)[PS][CT], const Frag (&u)[kSteps],
                                            const bool (&mine)[4], f32x4 (&res)[CT]) const
    {
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            f32x4 acc = {0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                acc = mfma16(u[s].v, w[kHalf ? 0 : s % PS][t].v, acc);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                res[t][i] = mine[i] ? acc[i] : res[t][i];
        }
    }
    // A row without an adapter is copied bit for bit.
    __device__ __forceinline__ void store(uint16_t *y, const int32_t (&row)[4], const int32_t (&id)[4],
                                          const bool (&wanted)[4], const piece (&b)[4],
                                          const f32x4 (&res)[CT]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!wanted[i] || col >= D)
                continue;
            piece o;
#pragma unroll
            for (int t = 0; t < CT; t += 2) {
                const uint32_t v = pack_bf16(bf16_lo(b[i][t / 2]) + res[t][i], bf16_hi(b[i][t / 2]) + res[t + 1][i]);
                o[t / 2] = id[i] >= 0 ? v : b[i][t / 2];
            }
            *(piece *)(y + (int64_t)row[i] * D + col) = o;
        }
    }
};

// Many rows: a wave keeps its columns of one adapter's matrix in registers and
// walks row tiles.  Base rows and parts come through the wave's own ring of LDS
// slots, kAhead tiles ahead: so many bytes in flight would not fit the registers,
// and no wave waits for another.
constexpr int kAhead = 2;
constexpr int kTileRun = 32;  // row tiles whose rows and adapters are looked up at once

template <int PS, bool kHalf, int CT>
struct ExpandRing {
    static constexpr int kSteps = kHalf ? 1 : 2 * PS;
    static constexpr int kLanesRow = 2 * CT;              // lanes, 16 bytes each, of a row
    static constexpr int kBaseInstr = 16 * kLanesRow / 64;
    static constexpr int kLoads = kBaseInstr + kSteps;    // of a tile
    static constexpr int kBaseBytes = 16 * CT * 32;
    static constexpr int kSlot = kBaseBytes + kSteps * 1024;
    static constexpr int kLds = 4 * (kAhead + 1) * kSlot;
    static_assert(kAhead * (kLoads + 4) <= 63, "outstanding accesses must fit vmcnt");
};

template <int PS, bool kHalf, int CT, bool kNN>
__global__ __launch_bounds__(kAdBlock) void expand_kernel(ExpandArgs a)
{
    using X = Expand<PS, kHalf, CT, kNN>;
    using G = ExpandRing<PS, kHalf, CT>;
    typedef typename X::piece piece;
    extern __shared__ __align__(16) char ring_all[];
    __shared__ int32_t rows[kTileRun * 16], ids[kTileRun * 16];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), g = lane >> 4;
    const X x(a.w, ((int32_t)blockIdx.x * 4 + wave) * 16 * CT);
    char *ring = ring_all + wave * (kAhead + 1) * G::kSlot;
    const bool copy = a.y != a.base;
    const int64_t tiles = ((int64_t)a.r.rows + 15) / 16;
    const int64_t last = ((int64_t)blockIdx.y + 1) * a.tiles < tiles ? ((int64_t)blockIdx.y + 1) * a.tiles : tiles;
    Frag wf[PS][CT];
    int32_t have = -1;
    for (int64_t first = (int64_t)blockIdx.y * a.tiles; first < last; first += kTileRun) {
        const int32_t n = (int32_t)(last - first < kTileRun ? last - first : kTileRun);
        __syncthreads();
        for (int32_t i = (int)threadIdx.x; i < n * 16; i += kAdBlock) {
            const int32_t row = a.r.row(first * 16 + i), id = a.r.id(row);
            rows[i] = id >= 0 || copy ? row : -1;  // neither read nor written
            ids[i] = id;
        }
        __syncthreads();
        if (x.c0 >= x.D)
            continue;
        // As many loads for every tile, also past the last one.
        auto issue = [&](int32_t t, int slot) {
            char *to = ring + slot * G::kSlot;
            const int32_t c = x.c0 + lane % G::kLanesRow * 8;
#pragma unroll
            for (int v = 0; v < G::kBaseInstr; ++v) {
                const int32_t row = t < n ? rows[t * 16 + (v * 64 + lane) / G::kLanesRow] : -1;
                dma16(row >= 0 && c < x.D ? (const void *)(a.base + (int64_t)row * x.D + c) : kZeros, to + v * 1024);
            }
#pragma unroll
            for (int s = 0; s < G::kSteps; ++s)
                dma16(t < n ? (const void *)(a.parts + (((first + t) * G::kSteps + s) * 64 + lane) * 8) : kZeros,
                      to + G::kBaseBytes + s * 1024);
        };
#pragma unroll
        for (int t = 0; t < kAhead; ++t)
            issue(t, t);
        int slot = 0, stored = 0;  // stored: tiles just before this one whose four stores were issued, kAhead at most
        for (int32_t t = 0; t < n; ++t) {
            wave_sync();
            issue(t + kAhead, slot ? slot - 1 : kAhead);
            // the tile's loads have landed once only what was issued after them is
            // outstanding: kAhead tiles' loads, and the stores in between
            if (stored == 2)
                wait_vm<kAhead * G::kLoads + 2 * 4>();
            else if (stored == 1)
                wait_vm<kAhead * G::kLoads + 4>();
            else
                wait_vm<kAhead * G::kLoads>();
            asm volatile("" ::: "memory");
            const char *at = ring + slot * G::kSlot;
            slot = slot == kAhead ? 0 : slot + 1;
            int32_t row[4], id[4];
            piece b[4];
            Frag u[G::kSteps];
            bool left[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                row[i] = rows[t * 16 + g * 4 + i];
                id[i] = ids[t * 16 + g * 4 + i];
                left[i] = id[i] >= 0;
                b[i] = *(const piece *)(at + (g * 4 + i) * CT * 32 + (lane & 15) * CT * 2);
            }
#pragma unroll
            for (int s = 0; s < G::kSteps; ++s) {
                u[s].v = *(const bf16x8 *)(at + G::kBaseBytes + s * 1024 + lane * 16);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    u[s].w[j] = x.in[kHalf ? 0 : s % PS] ? u[s].w[j] : 0;
            }
            f32x4 res[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c)
                res[c] = f32x4{0, 0, 0, 0};
            for (;;) {
                int32_t cur = -1;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t some = ballot(left[i]);
                    if (cur < 0 && some)
                        cur = __builtin_amdgcn_readlane(id[i], __builtin_ctzll(some));
                }
                if (cur < 0)
                    break;
                if (cur != have) {
                    have = cur;
                    x.load_w(a.w.first + cur * a.w.stride, wf);
                }
                bool mine[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mine[i] = id[i] == cur;
                    left[i] = left[i] && !mine[i];
                }
                x.product(wf, u, mine, res);
            }
            bool wanted[4];
            uint64_t all = ~(uint64_t)0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wanted[i] = row[i] >= 0;
                all &= ballot(wanted[i] && x.col < x.D);
            }
            x.store(a.y, row, id, wanted, b, res);
            stored = all == ~(uint64_t)0 ? (stored < kAhead ? stored + 1 : kAhead) : 0;
        }
        wait_vm<0>();  // nothing is on its way into the LDS when it is given back
    }
}

// Few rows: the four waves of a workgroup and gridDim.z of them share a row tile
// and its 16 CT columns, each with some of the tile's adapters and their rows.
template <int PS, bool kHalf, int CT, bool kNN, bool kJoin>
__global__ __launch_bounds__(kAdBlock) void expand_few_kernel(ExpandArgs a)
{
    using X = Expand<PS, kHalf, CT, kNN>;
    const int wave = (int)threadIdx.x >> 6, m = lane_id() & 15, g = lane_id() >> 4;
    const X x(a.w, (int32_t)blockIdx.x * 16 * CT);
    const uint32_t share = blockIdx.z * 4 + wave, shares = gridDim.z * 4;
    const int64_t p0 = (int64_t)blockIdx.y * 16;
    // of position m, and of this lane's results
    const int32_t u_row = a.r.row(p0 + m), u_id = a.r.id(u_row);
    uint64_t left = ballot(u_id >= 0), taken = share == 0 ? ballot(u_row >= 0 && u_id < 0 && a.y != a.base) : 0;
    uint64_t todo = 0;
    for (uint32_t turn = 0; left; turn = turn + 1 == shares ? 0 : turn + 1) {
        const uint64_t mine = ballot(u_id == __builtin_amdgcn_readlane(u_id, __builtin_ctzll(left)));
        left &= ~mine;
        todo |= turn == share ? mine : 0;
    }
    taken |= todo;
    const bool write_total = kJoin && x.c0 == 0 && share == 0;
    if (!taken && !write_total)
        return;
    int32_t row[4], id[4];
    bool wanted[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        row[i] = __builtin_amdgcn_ds_bpermute((g * 4 + i) * 4, u_row);
        id[i] = __builtin_amdgcn_ds_bpermute((g * 4 + i) * 4, u_id);
        wanted[i] = taken >> (g * 4 + i) & 1;
    }
    typename X::piece b[4];
    x.load_base(a.base, row, wanted, b);
    Frag u[X::kSteps];
    if constexpr (kJoin) {
        const float s = u_id >= 0 ? a.scale[u_id] : 0.0f;
#pragma unroll
        for (int k = 0; k < PS; ++k) {
            f32x4 v0 = {0, 0, 0, 0}, v1 = {0, 0, 0, 0};
            if (u_row >= 0 && x.in[k] && (write_total || (todo >> m & 1))) {
                const float *p = a.sums + (int64_t)u_row * x.rank + x.chunk[k];
                v0 = *(const f32x4 *)p;
                v1 = *(const f32x4 *)(p + 4);
                for (int32_t q = 1; q < a.splits; ++q) {
                    p += (int64_t)a.r.rows * x.rank;
                    v0 += *(const f32x4 *)p;
                    v1 += *(const f32x4 *)(p + 4);
                }
                if (write_total) {
                    float *o = a.total + (int64_t)u_row * x.rank + x.chunk[k];
                    *(f32x4 *)o = v0;
                    *(f32x4 *)(o + 4) = v1;
                }
            }
            v0 *= s;
            v1 *= s;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t hi, lo;
                split2(j < 2 ? v0[2 * j] : v1[2 * j - 4], j < 2 ? v0[2 * j + 1] : v1[2 * j - 3], &hi, &lo);
                if (kHalf) {
                    u[0].w[j] = g < 2 ? hi : lo;
                } else {
                    u[k].w[j] = hi;
                    u[PS + k].w[j] = lo;
                }
            }
        }
    } else {
        x.load_parts(a.parts, blockIdx.y, u);
    }
    f32x4 res[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t)
        res[t] = f32x4{0, 0, 0, 0};
    while (todo) {
        const int32_t cur = __builtin_amdgcn_readlane(u_id, __builtin_ctzll(todo));
        Frag wf[PS][CT];
        x.load_w(a.w.first + cur * a.w.stride, wf);
        todo &= ~ballot(u_id == cur);
        bool mine[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mine[i] = id[i] == cur;
        x.product(wf, u, mine, res);
    }
    x.store(a.y, row, id, wanted, b, res);
}

// ---------------------------------------------------------------------------
// wgrad
// ---------------------------------------------------------------------------

struct WgradArgs {
    AdRows r;  // order: the plan's
    const int32_t *off, *keep;
    int32_t rank, in_dim, out_dim, chunk, nchunks, blocks_a, accumulate;
    int64_t stride, a_off, b_off;
    const uint16_t *t_du, *t_u;  // as adapter_prep_kernel leaves them
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

// T tiles of 16 of the rank against 16 CT columns a wave.  blockIdx.x: columns
// of x (dA), then of dy (dB); blockIdx.y: a chunk of positions, whole steps of 32.
// Positions of a step that belong to another adapter are zeros in both operands.
// The sums of an adapter whose rows lie in one chunk go to their place, those of a
// longer one to a slot of the workspace: chunk + adapter, which no two pieces
// share, since from one piece to the next the chunk or the adapter grows and
// neither falls.
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
    const uint16_t *pp = (is_a ? a.t_du : a.t_u) + lane * 8;
    const int64_t window = (int64_t)rank * (a.in_dim + a.out_dim);
    int32_t p = (int32_t)blockIdx.y * a.chunk;
    const int32_t p_end = rows - p < a.chunk ? rows : p + a.chunk;

    while (p < p_end) {
        const int32_t row = a.r.order[p];
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

        f32x4 acc[T][CT];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int c = 0; c < CT; ++c)
                acc[t][c] = f32x4{0, 0, 0, 0};

        // The rows of the step at `at` (a multiple of 32); those outside [p, end)
        // are some row inside.
        auto rows_of = [&](int32_t at, int32_t (&r)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int32_t pos = at + g * 8 + j;
                const int32_t i = a.r.order[pos < p || pos >= end ? p : pos];
                r[j] = (uint32_t)i < (uint32_t)rows ? i : 0;
            }
        };
        auto load_q = [&](const int32_t (&r)[8], Halves<CT> (&q)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                q[j] = load_halves<CT>(qp + (int64_t)r[j] * D);
        };
        auto step = [&](int32_t at, Halves<CT> (&q)[8]) {
            const uint16_t *f = pp + (int64_t)(at / kStep) * 3 * T * 512;
            const int32_t lo = p - at - g * 8, hi = end - at - g * 8;  // positions of this lane's 8
            const bool edge = at < p || at + kStep > end;
            if (edge) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        q[j].h[c] = j >= lo && j < hi ? q[j].h[c] : 0;
            }
            Frag qf[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    qf[c].w[j] = (uint32_t)q[2 * j].h[c] | (uint32_t)q[2 * j + 1].h[c] << 16;
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int b = 0; b < 3; ++b) {
                    Frag pf;
                    pf.v = *(const bf16x8 *)(f + (b * T + t) * 512);
                    if (edge) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            pf.h[j] = j >= lo && j < hi ? pf.h[j] : 0;
                    }
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        acc[t][c] = mfma16(pf.v, qf[c].v, acc[t][c]);
                }
        };
        int32_t at = p / kStep * kStep, r[8];
        Halves<CT> q[8], q2[8];
        rows_of(at, r);
        load_q(r, q);
        if (at + kStep < end)
            rows_of(at + kStep, r);
        for (; at < end; at += kStep) {
            if (at + kStep < end)
                load_q(r, q2);
            if (at + 2 * kStep < end)
                rows_of(at + 2 * kStep, r);
            step(at, q);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                q[j] = q2[j];
        }

        const int32_t ch = (int32_t)blockIdx.y;
        const bool direct = first / a.chunk == (first + cnt - 1) / a.chunk;
        const bool add = direct && a.accumulate;
        float *o = direct ? a.d_bank + e * a.stride + (is_a ? a.a_off : a.b_off)
                          : a.part + (ch + e) * window + (is_a ? 0 : (int64_t)rank * a.in_dim);
        if (col < D) {
            // a lane's results: indexes 16 t + 4 g .. + 3 of the rank, CT columns
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const int32_t at_r = t * 16 + g * 4;
                if (at_r >= rank)
                    continue;
                if (is_a) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float *z = o + (int64_t)(at_r + i) * D + col;
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
                        f32x4 *z = (f32x4 *)(o + (int64_t)(col + c) * rank + at_r);
                        *z = add ? *z + acc[t][c] : acc[t][c];
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

// Parts of a contraction over workgroups: until there are about 512.
int split_count(int32_t rows, int32_t D, int most)
{
    const bool few = rows <= kFewRows;
    const int64_t tiles = few ? (rows + 15) / 16 : ((int64_t)rows + 63) / 64;
    const int32_t steps = (D + 127) / 128;  // two stages, or a step a wave
    int64_t s = 512 / tiles;
    s = s < most ? s : most;
    s = s < steps ? s : steps;
    return (int)(s < 1 ? 1 : s);
}

// Tiles of 16 that a rank takes, a power of two.
int rank_tiles(int32_t rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }

// The kernel's dynamic-LDS limit raised to what it takes, once per device.
int raise_lds(const void *kernel, int bytes, bool (&raised)[64])
{
    int dev = 0;
    if (bytes <= 48 * 1024)
        return MOONEP_OK;
    if (hipGetDevice(&dev) != hipSuccess)
        return MOONEP_ERR_HIP;
    if (dev >= 0 && dev < 64 && raised[dev])
        return MOONEP_OK;
    if (hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) != hipSuccess)
        return MOONEP_ERR_HIP;
    if (dev >= 0 && dev < 64)
        raised[dev] = true;
    return MOONEP_OK;
}

template <int T, bool kNN>
int shrink_as(const ShrinkArgs &a, int splits, hipStream_t st)
{
    const int32_t rows = a.r.rows;
    if (rows <= kFewRows) {
        hipLaunchKernelGGL((shrink_few_kernel<T, kNN>), dim3((rows + 15) / 16, splits, 4), dim3(kAdBlock), 0,
                           st, a);
        return MOONEP_OK;
    }
    using G = ShrinkCfg<T, kNN>;
    static bool raised[64] = {};
    if (raise_lds((const void *)shrink_kernel<T, kNN>, G::kLds, raised) != MOONEP_OK)
        return MOONEP_ERR_HIP;
    hipLaunchKernelGGL((shrink_kernel<T, kNN>), dim3((unsigned)(((int64_t)rows + 63) / 64), splits),
                       dim3(kAdBlock), G::kLds, st, a);
    return MOONEP_OK;
}

template <bool kNN>
int shrink(const ShrinkArgs &a, int splits, hipStream_t st)
{
    switch (rank_tiles(a.w.rank)) {
    case 1: return shrink_as<1, kNN>(a, splits, st);
    case 2: return shrink_as<2, kNN>(a, splits, st);
    case 4: return shrink_as<4, kNN>(a, splits, st);
    default: return shrink_as<8, kNN>(a, splits, st);
    }
}

void prepare(const PrepArgs &a, hipStream_t st)
{
    const size_t lds = a.t_u ? (size_t)2 * 3 * a.tiles * 512 * 2 : 0;
    hipLaunchKernelGGL(adapter_prep_kernel, dim3((unsigned)(((int64_t)a.r.rows + kStep - 1) / kStep)),
                       dim3(kAdBlock), lds, st, a);
}

template <int PS, bool kHalf, int CT, bool kNN>
int expand_as(ExpandArgs a, hipStream_t st)
{
    const int64_t tiles = ((int64_t)a.r.rows + 15) / 16;
    if (a.r.rows <= kFewRows) {
        const dim3 grid((unsigned)((a.w.D + 63) / 64), (unsigned)tiles, 4);
        if constexpr (!kNN) {
            if (a.sums) {
                hipLaunchKernelGGL((expand_few_kernel<PS, kHalf, 4, kNN, true>), grid, dim3(kAdBlock), 0, st, a);
                return MOONEP_OK;
            }
        }
        hipLaunchKernelGGL((expand_few_kernel<PS, kHalf, 4, kNN, false>), grid, dim3(kAdBlock), 0, st, a);
        return MOONEP_OK;
    }
    const int64_t blocks = (a.w.D + 64 * CT - 1) / (64 * CT);
    int64_t per = tiles * blocks / 1024;
    per = per < 1 ? 1 : (per > 32 ? 32 : per);
    while ((tiles + per - 1) / per > 65535)
        per *= 2;
    a.tiles = (int32_t)per;
    using G = ExpandRing<PS, kHalf, CT>;
    static bool raised[64] = {};
    if (raise_lds((const void *)expand_kernel<PS, kHalf, CT, kNN>, G::kLds, raised) != MOONEP_OK)
        return MOONEP_ERR_HIP;
    hipLaunchKernelGGL((expand_kernel<PS, kHalf, CT, kNN>),
                       dim3((unsigned)blocks, (unsigned)((tiles + per - 1) / per)), dim3(kAdBlock), G::kLds,
                       st, a);
    return MOONEP_OK;
}

template <bool kNN>
int expand(const ExpandArgs &a, hipStream_t st)
{
    switch (rank_tiles(a.w.rank)) {
    case 1: return expand_as<1, true, 8, kNN>(a, st);
    case 2: return expand_as<1, false, 8, kNN>(a, st);
    case 4: return expand_as<2, false, 8, kNN>(a, st);
    default: return expand_as<4, false, 4, kNN>(a, st);
    }
}

template <int T, int CT>
void wgrad_as(WgradArgs a, hipStream_t st)
{
    a.blocks_a = (a.in_dim + 64 * CT - 1) / (64 * CT);
    const int32_t blocks = a.blocks_a + (a.out_dim + 64 * CT - 1) / (64 * CT);
    hipLaunchKernelGGL((wgrad_kernel<T, CT>), dim3(blocks, a.nchunks), dim3(kAdBlock), 0, st, a);
}

// Consecutive arrays of the workspace, each at a multiple of 256 bytes.
struct Carve {
    char *at;
    template <class X>
    X *take(size_t n)
    {
        at = (char *)(((uintptr_t)at + 255) & ~(uintptr_t)255);
        X *p = (X *)at;
        at += n * sizeof(X);
        return p;
    }
};

size_t steps_of(int64_t rows) { return (size_t)((rows + kStep - 1) / kStep); }

}  // namespace

namespace {

// Elements of expand's parts, and of one of wgrad's arrays.
size_t parts_size(int64_t rows, int32_t rank) { return (size_t)((rows + 15) / 16) * Parts(rank).steps() * 512; }
size_t turned_size(int64_t rows, int32_t rank) { return steps_of(rows) * 3 * rank_tiles(rank) * 512; }

}  // namespace

size_t adapter_workspace(int64_t rows, const moonep_adapters &ad)
{
    // partial sums and the parts: 4 splits rank + 64 steps bytes a row, at most 64
    // rank for every rank (rank 8: 448 + 64; 72: 4032 + 512), and 15 rows more of parts
    return (size_t)rows * ad.rank * 64 + 65536;
}

size_t adapter_bwd_workspace(int64_t rows, const moonep_adapters &ad)
{
    // partial sums, the parts and wgrad's two arrays (192 bytes a row for each tile of
    // the rank): at most 68 rank for every rank (rank 8: 256 + 64 + 192), and up to 31
    // rows more; the pieces of the gradients take the place of the sums
    return (size_t)rows * ad.rank * 68 +
           (size_t)(kMostChunks + ad.n) * ad.rank * ((size_t)ad.in_dim + ad.out_dim) * 4 + 65536;
}

int launch_adapter(int32_t rows, const moonep_adapters &ad, const int32_t *ids, const int32_t *order,
                   const uint16_t *x, const uint16_t *bank, const float *scale, const uint16_t *base,
                   float *u, uint16_t *y, void *ws, hipStream_t st)
{
    if (rows == 0)
        return MOONEP_OK;
    const AdRows r{ids, order, rows, ad.n};
    const bool few = rows <= kFewRows;
    const int splits = split_count(rows, ad.in_dim, kMostSplits);
    Carve carve{(char *)ws};
    float *sums = splits > 1 || few ? carve.take<float>((size_t)splits * rows * ad.rank) : u;
    uint16_t *parts = few ? nullptr : carve.take<uint16_t>(parts_size(rows, ad.rank));
    const bool ready = !few && splits == 1;  // shrink makes the parts itself
    const int rc = shrink<false>(ShrinkArgs{r, {bank + ad.a_offset, ad.stride, ad.rank, ad.in_dim}, x,
                                            ready ? scale : nullptr, sums, ready ? parts : nullptr},
                                 splits, st);
    if (rc != MOONEP_OK)
        return rc;
    if (!few && !ready)
        prepare(PrepArgs{r, scale, ad.rank, rank_tiles(ad.rank), splits, sums, u, parts, 1, nullptr, nullptr,
                         nullptr}, st);
    if (expand<false>(ExpandArgs{r, {bank + ad.b_offset, ad.stride, ad.rank, ad.out_dim}, parts, base, y, 0,
                                 few ? sums : nullptr, u, scale, splits}, st) != MOONEP_OK)
        return MOONEP_ERR_HIP;
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
    const size_t plane = (size_t)rows * ad.rank, turned = d_bank ? turned_size(rows, ad.rank) : 0;
    Carve carve{(char *)ws};
    uint16_t *parts = carve.take<uint16_t>(dx ? parts_size(rows, ad.rank) : 0);
    uint16_t *t_du = carve.take<uint16_t>(turned);
    uint16_t *t_u = carve.take<uint16_t>(turned);
    if (rows) {
        const int splits = split_count(rows, ad.out_dim, kMostSplitsBwd);
        Carve sums = carve;  // done with before the gradients' pieces are made
        float *du = sums.take<float>(splits * plane);
        const int rc = shrink<true>(ShrinkArgs{r, {bank + ad.b_offset, ad.stride, ad.rank, ad.out_dim}, dy,
                                               scale, du, nullptr}, splits, st);
        if (rc != MOONEP_OK)
            return rc;
        prepare(PrepArgs{r, scale, ad.rank, rank_tiles(ad.rank), splits, du, nullptr, dx ? parts : nullptr, 0,
                         u, d_bank ? t_du : nullptr, d_bank ? t_u : nullptr}, st);
        if (dx && expand<true>(ExpandArgs{r, {bank + ad.a_offset, ad.stride, ad.rank, ad.in_dim}, parts,
                                          dx_base, dx, 0, nullptr, nullptr, nullptr, 0}, st) != MOONEP_OK)
            return MOONEP_ERR_HIP;
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
        a.t_du = t_du;
        a.t_u = t_u;
        a.x = x;
        a.dy = dy;
        const int64_t window = (int64_t)ad.rank * ((int64_t)ad.in_dim + ad.out_dim);
        a.part = carve.take<float>((size_t)(kMostChunks + ad.n) * window);
        a.d_bank = d_bank;
        // chunks of at least 128 positions, 64 at most, for about 512 workgroups
        const int32_t width = ad.rank <= 32 ? 512 : 256, blocks = (ad.in_dim + ad.out_dim + width - 1) / width;
        int32_t chunks = 512 / blocks;
        chunks = chunks < 1 ? 1 : (chunks > kMostChunks ? kMostChunks : chunks);
        int64_t chunk = ((int64_t)rows + chunks - 1) / chunks;
        chunk = (chunk + kStep - 1) / kStep * kStep;
        chunk = chunk < 128 ? 128 : chunk;
        a.chunk = (int32_t)chunk;
        a.nchunks = (int32_t)(((int64_t)rows + chunk - 1) / chunk);
        if (rows) {
            if (ad.rank <= 16)
                wgrad_as<1, 8>(a, st);
            else if (ad.rank <= 32)
                wgrad_as<2, 8>(a, st);
            else if (ad.rank <= 64)
                wgrad_as<4, 4>(a, st);
            else
                wgrad_as<8, 4>(a, st);
        }
        const int64_t nb = (window + kAdBlock * 4 - 1) / (kAdBlock * 4);
        hipLaunchKernelGGL(wgrad_join_kernel, dim3((unsigned)(nb < 128 ? nb : 128), ad.n), dim3(kAdBlock),
                           0, st, a);
    }
    return status();
}

}  // namespace moonep
