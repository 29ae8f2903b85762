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
// Parts of a contraction over workgroups, and chunks of rows of the gradients, that the
// workspaces have room for.
constexpr int kMostSplits = 14, kMostSplitsBwd = 8;
constexpr int kMostChunks = 64;
// Workgroups that share a tile's adapters (us with 1, 4 and 8: 16 rows of 16 adapters
// 12.6, 11.8, 11.8; 1531 rows of 24: 24.0, 17.1, 17.1; 32768 rows in prompts of 800: 191,
// 183, 183).
constexpr unsigned kShares = 4;

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

// Bits of the first bf16 part of a, whose nearest bf16 has bits `near`: that, but a's upper
// half where a is finite and the nearest is not (from 255.5 2^120 on).
__device__ __forceinline__ uint32_t first_part(float a, uint32_t near)
{
    return (near & 0x7FFF) == 0x7F80 ? __float_as_uint(a) >> 16 : near;
}

// Two bf16 parts of a pair of values, packed: 16 bits of each.  The second part
// of an infinity is 0.
__device__ __forceinline__ void split2(float a, float b, uint32_t *hi, uint32_t *lo)
{
    const uint32_t near = pack_bf16(a, b);
    const uint32_t h = first_part(a, near & 0xFFFF) | first_part(b, near >> 16) << 16;
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
    __host__ __device__ explicit Parts(int32_t rank)
        : per(rank <= 16 ? 2 : rank <= 32 ? 4 : rank <= 64 ? 8 : 16)
    {
    }
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

// kStream: non-temporal, for rows that `streams` says go past the caches.
template <bool kStream = false>
__device__ __forceinline__ void dma16(const void *src, char *dst)
{
    __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void *)dst, 16, 0,
                                     kStream ? 2 : 0);
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
// LDS stages of 64 values of the contraction, filled by LDS-DMA.  The matrix's stage is
// [16 T][64], or with kNN what memory has: 64 rows of rank.  blockIdx.y is one of
// gridDim.y parts of the contraction.  Of a tile's adapters each of gridDim.z
// workgroups has every gridDim.z-th, with their rows, and those without one end at
// once: a tile at the border of two would otherwise take twice as long as all
// others, and the launch with it.  They come last, so that the tiles with one adapter
// start without them, and LDS is left for them.
// Bound by memory: 32768 x 4096 rows in 44 us (6.1 TB/s) against rank 16, 75 against
// eight adapters of rank 64; stages of 128 values, 128 positions and deeper rings were
// no faster.
template <int T, bool kNN, int S>
struct ShrinkCfg {
    static constexpr int kRows = 64, kK = 64, kRowBytes = 2 * kK;
    static constexpr int kStageX = kRows * kRowBytes, kStageW = 16 * T * kRowBytes;
    static constexpr int kStageBytes = kStageX + kStageW;
    static constexpr int kXInstr = kStageX / 4096;          // loads of a wave for the stage's rows
    static constexpr int kWInstr = kStageW < 4096 ? 1 : kStageW / 4096;  // and for its matrix
    static constexpr int kPerStage = kXInstr + kWInstr;
    static constexpr int kLds = S * kStageBytes;
    // 16-byte chunk c of row r of a stage sits at c ^ swz(r): rows of 128 bytes share the
    // banks by two
    __device__ static constexpr int swz(int r) { return r / 2 % 8; }
    // of kNN's matrix, for the rank that fills the tiles: a transposing read takes 32 bytes
    // of rows 4 j .. + 3 and of the rows 8 further, which would share their banks
    // (32768 rows, 4096 wide, rank 128: 146 us without it, 87 with it)
    __device__ static constexpr int swz_nn(int r)
    {
        return T == 1 ? 0 : (T == 8 ? (r & 3) << 2 : T == 4 ? (r >> 1 & 1) << 2 : 0) | (r >> 3 & 1) << 1;
    }
};

template <int T, bool kNN, int S, bool kStream>
__global__ __launch_bounds__(kAdBlock) void shrink_kernel(ShrinkArgs a)
{
    using G = ShrinkCfg<T, kNN, S>;
    extern __shared__ __align__(16) char ring[];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int m = lane & 15, g = lane >> 4;
    const int32_t D = a.w.D, rank = a.w.rank;
    const uint32_t share = blockIdx.z, shares = gridDim.z;
    const int64_t p0 = (int64_t)blockIdx.x * G::kRows;
    const int32_t steps = (D + G::kK - 1) / G::kK;
    const int32_t k0 = (int32_t)((int64_t)steps * blockIdx.y / gridDim.y);
    const int32_t nk = (int32_t)((int64_t)steps * (blockIdx.y + 1) / gridDim.y) - k0;

    // every position of the workgroup, the same in every wave
    const int32_t id_all = a.r.id(a.r.row(p0 + lane));
    uint64_t todo = 0, left = ballot(id_all >= 0), taken = share ? 0 : ~left;
    for (uint32_t turn = 0; left; turn = turn + 1 == shares ? 0 : turn + 1) {
        const uint64_t same = ballot(id_all == __builtin_amdgcn_readlane(id_all, __builtin_ctzll(left)));
        left &= ~same;
        todo |= turn == share ? same : 0;
    }
    taken |= todo;
    if (!taken)
        return;
    // Neighbours on an XCD begin 512 bytes apart and go round: rows of a power of two
    // bytes, all read at one column, would keep few of the memory's channels busy
    // (32768 x 4096, rank 16, begun alike: 54 us for 44).
    const int32_t begin = nk ? (int32_t)(blockIdx.x / 8 * (256 / G::kK) % nk) : 0;
    // this lane's chunk and row, of its wave's loads of a stage of rows
    const uint16_t *xp[G::kXInstr];
    int xc[G::kXInstr];
#pragma unroll
    for (int v = 0; v < G::kXInstr; ++v) {
        const int r = ((v * 4 + wave) * 64 + lane) / 8;
        const int32_t row = a.r.row(p0 + r);
        xc[v] = ((lane % 8) ^ G::swz(r)) * 8;
        xp[v] = a.x + (int64_t)(row < 0 ? 0 : row) * D + xc[v];
    }
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
        const int32_t kn = kNN ? rank / 8 : G::kStageW / 1024;  // KiB of the matrix's stage
        const uint16_t *wp[G::kWInstr];
        int wk[G::kWInstr];  // the value of the contraction that this lane's chunk begins at, in a stage
#pragma unroll
        for (int v = 0; v < G::kWInstr; ++v) {
            const int at = (v * 4 + wave) % kn * 64 + lane;  // waves without a load of their own repeat one
            if (kNN) {
                wk[v] = at * 8 / rank;
                wp[v] = w + (at ^ (rank == 16 * T ? G::swz_nn(wk[v]) : 0)) * 8;
            } else {
                const int r = at / 8;
                wk[v] = ((at % 8) ^ G::swz(r)) * 8;
                wp[v] = w + (int64_t)(r < rank ? r : 0) * D + wk[v];
            }
        }
        auto issue = [&](int32_t kt, int st) {
            char *to = ring + st * G::kStageBytes;
            const int32_t k = (k0 + (kt + begin < nk ? kt + begin : kt + begin - nk)) * G::kK;
#pragma unroll
            for (int v = 0; v < G::kXInstr; ++v)
                dma16<kStream>(k + xc[v] < D ? (const void *)(xp[v] + k) : kZeros,
                               to + (v * 4 + wave) * 1024);
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
        for (int st = 0; st + 1 < S; ++st)
            if (st < nk)
                issue(st, st);
        const bool mine = ballot(id == cur) != 0;
        int now = 0;
        for (int32_t kt = 0; kt < nk; ++kt) {
            if (kt + S - 2 < nk)
                wait_vm<(S - 2) * G::kPerStage>();
            else
                wait_vm<0>();
            lds_barrier();  // the stage is visible to all, the one before is free
            if (kt + S - 1 < nk)
                issue(kt + S - 1, now ? now - 1 : S - 1);
            const char *x = ring + now * G::kStageBytes, *ws = x + G::kStageX;
            now = now + 1 == S ? 0 : now + 1;
            if (!mine)
                continue;
#pragma unroll
            for (int ks = 0; ks < G::kK / 32; ++ks) {
                Frag xf, wf[T];
                const int chunk = ((ks * 4 + g) ^ G::swz(m)) << 4;
                xf.v = *(const bf16x8 *)(x + (wave * 16 + m) * G::kRowBytes + chunk);
                if constexpr (kNN) {
                    const uint32_t at =
                        (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char *)ws +
                        (ks * 32 + g * 8 + (m >> 2)) * rank * 2 + (m & 3) * 8;
                    const int sw = rank == 16 * T ? G::swz_nn(g * 8 + (m >> 2)) * 16 : 0;
                    constexpr int N = T < 4 ? T : 4;
#pragma unroll
                    for (int t = 0; t < T; t += N) {
                        uint32_t lo[N], hi[N];
                        Frag f[N];
#pragma unroll
                        for (int q = 0; q < N; ++q) {
                            lo[q] = at + ((t + q) * 32 ^ sw);
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
                        wf[t].v = *(const bf16x8 *)(ws + (t * 16 + m) * G::kRowBytes + chunk);
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
    if (row < 0 || !(taken >> (wave * 16 + m) & 1))
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

// Few rows: 16 positions a workgroup, operands straight into registers.  The
// waves share the rows, each with a part of the contraction, of which blockIdx.y
// is one of gridDim.y parts; their sums are joined in LDS.  Of a tile's
// adapters, workgroup blockIdx.z has every gridDim.z-th, and their rows.  The 16
// rows of the instruction's tile t are indexes m T + t of the rank, so that a
// lane's results are 4 T consecutive ones.  Bound by latency (16 rows of 16
// adapters, 2048 wide, rank 16: 5.5 us of a kernel, 6.6 with the adapters one after
// the other).
template <int T, bool kNN, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void shrink_few_kernel(ShrinkArgs a)
{
    constexpr int U = T <= 4 ? 4 : 2;  // steps in flight
    const int lane = lane_id(), wave = (int)threadIdx.x >> 6;
    const int m = lane & 15, g = lane >> 4;
    const int32_t D = a.w.D, rank = a.w.rank;
    const int64_t pos = (int64_t)blockIdx.x * 16 + m;
    const int32_t steps = (D + 31) / 32;
    const int32_t cuts = (int32_t)gridDim.y * WAVES, cut = (int32_t)blockIdx.y * WAVES + wave;
    const int32_t k0 = (int32_t)((int64_t)steps * cut / cuts);
    const int32_t k1 = (int32_t)((int64_t)steps * (cut + 1) / cuts);
    const int32_t full = k1 < D / 32 ? k1 : D / 32;  // steps before this have all 32

    const int32_t row = a.r.row(pos), id = a.r.id(row);
    const uint16_t *xp = a.x + (int64_t)(row < 0 ? 0 : row) * D + g * 8;
    const int32_t r0 = m * T < rank ? m * T : 0;  // lanes past the rank repeat index 0: not stored
    uint64_t todo = ballot(id >= 0), store = blockIdx.z == 0 ? ballot(row >= 0 && id < 0) : 0;
    f32x4 res[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
        res[t] = f32x4{0, 0, 0, 0};

    for (uint32_t turn = 0; todo; turn = turn + 1 == gridDim.z ? 0 : turn + 1) {
        const int32_t cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        const uint64_t mine = ballot(id == cur);
        todo &= ~mine;
        if (turn != blockIdx.z)
            continue;
        store |= mine;
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
        f32x4 acc[T];
#pragma unroll
        for (int t = 0; t < T; ++t)
            acc[t] = f32x4{0, 0, 0, 0};
        int32_t k = k0;
        for (; k + U <= full; k += U) {
            Frag x[U], f[U][T];
#pragma unroll
            for (int u = 0; u < U; ++u)
                x[u].v = *(const bf16x8 *)(xp + (k + u) * 32);
#pragma unroll
            for (int u = 0; u < U; ++u)
                load_w(k + u, f[u]);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int t = 0; t < T; ++t)
                    acc[t] = mfma16(f[u][t].v, x[u].v, acc[t]);
        }
        for (; k < k1; ++k) {
            // the last step may end inside: chunks past D are zeros in both operands
            Frag x{}, f[T]{};
            if (k * 32 + g * 8 < D) {
                x.v = *(const bf16x8 *)(xp + k * 32);
                load_w(k, f);
            }
#pragma unroll
            for (int t = 0; t < T; ++t)
                acc[t] = mfma16(f[t].v, x.v, acc[t]);
        }
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                res[t][j] = id == cur ? acc[t][j] : res[t][j];
    }

    __shared__ f32x4 join[WAVES][T][64];
#pragma unroll
    for (int t = 0; t < T; ++t)
        join[wave][t][lane] = res[t];
    __syncthreads();
    if (wave || !(store >> lane & 1))
        return;
    const float s = id >= 0 && a.scale ? a.scale[id] : 1.0f;
    const Parts parts(rank);
    float v[4 * T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
        f32x4 sum = join[0][t][lane];
#pragma unroll
        for (int q = 1; q < WAVES; ++q)
            sum += join[q][t][lane];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j * T + t] = a.parts ? sum[j] : sum[j] * s;
    }
    float *o = a.out + ((int64_t)blockIdx.y * a.r.rows + row) * rank;
#pragma unroll
    for (int q = 0; q < T; ++q) {
        const int32_t c = g * 4 * T + q * 4;
        if (c >= rank)
            continue;
        const f32x4 part = {v[q * 4], v[q * 4 + 1], v[q * 4 + 2], v[q * 4 + 3]};
        *(f32x4 *)(o + c) = part;
        if (a.parts)
            parts.put(a.parts, pos, c, part * s);
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
    const uint32_t hi = first_part(a, pack_bf16(a, 0.0f) & 0xFFFF);
    const float h = bf16_lo(hi);
    const float r = __builtin_isfinite(h) ? a - h : 0.0f;
    const uint32_t mid = pack_bf16(r, 0.0f);
    *p0 = (uint16_t)hi;
    *p1 = (uint16_t)mid;
    *p2 = (uint16_t)pack_bf16(r - bf16_lo(mid), 0.0f);
}

// One workgroup: 32 positions and 32 values of the rank, 4 a thread.
__global__ __launch_bounds__(kAdBlock) void adapter_prep_kernel(PrepArgs a)
{
    // both arrays' step and two tiles, as they leave
    __shared__ __align__(16) uint16_t turned[2][3][2 * 512];
    const int p = (int)threadIdx.x & 31, part = (int)threadIdx.x >> 5;
    const int32_t rank = a.rank, c = (int32_t)blockIdx.y * 32 + part * 4;
    const int64_t pos = (int64_t)blockIdx.x * kStep + p;
    const int32_t row = a.r.row(pos), id = a.r.id(row);
    const float s = id >= 0 ? a.scale[id] : 0.0f, by = a.scale_parts ? s : 1.0f;
    if (c < rank) {
        f32x4 v = {0, 0, 0, 0}, w = {0, 0, 0, 0};
        if (id >= 0) {
            const float *q = a.sums + (int64_t)row * rank + c;
            v = *(const f32x4 *)q;
            if (a.t_u)
                w = *(const f32x4 *)(a.u + (int64_t)row * rank + c) * s;
#pragma unroll 4
            for (int32_t i = 1; i < a.splits; ++i)
                v += *(const f32x4 *)(q + i * ((int64_t)a.r.rows * rank));
        }
        if (row >= 0 && a.total)
            *(f32x4 *)(a.total + (int64_t)row * rank + c) = v;
        if (row >= 0 && a.parts)
            Parts(rank).put(a.parts, pos, c, v * by);
        if (a.t_u) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = part * 4 + j, at = (r / 16 * 64 + p / 8 * 16 + r % 16) * 8 + p % 8;
                split3(v[j], &turned[0][0][at], &turned[0][1][at], &turned[0][2][at]);
                split3(w[j], &turned[1][0][at], &turned[1][1][at], &turned[1][2][at]);
            }
        }
    }
    if (!a.t_u)
        return;
    __syncthreads();
    const int tiles = a.tiles < 2 ? 1 : 2;
    for (int i = (int)threadIdx.x; i < 2 * 3 * tiles * 64; i += kAdBlock) {
        const int chunk = i % (tiles * 64), b = i / (tiles * 64);  // array and part
        u32x4 *to = (u32x4 *)(b < 3 ? a.t_sum : a.t_u) +
                    (((int64_t)blockIdx.x * 3 + b % 3) * a.tiles + blockIdx.y * 2) * 64;
        to[chunk] = ((const u32x4 *)turned[b / 3][b % 3])[chunk];
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
        for (int s = 0; s < kSteps; ++s)
            f[s].v = *(const bf16x8 *)(parts + ((tile * kSteps + s) * 64 + lane_id()) * 8);
    }
    // Zeros for chunks past the rank, where the parts hold nothing.
    __device__ __forceinline__ void mask_parts(Frag (&f)[kSteps]) const
    {
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                f[s].w[j] = in[kHalf ? 0 : s % PS] ? f[s].w[j] : 0;
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
    // Whether the wave holds a NaN: a maximum that is one if any value is (32768 x 4096 rows,
    // rank 8 to 64, the whole call: 175 to 199 us without the question, 176 to 200.5 with it).
    __device__ __forceinline__ bool any_nan(const f32x4 (&res)[CT]) const
    {
        float m = 0.0f;
#pragma unroll
        for (int t = 0; t < CT; t += 2)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, res[t][i]), res[t + 1][i]);
        return ballot(__builtin_isnan(m)) != 0;
    }
    // For rows that any_nan holds of, once they are stored.  A value's second part may be 0
    // or of the first's other sign, so that an infinite weight makes a NaN of the two: there
    // the first part alone gives what the value itself does.
    __device__ __forceinline__ void store_nans_again(const Frag (&w)[PS][CT], const Frag (&u)[kSteps],
                                                     const bool (&mine)[4], const int32_t (&row)[4],
                                                     const piece (&b)[4], uint16_t *y) const
    {
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            f32x4 both = {0, 0, 0, 0}, first = {0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                both = mfma16(u[s].v, w[kHalf ? 0 : s % PS][t].v, both);
#pragma unroll
            for (int s = 0; s < PS; ++s) {
                Frag uf = u[s], wf = w[s][t];
#pragma unroll
                for (int j = 0; kHalf && j < 4; ++j) {  // zeros in both for lanes of the second
                    uf.w[j] = lane_id() < 32 ? uf.w[j] : 0;
                    wf.w[j] = lane_id() < 32 ? wf.w[j] : 0;
                }
                first = mfma16(uf.v, wf.v, first);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (mine[i] && col < D && __builtin_isnan(both[i])) {
                    const float base = t % 2 ? bf16_hi(b[i][t / 2]) : bf16_lo(b[i][t / 2]);
                    y[(int64_t)row[i] * D + col + t] = (uint16_t)pack_bf16(base + first[i], 0.0f);
                }
            __builtin_amdgcn_sched_barrier(0);  // one tile after the other, for registers
        }
    }
    // A row without an adapter is copied bit for bit.
    template <bool kStream>
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
                const uint32_t v = pack_bf16(bf16_lo(b[i][t / 2]) + res[t][i],
                                             bf16_hi(b[i][t / 2]) + res[t + 1][i]);
                o[t / 2] = id[i] >= 0 ? v : b[i][t / 2];
            }
            piece *to = (piece *)(y + (int64_t)row[i] * D + col);
            if constexpr (kStream)
                __builtin_nontemporal_store(o, to);
            else
                *to = o;
        }
    }
};

// Many rows: a wave keeps its columns of one adapter's matrix in registers and
// walks row tiles.  Bound by memory: 32768 x 4096 base rows and results in 98 us (5.5
// TB/s) up to rank 32, 112 at 64; at 128 in 168 forward and 178 backward, by the parts,
// which come from the L2 once for every 64 or 128 columns (64 in the backward: 279).
// Base rows come through the wave's own ring of LDS slots (so many bytes in flight would
// not fit the registers), requested kAhead tiles ahead, and parts one tile ahead into
// registers; no wave waits for another.  The parts enter the registers of the next tile
// behind a wait for everything requested, so a tile costs a round trip, which only the
// SIMD's other waves hide.
constexpr int kAhead = 2;
constexpr int kTileRun = 32;  // row tiles whose rows and adapters are looked up at once

template <int PS, bool kHalf, int CT>
struct ExpandRing {
    static constexpr int kSteps = kHalf ? 1 : 2 * PS;
    static constexpr int kLanesRow = 2 * CT;              // lanes, 16 bytes each, of a row
    static constexpr int kInstr = 16 * kLanesRow / 64;    // loads of a tile
    static constexpr int kSlot = 16 * CT * 32;
    static constexpr int kLds = 4 * (kAhead + 1) * kSlot;
    static_assert(kAhead * kInstr + kSteps <= 63, "outstanding accesses must fit vmcnt");
};

template <int PS, bool kHalf, int CT, bool kNN, bool kStream>
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
    const int64_t next = ((int64_t)blockIdx.y + 1) * a.tiles, last = next < tiles ? next : tiles;
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
            for (int v = 0; v < G::kInstr; ++v) {
                const int32_t row = t < n ? rows[t * 16 + (v * 64 + lane) / G::kLanesRow] : -1;
                dma16<kStream>(row >= 0 && c < x.D ? (const void *)(a.base + (int64_t)row * x.D + c)
                                                   : kZeros, to + v * 1024);
            }
        };
        Frag u[G::kSteps], u2[G::kSteps];
        x.load_parts(a.parts, first, u);
#pragma unroll
        for (int t = 0; t < kAhead; ++t)
            issue(t, t);
        int slot = 0;
        for (int32_t t = 0; t < n; ++t) {
            wave_sync();
            x.load_parts(a.parts, first + (t + 1 < n ? t + 1 : t), u2);
            issue(t + kAhead, slot ? slot - 1 : kAhead);
            // The tile's rows have landed once only what was issued after them is outstanding:
            // the rows of the kAhead tiles after it and one tile's parts (the first tile's
            // come before the ring is begun; later ones' stand between, and are needed now
            // as well).  Matrices and stores, which are not counted, only make it wait for more.
            wait_vm<kAhead * G::kInstr + G::kSteps>();
            asm volatile("" ::: "memory");
            const char *at = ring + slot * G::kSlot;
            slot = slot == kAhead ? 0 : slot + 1;
            int32_t row[4], id[4];
            piece b[4];
            bool left[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                row[i] = rows[t * 16 + g * 4 + i];
                id[i] = ids[t * 16 + g * 4 + i];
                left[i] = id[i] >= 0;
                b[i] = *(const piece *)(at + (g * 4 + i) * CT * 32 + (lane & 15) * CT * 2);
            }
            x.mask_parts(u);
            f32x4 res[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c)
                res[c] = f32x4{0, 0, 0, 0};
            // the next adapter of the rows left, its matrix and its rows; false if there is none
            bool mine[4];
            auto next_adapter = [&]() -> bool {
                int32_t cur = -1;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t some = ballot(left[i]);
                    if (cur < 0 && some)
                        cur = __builtin_amdgcn_readlane(id[i], __builtin_ctzll(some));
                }
                if (cur < 0)
                    return false;
                if (cur != have) {
                    have = cur;
                    x.load_w(a.w.first + cur * a.w.stride, wf);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mine[i] = id[i] == cur;
                    left[i] = left[i] && !mine[i];
                }
                return true;
            };
            while (next_adapter())
                x.product(wf, u, mine, res);
            bool wanted[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                wanted[i] = row[i] >= 0;
            const bool nan = x.any_nan(res);
            x.template store<kStream>(a.y, row, id, wanted, b, res);
            if (nan) {
                wait_vm<0>();
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    left[i] = id[i] >= 0;
                while (next_adapter())
                    x.store_nans_again(wf, u, mine, row, b, a.y);
            }
#pragma unroll
            for (int k = 0; k < G::kSteps; ++k)
                u[k] = u2[k];
        }
        wait_vm<0>();  // nothing is on its way into the LDS when it is given back
    }
}

// Few rows: the four waves of a workgroup, and `parts` of them, share a row tile and
// its 16 CT columns, each with some of the tile's adapters and their rows.
template <int PS, bool kHalf, int CT, bool kNN, bool kJoin>
__device__ __forceinline__ void expand_few(const ExpandArgs &a, uint32_t block, uint32_t tile, uint32_t part,
                                           uint32_t parts)
{
    using X = Expand<PS, kHalf, CT, kNN>;
    const int wave = (int)threadIdx.x >> 6, m = lane_id() & 15, g = lane_id() >> 4;
    const X x(a.w, (int32_t)block * 16 * CT);
    const uint32_t share = part * 4 + wave, shares = parts * 4;
    const int64_t p0 = (int64_t)tile * 16;
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
        f32x4 v[PS][2];
#pragma unroll
        for (int k = 0; k < PS; ++k)
            v[k][0] = v[k][1] = f32x4{0, 0, 0, 0};
        if (u_row >= 0 && (write_total || (todo >> m & 1))) {
            const float *p = a.sums + (int64_t)u_row * x.rank;
            // several parts' loads in flight (100 rows of 16 adapters, 4096 wide, rank 64, both
            // kernels: 18.6 us one after the other, 14.8)
#pragma unroll 4
            for (int32_t q = 0; q < a.splits; ++q, p += (int64_t)a.r.rows * x.rank)
#pragma unroll
                for (int k = 0; k < PS; ++k) {
                    v[k][0] += *(const f32x4 *)(p + x.chunk[k]);
                    v[k][1] += *(const f32x4 *)(p + x.chunk[k] + 4);
                }
        }
#pragma unroll
        for (int k = 0; k < PS; ++k) {
            if (u_row >= 0 && write_total && x.in[k]) {
                float *o = a.total + (int64_t)u_row * x.rank + x.chunk[k];
                *(f32x4 *)o = v[k][0];
                *(f32x4 *)(o + 4) = v[k][1];
            }
            const f32x4 v0 = x.in[k] ? v[k][0] * s : f32x4{0, 0, 0, 0};
            const f32x4 v1 = x.in[k] ? v[k][1] * s : f32x4{0, 0, 0, 0};
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
        x.load_parts(a.parts, tile, u);
        x.mask_parts(u);
    }
    f32x4 res[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t)
        res[t] = f32x4{0, 0, 0, 0};
    uint64_t again = todo;  // loops of their own: one for both took 0.3 of 6 us more
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
    const bool nan = x.any_nan(res);
    x.template store<false>(a.y, row, id, wanted, b, res);
    if (!nan)
        return;
    wait_vm<0>();
    while (again) {
        const int32_t cur = __builtin_amdgcn_readlane(u_id, __builtin_ctzll(again));
        Frag wf[PS][CT];
        x.load_w(a.w.first + cur * a.w.stride, wf);
        again &= ~ballot(u_id == cur);
        bool mine[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mine[i] = id[i] == cur;
        x.store_nans_again(wf, u, mine, row, b, a.y);
    }
}

template <int PS, bool kHalf, int CT>
__global__ __launch_bounds__(kAdBlock) void expand_few_kernel(ExpandArgs a)
{
    expand_few<PS, kHalf, CT, false, true>(a, blockIdx.x, blockIdx.y, blockIdx.z, gridDim.z);
}

// ---------------------------------------------------------------------------
// wgrad
// ---------------------------------------------------------------------------

struct WgradArgs {
    AdRows r;  // order: the plan's
    const int32_t *off, *keep;
    int32_t rank, tiles, in_dim, out_dim, chunk, nchunks, blocks_a, blocks, accumulate;
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

// One workgroup: T tiles of 16 of the rank against 256 columns, 64 a wave: of x (dA),
// then of dy (dB); `part` counts these blocks within groups of T tiles.  Of its chunk
// of positions, whole steps of 32, it has every shares-th adapter.  Rows and
// rank values come through a ring of LDS stages of one step, filled by LDS-DMA; the
// rows' fragments, 8 positions of one column, through the transposing read.
// Positions of a step that belong to another adapter are zeros in both operands.
// The sums of an adapter whose rows lie in one chunk go to their place, those of a
// longer one to a slot of the workspace: chunk + adapter, which no two pieces
// share, since from one piece to the next the chunk or the adapter grows and
// neither falls.
// Bound by memory, the rows being read once: 32768 rows, 4096 -> 4096, rank 16, in
// 93 to 102 us (5.3 to 5.8 TB/s); rank 128, where the matrix instructions' three
// products are 206 GFLOP, 251.  Deeper rings, and one sequence of stages over the
// pieces, were no faster.
constexpr int kGradCols = 256;
constexpr int kStepRun = 32;  // steps whose rows are looked up at once

template <int T, int S>
struct WgradCfg {
    static constexpr int kRow = kGradCols * 2, kStageQ = kStep * kRow, kStageP = 3 * T * 1024;
    static constexpr int kStageBytes = kStageQ + kStageP;
    static constexpr int kQInstr = kStageQ / 4096;      // loads of a wave
    static constexpr int kPInstr = (3 * T + 3) / 4;
    static constexpr int kPerStage = kQInstr + kPInstr;
    static constexpr int kLds = S * kStageBytes;
    // 16-byte chunk c of row r sits at c ^ swz(r): a transposing read takes 32 bytes of
    // rows 4 j .. + 3 and, with the neighbouring 16 lanes, of the rows 8 further
    __device__ static constexpr int swz(int r) { return (r & 3) << 2 | (r >> 3 & 1) << 1; }
};

// Whether a value of the wave's fragments is an infinity or a NaN: 0 times those is a NaN.
template <int N>
__device__ __forceinline__ bool any_not_finite(const Frag (&f)[N])
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    float sum[N] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int c = 0; c < N; ++c)
            sum[c] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, f[c].w[j]), bf16x2{0, 0}, sum[c],
                                                     false);
    float m = 0.0f;
#pragma unroll
    for (int c = 0; c < N; ++c)
        m = __builtin_elementwise_maximum(m, sum[c]);
    return ballot(__builtin_isnan(m)) != 0;
}

// A pair of bf16 with 0 in the place of infinities and NaN.
__device__ __forceinline__ uint32_t finite_or_0(uint32_t w)
{
    return ((w & 0x7F80) == 0x7F80 ? 0 : w & 0xFFFF) | ((w >> 16 & 0x7F80) == 0x7F80 ? 0 : w & 0xFFFF0000);
}

template <int T, int S, bool kStream>
__device__ __forceinline__ void wgrad(const WgradArgs &a, uint32_t part, uint32_t chunk, uint32_t share,
                                      uint32_t shares, char *ring)
{
    using G = WgradCfg<T, S>;
    const int32_t block = (int32_t)part % a.blocks, tile0 = (int32_t)part / a.blocks * T;
    __shared__ int32_t row_of[kStepRun * kStep], id_of[kStepRun * kStep];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int m = lane & 15, g = lane >> 4;
    const bool is_a = block < a.blocks_a;
    const int32_t D = is_a ? a.in_dim : a.out_dim, rank = a.rank, rows = a.r.rows;
    const int32_t c0 = (block - (is_a ? 0 : a.blocks_a)) * kGradCols;
    const uint16_t *q = is_a ? a.x : a.dy;
    const uint16_t *t_p = is_a ? a.t_du : a.t_u;
    const int64_t window = (int64_t)rank * (a.in_dim + a.out_dim);
    const int32_t p_begin = (int32_t)chunk * a.chunk;
    const int32_t p_end = rows - p_begin < a.chunk ? rows : p_begin + a.chunk;

    // this lane's row of a step and chunk, of its wave's loads; columns past D are
    // not stored
    int q_row[G::kQInstr];
    int32_t q_col[G::kQInstr];
#pragma unroll
    for (int v = 0; v < G::kQInstr; ++v) {
        const int at = (v * 4 + wave) * 64 + lane;
        q_row[v] = at / (G::kRow / 16);
        q_col[v] = c0 + ((at % (G::kRow / 16)) ^ G::swz(q_row[v])) * 8;
    }
    // LDS address of tile 0's fragment in stage 0: rows 8 g + m / 4 and four further;
    // tile c of the wave is at ^ (c / 2 << 6) ^ (c % 2 << 5)
    const uint32_t q_at = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char *)ring +
                          (g * 8 + (m >> 2)) * G::kRow +
                          (((wave * 2) ^ (m >> 2)) << 6 | (g & 1) << 5 | (m & 3) << 3);

    f32x4 acc[T][4];
    int32_t held = -1, cnt = 0, first = 0;  // the adapter whose sums these are, and its rows
    auto put = [&]() {
        const int32_t ch = (int32_t)chunk;
        const bool direct = cnt && first / a.chunk == ch && (first + cnt - 1) / a.chunk == ch;
        const bool add = direct && a.accumulate;
        float *o = direct ? a.d_bank + held * a.stride + (is_a ? a.a_off : a.b_off)
                          : a.part + (ch + held) * window + (is_a ? 0 : (int64_t)rank * a.in_dim);
        // a lane's results: indexes 16 t + 4 g .. + 3 of the rank, column m of each tile
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int32_t at_r = (tile0 + t) * 16 + g * 4;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int32_t col = c0 + wave * 64 + c * 16 + m;
                if (at_r >= rank || col >= D)
                    continue;
                if (is_a) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float *z = o + (int64_t)(at_r + i) * D + col;
                        *z = add ? *z + acc[t][c][i] : acc[t][c][i];
                    }
                } else {
                    f32x4 *z = (f32x4 *)(o + (int64_t)col * rank + at_r);
                    *z = add ? *z + acc[t][c] : acc[t][c];
                }
            }
        }
    };

    int32_t r0 = p_begin - kStepRun * kStep, n = 0;  // the run
    int32_t end = 0;                                 // of the piece before
    uint32_t piece = 0;
    for (;;) {
        // the next piece that is this workgroup's: positions [p, end) of the run, of one adapter
        int32_t p, id = -1;
        for (;;) {
            if (end >= n) {
                r0 += kStepRun * kStep;
                if (r0 >= p_end)
                    break;
                n = p_end - r0 < kStepRun * kStep ? p_end - r0 : kStepRun * kStep;
                end = 0;
                __syncthreads();  // the run before is done with the ring and the tables
                for (int32_t i = (int)threadIdx.x; i < (n + kStep - 1) / kStep * kStep; i += kAdBlock) {
                    const int32_t row = i < n ? a.r.row(r0 + i) : -1;
                    row_of[i] = row;
                    id_of[i] = a.r.id(row);
                }
                __syncthreads();
            }
            p = end;
            id = __builtin_amdgcn_readfirstlane(id_of[p]);
            uint64_t other = 0;
            for (; !other; end += 64) {
                const int32_t i = end + lane;
                other = ballot(i >= n || id_of[i < n ? i : 0] != id);
            }
            end += __builtin_ctzll(other) - 64;
            if (id >= 0 && piece++ % shares == share)
                break;
            id = -1;
        }
        if (held >= 0 && id != held)
            put();
        if (id < 0)
            break;
        if (id != held) {
            held = id;
            cnt = adapter_rows(a.off, a.keep, held, rows, &first);
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    acc[t][c] = f32x4{0, 0, 0, 0};
        }
        const int32_t s0 = p / kStep, steps = (end + kStep - 1) / kStep - s0;
        auto issue = [&](int32_t t, int slot) {
            char *to = ring + slot * G::kStageBytes;
#pragma unroll
            for (int v = 0; v < G::kQInstr; ++v) {
                const int32_t pos = (s0 + t) * kStep + q_row[v];
                const int32_t r = pos >= p && pos < end ? row_of[pos] : -1;
                dma16<kStream>(r >= 0 && q_col[v] < D ? (const void *)(q + (int64_t)r * D + q_col[v])
                                                      : kZeros, to + (v * 4 + wave) * 1024);
            }
            const uint16_t *src = t_p + ((int64_t)(r0 / kStep + s0 + t) * 3 * a.tiles + tile0) * 512 + lane * 8;
#pragma unroll
            for (int v = 0; v < G::kPInstr; ++v) {
                const int i = (v * 4 + wave) % (3 * T);  // waves without a load of their own repeat one
                dma16(src + (i / T * a.tiles + i % T) * 512, to + G::kStageQ + i * 1024);
            }
        };
        lds_barrier();  // the piece before is done with the ring
#pragma unroll
        for (int t = 0; t + 1 < S; ++t)
            if (t < steps)
                issue(t, t);
        int now = 0;
        for (int32_t t = 0; t < steps; ++t) {
            if (t + S - 2 < steps)
                wait_vm<(S - 2) * G::kPerStage>();
            else
                wait_vm<0>();
            lds_barrier();  // the stage is visible to all, the one before is free
            if (t + S - 1 < steps)
                issue(t + S - 1, now ? now - 1 : S - 1);
            const char *stage = ring + now * G::kStageBytes;
            Frag qf[4];
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                lo[c] = (q_at ^ (uint32_t)(c / 2 << 6 | c % 2 << 5)) + now * G::kStageBytes;
                hi[c] = lo[c] + 4 * G::kRow;
            }
            now = now + 1 == S ? 0 : now + 1;
            tr_frags<4>(lo, hi, qf);
            const int32_t at = (s0 + t) * kStep;
            const int32_t from = p - at - g * 8, to = end - at - g * 8;  // of this lane's 8 positions
            uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};
            if (at < p || at + kStep > end) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    keep[j] = (2 * j >= from && 2 * j < to ? 0xFFFFu : 0) |
                              (2 * j + 1 >= from && 2 * j + 1 < to ? 0xFFFF0000u : 0);
            }
            // The later parts of a rank value may be 0 or of the first's other sign: with an
            // infinite value of a row they would make a NaN.  They meet 0 in its place (the whole
            // call on 32768 rows, 4096 -> 4096: no slower up to rank 64, 581 -> 592 us at 128).
            const bool not_all = any_not_finite(qf);
#pragma unroll
            for (int b = 0; b < 3; ++b) {
                if (b == 1 && not_all)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            qf[c].w[j] = finite_or_0(qf[c].w[j]);
#pragma unroll
                for (int k = 0; k < T; ++k) {
                    Frag pf;
                    pf.v = *(const bf16x8 *)(stage + G::kStageQ + (b * T + k) * 1024 + lane * 16);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        pf.w[j] &= keep[j];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[k][c] = mfma16(pf.v, qf[c].v, acc[k][c]);
                }
            }
        }
    }
    if (a.nchunks > 1 || a.accumulate)
        return;
    // no adapter has rows in several chunks, and no join follows: those without any get
    // their zeros here
    const int32_t cols = D - c0 < kGradCols ? D - c0 : kGradCols;
    const int32_t i0 = tile0 * 16, i1 = rank - i0 < T * 16 ? rank : i0 + T * 16;
    for (int32_t e0 = 0; e0 < a.r.n; e0 += 64) {
        const int32_t e = e0 + lane;
        uint64_t empty = ballot(e < a.r.n && (uint32_t)e % shares == share &&
                                adapter_rows(a.off, a.keep, e < a.r.n ? e : 0, rows, &first) == 0);
        for (; empty; empty &= empty - 1) {
            float *o = a.d_bank + (e0 + __builtin_ctzll(empty)) * a.stride + (is_a ? a.a_off : a.b_off);
            if (is_a) {
                if ((int32_t)threadIdx.x < cols)
                    for (int32_t i = i0; i < i1; ++i)
                        o[(int64_t)i * D + c0 + threadIdx.x] = 0.0f;
            } else {
                for (int32_t i = (int)threadIdx.x; i < cols * T * 4; i += kAdBlock) {
                    const int32_t at_r = i0 + i % (T * 4) * 4;
                    if (at_r < i1)
                        *(f32x4 *)(o + (int64_t)(c0 + i / (T * 4)) * rank + at_r) = f32x4{0, 0, 0, 0};
                }
            }
        }
    }
}

template <int T, int S, bool kStream>
__global__ __launch_bounds__(kAdBlock) void wgrad_kernel(WgradArgs a)
{
    extern __shared__ __align__(16) char ring[];
    wgrad<T, S, kStream>(a, blockIdx.x, blockIdx.y, blockIdx.z, gridDim.z, ring);
}

// Few rows: the gradients and the rows of d_x in one launch, which they share by
// workgroups (200 rows of 16 adapters, 4096 -> 4096, rank 16, 28.7 -> 24.9 us with
// the join left out as well; 55 of 20, 840 -> 104, rank 32: 23.3 -> 19.0).
template <int PS, bool kHalf, int CT, int T, int S>
__global__ __launch_bounds__(kAdBlock) void few_grads_kernel(WgradArgs a, ExpandArgs e, uint32_t parts,
                                                             uint32_t shares, uint32_t dx_blocks, uint32_t dx_parts)
{
    extern __shared__ __align__(16) char ring[];
    const uint32_t each = parts * a.nchunks;
    if (blockIdx.x < each * shares) {
        wgrad<T, S, false>(a, blockIdx.x % parts, blockIdx.x / parts % a.nchunks, blockIdx.x / each, shares, ring);
        return;
    }
    const uint32_t i = blockIdx.x - each * shares, tile = i / dx_blocks;
    expand_few<PS, kHalf, CT, true, false>(e, i % dx_blocks, tile / dx_parts, tile % dx_parts, dx_parts);
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
#pragma unroll 4
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

// Rows for which the kernels for few are taken: 256, up to which a narrower limit is
// slower (200 rows, 4096 wide, rank 64, backward: 44 us for 50), or 1024 of narrow ones.
// 16 adapters, us of the other kernels and of these, by rows x width of both sides:
//   forward, rank 16: 300 x 4096: 17.6, 13.2   500 x 2048: 13.7, 11.4   1000 x 4096: 20, 23
//   rank 64: 300 x 4096: 26.5, 24.6   1000 x 1024: 21, 16   500 x 4096: 27, 32
//   backward, rank 16: 300 x 4096: 31.5, 28.7   700 x 2048: 32, 27   500 x 4096: 33, 36
//   rank 128: 500 x 1024: 71, 58   700 x 2048: 94, 77   1000 x 4096: 136, 167.
bool few_rows(int32_t rows, const moonep_adapters &ad)
{
    return rows <= 256 || (rows <= 1024 && rows * ((int64_t)ad.in_dim + ad.out_dim) <= 3 << 20);
}

// Whether rows are read or written past the caches (non-temporal accesses): more than
// half of what the 256 MiB memory-side cache holds, of which the next call finds little there.
// 32768 rows, 4096 wide: forward of rank 64 202 -> 183 us, backward of rank 16 295 -> 269.
// With a call that reads the result the forward of 131 MB (16000 rows, rank 32) takes 151
// us for 154, of 33 MB 48 for 47, of 10 MB 27.5 for 26.
bool streams(int64_t rows, int64_t row_bytes) { return rows * row_bytes > (int64_t)128 << 20; }

int status() { return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_ERR_HIP; }

// Rows that shrink, forward and up to rank 32, takes 16 a workgroup of eight waves, each
// with a part of the contraction: no sums over workgroups, and so one launch less.  In us
// without it and with it, by rows x width: 1531 x 2048, rank 32: 24, 17; 8000 x 1024,
// rank 8: 23, 20; 4000 x 2048, rank 32: 29, 27; past the limit 3000 x 4096, rank 32: 35,
// 41; 8000 x 4096, rank 16: 60, 63; rank 64, 300 x 4096: 25, 29.  The backward's order of
// the matrix: 47, 66.  (Few rows go first.)
bool some_rows(int32_t rows, int32_t D, int32_t rank)
{
    return rows <= 8192 && (int64_t)rows * D <= 1 << 23 && rank <= 32;
}

// Parts of a contraction over workgroups: about one workgroup per CU, or where there are
// more tiles two of them, as long as that is nearer to 640 (304 tiles, 3744 wide: 129
// us, undivided 145).  Twice as many at fewer tiles were no faster up to rank 64 (65
// tiles, the whole backward: 62, 64; 2000 rows, 4096 wide, rank 64: 36, 43); above,
// where a CU's one workgroup has little in flight, they are (186 tiles, 5440 wide, rank
// 128, the whole backward: 263, 230).  Each part writes sums of 4 rank bytes a row, so
// that there are at most D / (share rank) parts; few rows need the workgroups more.
int split_count(int32_t rows, bool few, int32_t D, int32_t rank, int32_t share, int most)
{
    const int64_t tiles = few ? (rows + 15) / 16 : ((int64_t)rows + 63) / 64;
    const int32_t steps = (D + 127) / 128;  // two stages, or a step a wave
    int64_t s = tiles <= 256 ? (rank > 64 ? 512 : 256) / tiles : (640 + tiles / 2) / tiles;
    if (!few && s > D / (share * rank))
        s = D / (share * rank);
    s = s < most ? s : most;
    s = s < steps ? s : steps;
    return (int)(s < 1 ? 1 : s);
}

// For that: the forward's next step reads the sums, the backward's their parts as well.
// Us without it, with 4 and with 8: 1000 rows, 4096 wide, rank 128: 54, 41, 41; 2000:
// 56, 56, 49; backward, 500 rows, 1024 wide, rank 128: 71, 72, 83.
constexpr int32_t kShare = 8, kShareBwd = 4;

// Tiles of 16 that a rank takes, a power of two.
int rank_tiles(int32_t rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }

// The kernel's dynamic-LDS limit raised to what it takes, once per device.
template <class Kernel>
int raise_lds(Kernel kernel, int bytes, bool (&raised)[64])
{
    int dev = 0;
    if (bytes <= 48 * 1024)
        return MOONEP_OK;
    if (hipGetDevice(&dev) != hipSuccess)
        return MOONEP_ERR_HIP;
    if (dev >= 0 && dev < 64 && raised[dev])
        return MOONEP_OK;
    if (hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
        hipSuccess)
        return MOONEP_ERR_HIP;
    if (dev >= 0 && dev < 64)
        raised[dev] = true;
    return MOONEP_OK;
}

enum Form { kFew, kSome, kMany };

template <int T, bool kNN>
void shrink_as(const ShrinkArgs &a, Form form, int splits, hipStream_t st)
{
    const int32_t rows = a.r.rows;
    if (form == kFew) {
        hipLaunchKernelGGL((shrink_few_kernel<T, kNN, 4>), dim3((rows + 15) / 16, splits, kShares),
                           dim3(256), 0, st, a);
        return;
    }
    if constexpr (T <= 2 && !kNN) {
        if (form == kSome) {
            hipLaunchKernelGGL((shrink_few_kernel<T, kNN, 8>), dim3((rows + 15) / 16, splits, kShares),
                               dim3(512), 0, st, a);
            return;
        }
    }
    constexpr int kS = T == 8 ? 2 : T == 4 ? 3 : 4;  // 40 to 48 KiB: three workgroups a CU
    using G = ShrinkCfg<T, kNN, kS>;
    static_assert(G::kLds <= 48 * 1024, "no raised limit");
    const dim3 grid((unsigned)(((int64_t)rows + G::kRows - 1) / G::kRows), splits, kShares);
    // the backward's rows are read again by the gradients
    if constexpr (!kNN) {
        if (streams(rows, 2 * (int64_t)a.w.D)) {
            hipLaunchKernelGGL((shrink_kernel<T, kNN, kS, true>), grid, dim3(kAdBlock), G::kLds, st, a);
            return;
        }
    }
    hipLaunchKernelGGL((shrink_kernel<T, kNN, kS, false>), grid, dim3(kAdBlock), G::kLds, st, a);
}

template <bool kNN>
void shrink(const ShrinkArgs &a, Form form, int splits, hipStream_t st)
{
    switch (rank_tiles(a.w.rank)) {
    case 1: shrink_as<1, kNN>(a, form, splits, st); break;
    case 2: shrink_as<2, kNN>(a, form, splits, st); break;
    case 4: shrink_as<4, kNN>(a, form, splits, st); break;
    default: shrink_as<8, kNN>(a, form, splits, st);
    }
}

void prepare(const PrepArgs &a, hipStream_t st)
{
    hipLaunchKernelGGL(adapter_prep_kernel,
                       dim3((unsigned)(((int64_t)a.r.rows + kStep - 1) / kStep), (unsigned)(a.rank + 31) / 32),
                       dim3(kAdBlock), 0, st, a);
}

// Workgroups that share a few-rows tile and its columns, of `n` such (us with 4 and with
// one: 16 rows, 2048 wide, n = 32: 11.5, 12.1; 830 rows, 888 -> 2648, n = 2184: 30, 24).
uint32_t few_parts(uint32_t n) { return n <= 512 ? 4 : 1; }

template <int PS, bool kHalf, int CT, bool kNN>
void expand_as(ExpandArgs a, Form form, hipStream_t st)
{
    const int64_t tiles = ((int64_t)a.r.rows + 15) / 16;
    if constexpr (!kNN) {
        if (form == kFew) {
            const uint32_t few_blocks = (uint32_t)(a.w.D + 63) / 64;
            hipLaunchKernelGGL((expand_few_kernel<PS, kHalf, 4>),
                               dim3(few_blocks, (unsigned)tiles, few_parts(few_blocks * (uint32_t)tiles)),
                               dim3(kAdBlock), 0, st, a);
            return;
        }
    }
    const int64_t blocks = (a.w.D + 64 * CT - 1) / (64 * CT);
    // two workgroups per CU, all at once (32768 rows, 4096 wide, rank 64, the whole call:
    // 183 us; one per CU 222, four 208), or three with one tile each (4099 rows, 2048 wide,
    // the whole backward: 64.0 us, 62.5)
    int64_t per = tiles * blocks <= 768 ? 1 : (tiles * blocks + 511) / 512;
    per = per < (tiles + 65534) / 65535 ? (tiles + 65534) / 65535 : per;
    a.tiles = (int32_t)(per < tiles ? per : tiles);
    per = a.tiles;
    using G = ExpandRing<PS, kHalf, CT>;
    static_assert(G::kLds <= 48 * 1024, "no raised limit");
    const dim3 grid((unsigned)blocks, (unsigned)((tiles + per - 1) / per));
    if (streams(a.r.rows, 2 * (int64_t)a.w.D))
        hipLaunchKernelGGL((expand_kernel<PS, kHalf, CT, kNN, true>), grid, dim3(kAdBlock), G::kLds, st, a);
    else
        hipLaunchKernelGGL((expand_kernel<PS, kHalf, CT, kNN, false>), grid, dim3(kAdBlock), G::kLds, st, a);
}

template <bool kNN>
void expand(const ExpandArgs &a, Form form, hipStream_t st)
{
    switch (rank_tiles(a.w.rank)) {
    case 1: expand_as<1, true, 8, kNN>(a, form, st); break;
    case 2: expand_as<1, false, 8, kNN>(a, form, st); break;
    case 4: expand_as<2, false, 8, kNN>(a, form, st); break;
    default: expand_as<4, false, kNN ? 8 : 4, kNN>(a, form, st);
    }
}

// Column blocks times groups of T tiles of the rank.
uint32_t wgrad_parts(const WgradArgs &a, int T)
{
    return (uint32_t)(a.blocks * ((a.rank + 16 * T - 1) / (16 * T)));
}

// Workgroups for a chunk: about as many as it has adapters, 32 at most, while the launch
// is small (55 rows, 20 adapters, 840 -> 104, rank 32: the whole backward 61 -> 24 us; us
// with at most 16, 32 and 64: 361 rows of 129 adapters: 46, 39, 38; 200 of 200, 2048
// wide: 53, 49, 68); one where a chunk is more than one run, whose pieces may go on.
uint32_t wgrad_shares(const WgradArgs &a, uint32_t parts)
{
    const int64_t room = 2048 / ((int64_t)parts * a.nchunks);
    int64_t shares = a.r.n / a.nchunks + 1;
    shares = shares < 32 ? shares : 32;
    shares = shares < room ? shares : room;
    return shares < 1 || a.chunk > kStepRun * kStep ? 1 : (uint32_t)shares;
}

// Tiles of the rank that a workgroup takes: those there are, up to four (32768 rows, rank
// 128, the whole call: 496 us, with two 544, with all eight 60 more than with four; rank
// 64: 312, two 359), and fewer where that leaves less than a workgroup per CU (us with 4, 2 and 1 tiles: 1237
// rows, 536 -> 304, rank 128: 47, 41, 39; 97 rows of 102 adapters, 80 -> 2840, rank 32: -,
// 32, 27; but 500 rows of 16, 1024 wide, rank 128: 46, 49, 56).
int wgrad_tiles(const WgradArgs &a)
{
    int T = a.tiles < 4 ? a.tiles : 4;
    for (; T > 1; T /= 2) {
        const uint32_t parts = wgrad_parts(a, T);
        if ((int64_t)parts * a.nchunks * wgrad_shares(a, parts) >= 256)
            break;
    }
    return T;
}

template <int T, bool kStream>
int wgrad_as(const WgradArgs &a, hipStream_t st)
{
    using G = WgradCfg<T, 2>;
    static bool raised[64] = {};
    if (raise_lds(wgrad_kernel<T, 2, kStream>, G::kLds, raised) != MOONEP_OK)
        return MOONEP_ERR_HIP;
    const uint32_t parts = wgrad_parts(a, T);
    hipLaunchKernelGGL((wgrad_kernel<T, 2, kStream>), dim3(parts, a.nchunks, wgrad_shares(a, parts)), dim3(kAdBlock),
                       G::kLds, st, a);
    return MOONEP_OK;
}

template <bool kStream>
int wgrad_of(const WgradArgs &a, int T, hipStream_t st)
{
    switch (T) {
    case 1: return wgrad_as<1, kStream>(a, st);
    case 2: return wgrad_as<2, kStream>(a, st);
    default: return wgrad_as<4, kStream>(a, st);
    }
}

template <int PS, bool kHalf, int T>
int few_grads_as(const WgradArgs &a, const ExpandArgs &e, hipStream_t st)
{
    using G = WgradCfg<T, 2>;
    static bool raised[64] = {};
    if (raise_lds(few_grads_kernel<PS, kHalf, 4, T, 2>, G::kLds, raised) != MOONEP_OK)
        return MOONEP_ERR_HIP;
    const uint32_t parts = wgrad_parts(a, T), shares = a.d_bank ? wgrad_shares(a, parts) : 0;
    const uint32_t dx_blocks = e.y ? (uint32_t)(e.w.D + 63) / 64 : 0;
    const uint32_t tiles = (uint32_t)(e.r.rows + 15) / 16, dx_parts = few_parts(dx_blocks * tiles);
    hipLaunchKernelGGL((few_grads_kernel<PS, kHalf, 4, T, 2>),
                       dim3(parts * a.nchunks * shares + dx_blocks * tiles * dx_parts), dim3(kAdBlock),
                       shares ? G::kLds : 0, st, a, e, parts, shares, dx_blocks, dx_parts);
    return MOONEP_OK;
}

template <int PS, bool kHalf, int most>
int few_grads(const WgradArgs &a, const ExpandArgs &e, hipStream_t st)
{
    const int T = a.d_bank ? wgrad_tiles(a) : 1;
    if constexpr (most >= 4) {
        if (T == 4)
            return few_grads_as<PS, kHalf, 4>(a, e, st);
    }
    if constexpr (most >= 2) {
        if (T == 2)
            return few_grads_as<PS, kHalf, 2>(a, e, st);
    }
    return few_grads_as<PS, kHalf, 1>(a, e, st);
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
    template <class X>
    X *at_end() const  // the rest, for an array whose size is not counted on
    {
        return Carve(*this).take<X>(0);
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
    const bool few = few_rows(rows, ad);
    const Form form = few ? kFew : some_rows(rows, ad.in_dim, ad.rank) ? kSome : kMany;
    const int splits = form == kSome ? 1 : split_count(rows, few, ad.in_dim, ad.rank, kShare, kMostSplits);
    Carve carve{(char *)ws};
    float *sums = splits > 1 || few ? carve.take<float>((size_t)splits * rows * ad.rank) : u;
    uint16_t *parts = few ? nullptr : carve.take<uint16_t>(parts_size(rows, ad.rank));
    const bool ready = !few && splits == 1;  // shrink makes the parts itself
    shrink<false>(ShrinkArgs{r, {bank + ad.a_offset, ad.stride, ad.rank, ad.in_dim}, x,
                             ready ? scale : nullptr, sums, ready ? parts : nullptr},
                  form, splits, st);
    if (!few && !ready)
        prepare(PrepArgs{r, scale, ad.rank, rank_tiles(ad.rank), splits, sums, u, parts, 1, nullptr, nullptr,
                         nullptr}, st);
    expand<false>(ExpandArgs{r, {bank + ad.b_offset, ad.stride, ad.rank, ad.out_dim}, parts, base, y, 0,
                             sums, u, scale, splits}, form, st);
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
    const size_t turned = d_bank ? turned_size(rows, ad.rank) : 0;
    Carve carve{(char *)ws};
    uint16_t *parts = carve.take<uint16_t>(dx ? parts_size(rows, ad.rank) : 0);
    uint16_t *t_du = carve.take<uint16_t>(turned);
    uint16_t *t_u = carve.take<uint16_t>(turned);
    const bool few = few_rows(rows, ad);
    const ExpandArgs e{r, {bank + ad.a_offset, ad.stride, ad.rank, ad.in_dim}, parts, dx_base, dx, 0,
                       nullptr, nullptr, nullptr, 0};
    WgradArgs a{};
    if (d_bank) {
        const PlanLayout pl = plan_layout(E, 1);
        a.r = r;
        a.off = plan + pl.home_row_off;
        a.keep = plan + pl.keep;
        a.rank = ad.rank;
        a.tiles = rank_tiles(ad.rank);
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
        a.part = carve.at_end<float>();
        a.d_bank = d_bank;
        a.blocks_a = (ad.in_dim + kGradCols - 1) / kGradCols;
        const int32_t blocks = a.blocks = a.blocks_a + (ad.out_dim + kGradCols - 1) / kGradCols;
        // 64 chunks at most, for about 512 workgroups (32768 rows, 4096 -> 4096, the whole
        // call: 269 us; 256 of them 320, 1024 285), of at least 128 positions, and of 256
        // where that leaves 256 workgroups: most adapters' rows then lie in one chunk (4099
        // rows of 32 adapters, 2048 -> 1408: 62 -> 56; 2249 of 24, 88 -> 88: 56, 60 with
        // 256).  Few rows of many adapters are one chunk, as one run: their sums need no
        // joining (rank 128, 1024 wide, 1000 rows of 16: 72 -> 65, 500 of 2: 65, 66, 1000 of
        // one: 59, 93).
        int32_t chunks = 512 / blocks;
        chunks = chunks < 1 ? 1 : (chunks > kMostChunks ? kMostChunks : chunks);
        int64_t chunk = ((int64_t)rows + chunks - 1) / chunks;
        chunk = (chunk + kStep - 1) / kStep * kStep;
        int64_t least = (int64_t)rows * blocks / 256 / kStep * kStep;
        least = least < 128 ? 128 : least < 256 ? least : 256;
        if (few && (rows <= 256 || rows <= 64 * (int64_t)ad.n))
            least = kStepRun * kStep;
        chunk = chunk < least ? least : chunk;
        a.chunk = (int32_t)chunk;
        a.nchunks = (int32_t)(((int64_t)rows + chunk - 1) / chunk);
    }
    if (rows) {
        const int splits = split_count(rows, few, ad.out_dim, ad.rank, kShareBwd, kMostSplitsBwd);
        float *du = carve.at_end<float>();  // done with before the gradients' pieces are made
        shrink<true>(ShrinkArgs{r, {bank + ad.b_offset, ad.stride, ad.rank, ad.out_dim}, dy, scale, du,
                                nullptr}, few ? kFew : kMany, splits, st);
        prepare(PrepArgs{r, scale, ad.rank, rank_tiles(ad.rank), splits, du, nullptr, dx ? parts : nullptr, 0,
                         u, d_bank ? t_du : nullptr, d_bank ? t_u : nullptr}, st);
        int rc = MOONEP_OK;
        if (few) {
            switch (rank_tiles(ad.rank)) {
            case 1: rc = few_grads<1, true, 1>(a, e, st); break;
            case 2: rc = few_grads<1, false, 2>(a, e, st); break;
            case 4: rc = few_grads<2, false, 4>(a, e, st); break;
            default: rc = few_grads<4, false, 4>(a, e, st);
            }
        } else if (dx) {
            expand<true>(e, kMany, st);
        }
        if (!few && d_bank) {
            const int T = wgrad_tiles(a);
            // x and dy are read once where a workgroup has all of the rank
            const bool once = wgrad_parts(a, T) == (uint32_t)a.blocks;
            const int64_t D = ad.in_dim < ad.out_dim ? ad.in_dim : ad.out_dim;
            rc = once && streams(rows, 2 * D) ? wgrad_of<true>(a, T, st) : wgrad_of<false>(a, T, st);
        }
        if (rc != MOONEP_OK)
            return rc;
    }
    if (d_bank && a.nchunks != 1) {
        const int64_t window = (int64_t)ad.rank * ((int64_t)ad.in_dim + ad.out_dim);
        const int64_t nb = (window + kAdBlock * 4 - 1) / (kAdBlock * 4);
        const int64_t most = 2048 / ad.n > 128 ? 2048 / ad.n : 128;  // few adapters have more of them
        hipLaunchKernelGGL(wgrad_join_kernel, dim3((unsigned)(nb < most ? nb : most), ad.n), dim3(kAdBlock),
                           0, st, a);
    }
    return status();
}

}  // namespace moonep
