// gemm_bwd.hip -- the backward of the experts' products over the grouped
// buffer: the gradient of the rows and the gradients of the weights.
//
// With W(r) the [out, in] matrix of row r's segment (as in gemm.hip),
//   d_x[r, k]  = bf16( sum_n d_y[r, n] W(r)[n, k] )
//   g(s)[n, k] = (g(s)[n, k] +) sum over the rows r of segment s of
//                d_y[r, n] x[r, k], in fp32.
//
// Both walk the plan's segments with a persistent grid and a ring of LDS
// stages filled by LDS-DMA, as the forward product does, on the 32 x 32 x 16
// matrix instruction.  What differs is the memory order of the operands: the
// forward contracts over the contiguous axis of both, d_x over the rows of W,
// and g over the rows of both.  An operand whose contraction axis is the row
// stays as it is in memory in its stage, [BK rows][columns], and
// ds_read_b64_tr_b16 transposes on the way to the registers: 16 lanes read a
// block of 4 rows x 16 columns, 8 bytes each (lane s: row s / 4, columns 4 (s %
// 4) .. + 3), and lane d gets column d, rows 0 .. 3.  Two such reads make the 8
// values of k that a lane feeds to the instruction.  No transposed copy of the
// weights or the rows is written anywhere.
//
// Bank conflicts: the 32 lanes of half a wave read 4 rows x 64 bytes.  Stage
// rows are 256 or 512 bytes, a multiple of the 64 banks of 4 bytes, so the four
// would share 16 banks; the 64-byte piece p of row r is stored at piece
// p ^ (r % 4), which spreads them over all 64.
//
// Bounds, on 64 experts.  262144 rows, 2048 -> 1408: the matrix instructions, 1450 us
// (1.04 PFLOP/s; the pipe is busy 57% of the cycles in d_x and 62% in g, at 1.75 GHz,
// where loads and products share the power).  3904 rows, 1408 -> 2048: the weights'
// bytes in d_x (96 us, 4.1 TB/s) and the gradients' in g (170 us, 4.5 TB/s).
#include "segments.hpp"

namespace moonep {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

namespace {

// A lane's byte offset in a transposed stage of rows of RB bytes, for 32-column
// tile 0 and k-step 0; tile T is at offset ^ (T << 6), k-step ks at + ks 16 RB.
template <int RB>
__device__ __forceinline__ int tr_offset(int lane)
{
    const int row = (lane >> 5) * 8 + ((lane & 15) >> 2);
    return row * RB + ((row & 3) << 6) + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
}

// LDS byte address of a generic pointer into it.
__device__ __forceinline__ uint32_t lds_addr(const void *p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char *)p;
}

__device__ __forceinline__ bf16x8 join(s16x4 lo, s16x4 hi)
{
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The fragments at N LDS addresses, rows RB bytes apart.  In assembly, with its
// wait inside: before the builtin of this read the compiler waits for every
// LDS-DMA load in flight, the next stages' too, which leaves nothing to overlap.
template <int RB, int N>
__device__ __forceinline__ void tr_frags(const uint32_t (&at)[N], bf16x8 (&f)[N])
{
    static_assert(N == 2 || N == 4 || N == 6, "fragments a read");
    s16x4 r[2 * N];
    if constexpr (N == 2)
        asm volatile("ds_read_b64_tr_b16 %0, %4\n\t"
                     "ds_read_b64_tr_b16 %1, %4 offset:%6\n\t"
                     "ds_read_b64_tr_b16 %2, %5\n\t"
                     "ds_read_b64_tr_b16 %3, %5 offset:%6\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])
                     : "v"(at[0]), "v"(at[1]), "n"(4 * RB)
                     : "memory");
    else if constexpr (N == 4)
        asm volatile("ds_read_b64_tr_b16 %0, %8\n\t"
                     "ds_read_b64_tr_b16 %1, %8 offset:%12\n\t"
                     "ds_read_b64_tr_b16 %2, %9\n\t"
                     "ds_read_b64_tr_b16 %3, %9 offset:%12\n\t"
                     "ds_read_b64_tr_b16 %4, %10\n\t"
                     "ds_read_b64_tr_b16 %5, %10 offset:%12\n\t"
                     "ds_read_b64_tr_b16 %6, %11\n\t"
                     "ds_read_b64_tr_b16 %7, %11 offset:%12\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]),
                       "=&v"(r[6]), "=&v"(r[7])
                     : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(4 * RB)
                     : "memory");
    else
        asm volatile("ds_read_b64_tr_b16 %0, %12\n\t"
                     "ds_read_b64_tr_b16 %1, %12 offset:%18\n\t"
                     "ds_read_b64_tr_b16 %2, %13\n\t"
                     "ds_read_b64_tr_b16 %3, %13 offset:%18\n\t"
                     "ds_read_b64_tr_b16 %4, %14\n\t"
                     "ds_read_b64_tr_b16 %5, %14 offset:%18\n\t"
                     "ds_read_b64_tr_b16 %6, %15\n\t"
                     "ds_read_b64_tr_b16 %7, %15 offset:%18\n\t"
                     "ds_read_b64_tr_b16 %8, %16\n\t"
                     "ds_read_b64_tr_b16 %9, %16 offset:%18\n\t"
                     "ds_read_b64_tr_b16 %10, %17\n\t"
                     "ds_read_b64_tr_b16 %11, %17 offset:%18\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]),
                       "=&v"(r[6]), "=&v"(r[7]), "=&v"(r[8]), "=&v"(r[9]), "=&v"(r[10]), "=&v"(r[11])
                     : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "v"(at[4]), "v"(at[5]), "n"(4 * RB)
                     : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = join(r[2 * i], r[2 * i + 1]);
}

__device__ __forceinline__ void dma16(const char *src, char *dst)
{
    __builtin_amdgcn_global_load_lds((const void *)src,
                                     (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
}

template <bool kStream, class T>
__device__ __forceinline__ void put(T *p, T v)
{
    if constexpr (kStream)
        __builtin_nontemporal_store(v, p);
    else
        *p = v;
}

// Waits until at most N vector-memory operations of this wave are outstanding.
template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N >= 0 && N <= 63, "vmcnt");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

// A workgroup barrier that waits for this wave's LDS operations only: a
// __syncthreads would also wait for every load in flight.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
// d_x: rows of d_y against W, contracted over W's rows
// ---------------------------------------------------------------------------

// What the rows behind a segment's last are read as: zeros, so that they add
// nothing whatever the buffer holds there.
__device__ __align__(16) const uint32_t g_zero_row[4] = {0, 0, 0, 0};

template <int BM, int BN, int WM, int WN, int BK, int S>
struct DxCfg {
    static constexpr int kTM = WM / 32, kTN = WN / 32;
    static constexpr int kWM = BM / WM, kWN = BN / WN;
    static constexpr int kWavesG = kWM * kWN;
    static constexpr int kThreads = kWavesG * 64;
    static constexpr int kRowA = BK * 2, kRowB = BN * 2;  // bytes of a stage row
    static constexpr int kStageA = BM * kRowA, kStageB = BK * kRowB;
    static constexpr int kStageBytes = kStageA + kStageB;
    static constexpr int kAInstr = kStageA / 1024 / kWavesG, kBInstr = kStageB / 1024 / kWavesG;
    static constexpr int kPerStage = kAInstr + kBInstr;
    // The k-step whose reads the next stage's loads are issued behind: their address
    // arithmetic then runs under matrix instructions, and with more than two slots there
    // is time (256 x 256 tiles, four slots: 1515 -> 1490 us on the sweep).
    static constexpr int kIssueAt = S > 2 ? BK / 16 - 1 : 0;
    // Large tiles write d_x past the caches: it is 64 MiB at least where they are full, of
    // which the next call finds little there (sweep: 1478 -> 1457 us, and with a call that reads
    // it 277 -> 276 at 92 MB).  Narrow rows take them with less (14 MiB: 256 experts, 64
    // wide); that was not timed.
    static constexpr bool kStream = BM == 256;
    // Epilogue: each wave's own 16 rows of WN columns, apart from the ring, which
    // is loading the next item.
    static constexpr int kOutRow = WN * 2 + 16, kOutAt = S * kStageBytes;
    static constexpr int kPieces = WN / 8;  // 16-byte pieces of a row
    static constexpr int kOVec = 16 * kPieces / 64;
    static constexpr int kStores = kTM * 2 * kOVec;  // per wave and item
    static constexpr int kSegAt = kOutAt + kWavesG * 16 * kOutRow;
    static_assert(kStageA % (1024 * kWavesG) == 0 && kStageB % (1024 * kWavesG) == 0, "DMA rounds");
    static_assert(16 * kPieces % 64 == 0, "whole stores of 16 rows");
    // 16-byte chunk c of row r of the A part sits at c ^ swz(r), as in gemm.hip
    // (rows of 64 bytes share the banks by four, of 128 by two)
    __device__ static constexpr int swz(int r) { return BK == 64 ? r / 2 % 8 : r / 4 % 4; }
};

struct DxArgs {
    SegTables seg;
    int32_t in_dim, out_dim;
    const uint16_t *d_y, *w_home, *pool;
    int64_t w_stride, w_offset;
    uint16_t *d_x;
};

constexpr int kGroupM = 8;  // row tiles per item group, as in gemm.hip

template <int BM, int BN, int WM, int WN, int BK, int S>
__global__ __launch_bounds__((DxCfg<BM, BN, WM, WN, BK, S>::kThreads)) void expert_dx_kernel(DxArgs a)
{
    using G = DxCfg<BM, BN, WM, WN, BK, S>;
    extern __shared__ __align__(16) uint16_t lds[];
    char *ring = (char *)lds;
    int32_t *seg_start = (int32_t *)(ring + G::kSegAt);  // [E + cap + 1]
    __shared__ int scan_tmp[G::kWavesG];

    const int tid = (int)threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int32_t nseg = a.seg.E + a.seg.n_rep();
    const int32_t tiles = scan_tiles<BM, G::kWavesG>(a.seg, nseg, seg_start, scan_tmp);
    const int32_t nbn = (a.in_dim + BN - 1) / BN;  // the last block may be part-empty
    const int64_t items = (int64_t)tiles * nbn;
    const int P = (int)gridDim.x;
    const int64_t first = xcd_slot((int)blockIdx.x, P);
    if (first >= items)
        return;
    const int32_t nk = a.out_dim / BK;
    const int wm = wave / G::kWN, wn = wave % G::kWN;

    struct Item {
        int64_t m0;
        int32_t mrows, n0;
        const uint16_t *w;
    };
    auto locate = [&](int64_t it) -> Item {
        Item i;
        int32_t t, nb, len;
        item_of<kGroupM>(it, tiles, nbn, &t, &nb);
        const int32_t s = find_segment(seg_start, nseg, t);
        const int32_t mt = t - __builtin_amdgcn_readfirstlane(seg_start[s]);
        int64_t wrow;
        bool pooled;
        i.m0 = a.seg.segment(s, &len, &wrow, &pooled) + (int64_t)mt * BM;
        i.mrows = len - mt * BM < BM ? len - mt * BM : BM;
        i.n0 = nb * BN;
        i.w = (pooled ? a.pool : a.w_home) + wrow * a.w_stride + a.w_offset;
        return i;
    };

    // ---- the loads: the stages of all items in one sequence -------------------
    int64_t load_it = first;
    int32_t load_kt = 0;
    const char *a_base, *b_base;
    uint32_t a_off[G::kAInstr], b_off[G::kBInstr];
    auto begin_item = [&]() {
        const Item i = locate(load_it);
        a_base = (const char *)(a.d_y + i.m0 * a.out_dim);
        b_base = (const char *)(i.w + i.n0);
        // rows and columns past the end are not stored: the first serve them
#pragma unroll
        for (int v = 0; v < G::kAInstr; ++v) {
            const int row = ((v * G::kWavesG + wave) * 64 + lane) / (BK / 8);
            const int chunk = (lane % (BK / 8)) ^ G::swz(row);
            a_off[v] = (uint32_t)(row < i.mrows ? row : 0) * (uint32_t)a.out_dim * 2 + chunk * 16;
        }
#pragma unroll
        for (int v = 0; v < G::kBInstr; ++v) {
            constexpr int kCpr = G::kRowB / 16;
            const int at = (v * G::kWavesG + wave) * 64 + lane;
            const int row = at / kCpr, chunk = (at % kCpr) ^ ((row & 3) << 2);
            b_off[v] = (uint32_t)row * (uint32_t)a.in_dim * 2 + (i.n0 + chunk * 8 < a.in_dim ? chunk * 16 : 0);
        }
    };
    // Issues the next stage into slot `to`.  After the last item the loads go on
    // with zeros, which nobody computes: so every stage is followed by as many.
    auto issue = [&](int to) {
        if (load_kt == nk) {
            load_kt = 0;
            load_it += P;
            if (load_it < items)
                begin_item();
        }
        char *dst = ring + to * G::kStageBytes + wave * 1024;
        if (load_it >= items) {
#pragma unroll
            for (int v = 0; v < G::kPerStage; ++v)
                dma16((const char *)g_zero_row, dst + v * G::kWavesG * 1024);
            return;
        }
#pragma unroll
        for (int v = 0; v < G::kAInstr; ++v)
            dma16(a_base + a_off[v], dst + v * G::kWavesG * 1024);
#pragma unroll
        for (int v = 0; v < G::kBInstr; ++v)
            dma16(b_base + b_off[v], dst + G::kStageA + v * G::kWavesG * 1024);
        a_base += G::kRowA;
        b_base += (int64_t)BK * a.in_dim * 2;
        ++load_kt;
    };

    const int fr = lane & 31, fsw = G::swz(lane & 31), fhalf = lane >> 5;
    auto frag_a = [&](const char *base, int row0, int ks) -> bf16x8 {
        return *(const bf16x8 *)(base + (row0 + fr) * G::kRowA + (((2 * ks + fhalf) ^ fsw) << 4));
    };
    uint32_t b_at[G::kTN];
#pragma unroll
    for (int j = 0; j < G::kTN; ++j)
        b_at[j] = lds_addr(ring) + G::kStageA + (tr_offset<G::kRowB>(lane) ^ ((wn * G::kTN + j) << 6));
    char *mine = ring + G::kOutAt + wave * 16 * G::kOutRow;

    begin_item();
#pragma unroll
    for (int st = 0; st + 1 < S; ++st)
        issue(st);
    int now = 0;               // slot of the stage computed next; the ring runs on across items
    bool stores_ahead = false;  // behind the loads of this item's first stages, kStores were issued
    for (int64_t it = first; it < items; it += P) {
        const Item i = locate(it);
        f32x16 acc[G::kTM][G::kTN];
#pragma unroll
        for (int m = 0; m < G::kTM; ++m)
#pragma unroll
            for (int n = 0; n < G::kTN; ++n)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[m][n][r] = 0.0f;
        for (int32_t kt = 0; kt < nk; ++kt) {
            // This stage's loads have landed once only the S - 2 stages after it are
            // outstanding.  An item's first S - 1 were issued before the stores of the
            // item before: where all of those were issued, they need not be waited for.
            if (kt < S - 1 && stores_ahead)
                wait_vm<(S - 2) * G::kPerStage + G::kStores>();
            else
                wait_vm<(S - 2) * G::kPerStage>();
            lds_barrier();  // the stage is visible to all; the other slot is free
            const int free_slot = now ? now - 1 : S - 1;
            const char *sa = ring + now * G::kStageBytes;
#pragma unroll
            for (int ks = 0; ks < BK / 16; ++ks) {
                bf16x8 fa[G::kTM], fb[G::kTN];
                uint32_t at[G::kTN];
#pragma unroll
                for (int m = 0; m < G::kTM; ++m)
                    fa[m] = frag_a(sa, wm * WM + m * 32, ks);
#pragma unroll
                for (int n = 0; n < G::kTN; ++n)
                    at[n] = b_at[n] + now * G::kStageBytes + ks * 16 * G::kRowB;
                tr_frags<G::kRowB>(at, fb);
                if (ks == G::kIssueAt)
                    issue(free_slot);
                // W's columns as the instruction's rows: a lane's results are four
                // consecutive columns of one row of d_x
#pragma unroll
                for (int m = 0; m < G::kTM; ++m)
#pragma unroll
                    for (int n = 0; n < G::kTN; ++n)
                        acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[n], fa[m], acc[m][n], 0, 0, 0);
            }
            now = now + 1 == S ? 0 : now + 1;
        }
        // Epilogue: 16 rows at a time through the wave's own LDS, to whole lines.
        const bool full = i.mrows == BM && i.n0 + BN <= a.in_dim;
        stores_ahead = full;
#pragma unroll
        for (int m = 0; m < G::kTM; ++m)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if ((lane >> 4 & 1) == half) {
                    char *to = mine + (lane & 15) * G::kOutRow + (lane >> 5) * 8;
#pragma unroll
                    for (int n = 0; n < G::kTN; ++n)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            u32x2 v;
                            v[0] = pack_bf16(acc[m][n][4 * q], acc[m][n][4 * q + 1]);
                            v[1] = pack_bf16(acc[m][n][4 * q + 2], acc[m][n][4 * q + 3]);
                            *(u32x2 *)(to + n * 64 + q * 16) = v;
                        }
                }
                wave_sync();
#pragma unroll
                for (int v = 0; v < G::kOVec; ++v) {
                    const int idx = lane + v * 64, r = idx / G::kPieces, c = idx % G::kPieces;
                    const u32x4 piece = *(const u32x4 *)(mine + r * G::kOutRow + c * 16);
                    const int row = wm * WM + m * 32 + half * 16 + r, col = i.n0 + wn * WN + c * 8;
                    u32x4 *p = (u32x4 *)(a.d_x + (i.m0 + row) * a.in_dim + col);
                    if (full)
                        put<G::kStream>(p, piece);
                    else if (row < i.mrows && col < a.in_dim)
                        put<G::kStream>(p, piece);
                }
                wave_sync();
            }
    }
    wait_vm<0>();  // nothing is on its way into the LDS when it is given back
}

// ---------------------------------------------------------------------------
// g: both operands contracted over the segment's rows
// ---------------------------------------------------------------------------

template <int BM, int BN, int WM, int WN, int BK, int S>
struct DwCfg {
    static constexpr int kTM = WM / 32, kTN = WN / 32;
    static constexpr int kWM = BM / WM, kWN = BN / WN;
    static constexpr int kWavesG = kWM * kWN;
    static constexpr int kThreads = kWavesG * 64;
    static constexpr int kRowA = BM * 2, kRowB = BN * 2;
    static constexpr int kStageA = BK * kRowA, kStageB = BK * kRowB;
    static constexpr int kStageBytes = kStageA + kStageB;
    static constexpr int kAInstr = kStageA / 1024 / kWavesG, kBInstr = kStageB / 1024 / kWavesG;
    static constexpr int kPerStage = kAInstr + kBInstr;
    // Large tiles write the gradients past the caches: 80 MiB or more where they are full (64 of
    // 2048 x 1408, 3904 rows: 179 -> 175 us, without a call that reads them).  Narrow layers
    // take them with less (16 MiB: 512 experts, 64 -> 128); that was not timed.
    static constexpr bool kStream = BM == 256;
    static_assert(kStageA % (1024 * kWavesG) == 0 && kStageB % (1024 * kWavesG) == 0, "DMA rounds");
    static_assert(S >= 2 && (S - 2) * kPerStage <= 63, "outstanding loads must fit vmcnt");
};

struct DwArgs {
    SegTables seg;
    int32_t in_dim, out_dim, accumulate;
    const uint16_t *x, *d_y;
    int64_t G, g_offset;
    float *home, *rep;
};

template <int BM, int BN, int WM, int WN, int BK, int S>
__global__ __launch_bounds__((DwCfg<BM, BN, WM, WN, BK, S>::kThreads)) void expert_dw_kernel(DwArgs a)
{
    using G = DwCfg<BM, BN, WM, WN, BK, S>;
    extern __shared__ __align__(16) uint16_t lds[];
    char *ring = (char *)lds;
    const int tid = (int)threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int32_t nseg = a.seg.E + a.seg.n_rep();
    const int32_t nbm = (a.out_dim + BM - 1) / BM, nbn = (a.in_dim + BN - 1) / BN;
    const int64_t per = (int64_t)nbm * nbn, items = nseg * per;
    const int P = (int)gridDim.x, slot = xcd_slot((int)blockIdx.x, P);
    const int wm = wave / G::kWN, wn = wave % G::kWN;

    // The segments from the longest to the shortest (of equals the lower first):
    // each one's place is the number of those before it.
    int32_t *length = (int32_t *)(ring + S * G::kStageBytes);  // [nseg, padded to 4]
    int32_t *by_length = length + (nseg + 3) / 4 * 4;          // [nseg]
    for (int32_t i = tid; i < (nseg + 3) / 4 * 4; i += G::kThreads)
        length[i] = i < nseg ? a.seg.rows(i) : -1;
    __syncthreads();
    for (int32_t i = tid; i < nseg; i += G::kThreads) {
        const int32_t mine = length[i];
        int32_t place = 0;
        for (int32_t j = 0; j < nseg; j += 4) {
            const i32x4 o = *(const i32x4 *)(length + j);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                place += o[q] > mine || (o[q] == mine && j + q < i);
        }
        by_length[place] = i;
    }
    __syncthreads();

    // Rounds of P items, every other one backwards, so that whoever has a
    // round's longest item has the next one's shortest.
    const int64_t rounds = (items + P - 1) / P;
    struct Item {
        int32_t s, len, m0, n0;
    };
    auto locate = [&](int64_t round, Item *w) -> bool {
        const int64_t it = round * P + (round & 1 ? P - 1 - slot : slot);
        if (it >= items)
            return false;
        const int32_t at = (int32_t)(it / per), within = (int32_t)(it - at * per);
        w->s = __builtin_amdgcn_readfirstlane(by_length[at]);
        w->len = __builtin_amdgcn_readfirstlane(length[w->s]);
        w->m0 = within % nbm * BM;
        w->n0 = within / nbm * BN;
        return true;
    };

    // ---- the loads: the stages of all items in one sequence -------------------
    struct Load {
        int64_t round;
        int32_t left;  // rows from the next stage's first on
        const char *a_base, *b_base;
        uint32_t a_off[G::kAInstr], b_off[G::kBInstr];
    } ld;
    auto a_row = [&](int v) { return ((v * G::kWavesG + wave) * 64 + lane) / (G::kRowA / 16); };
    auto b_row = [&](int v) { return ((v * G::kWavesG + wave) * 64 + lane) / (G::kRowB / 16); };
    auto begin_item = [&]() {  // the next one with rows; none leaves left = 0
        Item w;
        ld.left = 0;
        while (++ld.round < rounds) {
            if (!locate(ld.round, &w) || !w.len)
                continue;
            const int64_t row0 = a.seg.first_row(w.s);
            ld.left = w.len;
            ld.a_base = (const char *)(a.d_y + row0 * a.out_dim + w.m0);
            ld.b_base = (const char *)(a.x + row0 * a.in_dim + w.n0);
            // columns past the end are not stored: the block's first serve them
#pragma unroll
            for (int v = 0; v < G::kAInstr; ++v) {
                const int row = a_row(v), chunk = (lane % (G::kRowA / 16)) ^ ((row & 3) << 2);
                ld.a_off[v] = (uint32_t)row * (uint32_t)a.out_dim * 2 +
                              (w.m0 + chunk * 8 < a.out_dim ? chunk * 16 : 0);
            }
#pragma unroll
            for (int v = 0; v < G::kBInstr; ++v) {
                const int row = b_row(v), chunk = (lane % (G::kRowB / 16)) ^ ((row & 3) << 2);
                ld.b_off[v] = (uint32_t)row * (uint32_t)a.in_dim * 2 +
                              (w.n0 + chunk * 8 < a.in_dim ? chunk * 16 : 0);
            }
            return;
        }
    };
    const char *zero = (const char *)g_zero_row;
    // Issues the next stage into slot `to`.  After the last item the loads go on
    // with zeros, which nobody computes: so every stage is followed by as many.
    auto issue = [&](int to) {
        if (ld.left <= 0)
            begin_item();
        char *dst = ring + to * G::kStageBytes + wave * 1024;
#pragma unroll
        for (int v = 0; v < G::kAInstr; ++v)
            dma16(a_row(v) < ld.left ? ld.a_base + ld.a_off[v] : zero, dst + v * G::kWavesG * 1024);
#pragma unroll
        for (int v = 0; v < G::kBInstr; ++v)
            dma16(b_row(v) < ld.left ? ld.b_base + ld.b_off[v] : zero,
                  dst + G::kStageA + v * G::kWavesG * 1024);
        ld.a_base += (int64_t)BK * a.out_dim * 2;
        ld.b_base += (int64_t)BK * a.in_dim * 2;
        ld.left -= BK;
    };

    // LDS addresses of this wave's fragments in slot 0, k-step 0
    uint32_t frag_at[G::kTM + G::kTN];
#pragma unroll
    for (int i = 0; i < G::kTM; ++i)
        frag_at[i] = lds_addr(ring) + (tr_offset<G::kRowA>(lane) ^ ((wm * G::kTM + i) << 6));
#pragma unroll
    for (int j = 0; j < G::kTN; ++j)
        frag_at[G::kTM + j] =
            lds_addr(ring) + G::kStageA + (tr_offset<G::kRowB>(lane) ^ ((wn * G::kTN + j) << 6));

    ld.round = -1;
    ld.left = 0;
    ld.a_base = ld.b_base = zero;
#pragma unroll
    for (int st = 0; st + 1 < S; ++st)
        issue(st);
    int now = 0;  // slot of the stage computed next
    for (int64_t round = 0; round < rounds; ++round) {
        Item w;
        if (!locate(round, &w))
            continue;
        f32x16 acc[G::kTM][G::kTN];
#pragma unroll
        for (int i = 0; i < G::kTM; ++i)
#pragma unroll
            for (int j = 0; j < G::kTN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[i][j][r] = 0.0f;

        const int32_t nk = (w.len + BK - 1) / BK;
        for (int32_t kt = 0; kt < nk; ++kt) {
            // this wave's loads of the stage have landed once only those of the S - 2
            // later ones are outstanding
            wait_vm<(S - 2) * G::kPerStage>();
            lds_barrier();  // the stage is visible to all; the one before is free
            const uint32_t stage = (uint32_t)(now * G::kStageBytes);
            const int free_slot = now ? now - 1 : S - 1;
            now = now + 1 == S ? 0 : now + 1;
#pragma unroll
            for (int ks = 0; ks < BK / 16; ++ks) {
                static_assert(G::kRowA == G::kRowB, "one distance for all fragments");
                uint32_t at[G::kTM + G::kTN];
                bf16x8 f[G::kTM + G::kTN];
#pragma unroll
                for (int i = 0; i < G::kTM + G::kTN; ++i)
                    at[i] = frag_at[i] + stage + ks * 16 * G::kRowA;
                tr_frags<G::kRowA>(at, f);
                // behind the stage's last reads, for their address arithmetic to run under
                // matrix instructions (sweep: 1620 us where it came first, 1467)
                if (ks == BK / 16 - 1)
                    issue(free_slot);
#pragma unroll
                for (int i = 0; i < G::kTM; ++i)
#pragma unroll
                    for (int j = 0; j < G::kTN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i], f[G::kTM + j],
                                                                            acc[i][j], 0, 0, 0);
            }
        }
        if (a.accumulate && !nk)
            continue;
        // a register's 32 lanes hold 32 consecutive columns: whole 128-byte lines
        float *out = w.s < a.seg.E ? a.home + w.s * a.G : a.rep + (int64_t)(w.s - a.seg.E) * a.G;
        out += a.g_offset;
#pragma unroll
        for (int i = 0; i < G::kTM; ++i)
#pragma unroll
            for (int j = 0; j < G::kTN; ++j) {
                const int32_t row = w.m0 + wm * WM + i * 32, col = w.n0 + wn * WN + j * 32;
                if (row < a.out_dim && col < a.in_dim) {
                    float *p = out + (int64_t)(row + (lane >> 5) * 4) * a.in_dim + col + (lane & 31);
                    if (a.accumulate) {
                        float old[16];
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            old[r] = p[(int64_t)((r >> 2) * 8 + (r & 3)) * a.in_dim];
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            acc[i][j][r] += old[r];
                    }
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        put<G::kStream>(p + (int64_t)((r >> 2) * 8 + (r & 3)) * a.in_dim, acc[i][j][r]);
                }
            }
    }
    wait_vm<0>();  // nothing is on its way into the LDS when it is given back
}

// The device's compute units, and the kernel's dynamic-LDS limit raised once
// per device to the most that any call needs.
template <class Kernel>
int prepare_launch(Kernel kernel, size_t most, bool (&raised)[64], int *cus)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
        return MOONEP_ERR_HIP;
    if (dev < 0 || dev >= 64 || !raised[dev]) {
        if (hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                (int)most) != hipSuccess)
            return MOONEP_ERR_HIP;
        if (dev >= 0 && dev < 64)
            raised[dev] = true;
    }
    return MOONEP_OK;
}

template <int BM, int BN, int WM, int WN, int BK, int S>
int run_dx(const DxArgs &a, hipStream_t st)
{
    using G = DxCfg<BM, BN, WM, WN, BK, S>;
    static bool raised[64] = {};
    int cus = 0;
    const int rc = prepare_launch(expert_dx_kernel<BM, BN, WM, WN, BK, S>,
                                  G::kSegAt + (size_t)(2 * kMaxExperts + kMaxRanks + 1) * 4, raised, &cus);
    if (rc != MOONEP_OK)
        return rc;
    const size_t bytes = G::kSegAt + (size_t)(a.seg.E + a.seg.pl.cap + 1) * 4;
    const int per_cu = (int)((160u << 10) / bytes);
    hipLaunchKernelGGL((expert_dx_kernel<BM, BN, WM, WN, BK, S>), dim3(cus * (per_cu > 1 ? per_cu : 1)),
                       dim3(G::kThreads), bytes, st, a);
    return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_ERR_HIP;
}

template <int BM, int BN, int WM, int WN, int BK, int S>
int run_dw(const DwArgs &a, hipStream_t st)
{
    using G = DwCfg<BM, BN, WM, WN, BK, S>;
    constexpr size_t kRing = (size_t)S * G::kStageBytes;
    static bool raised[64] = {};
    int cus = 0;
    const int rc = prepare_launch(expert_dw_kernel<BM, BN, WM, WN, BK, S>,
                                  kRing + (size_t)(2 * (2 * kMaxExperts + kMaxRanks) + 4) * 4, raised, &cus);
    if (rc != MOONEP_OK)
        return rc;
    const size_t bytes = kRing + (size_t)(2 * (a.seg.E + a.seg.pl.cap) + 4) * 4;
    const int per_cu = (int)((160u << 10) / bytes);
    hipLaunchKernelGGL((expert_dw_kernel<BM, BN, WM, WN, BK, S>), dim3(cus * (per_cu > 1 ? per_cu : 1)),
                       dim3(G::kThreads), bytes, st, a);
    return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_ERR_HIP;
}

}  // namespace

// Tiles of 256 x 256, eight waves, or of 128 x 128 and less, four waves and two
// workgroups per CU, measured on 64 experts, 2048 -> 1408 (d_x) and 1408 -> 2048
// (g), us, large tile first:
//   d_x, by mean rows of an expert:   32: 112, 92    61: 117, 95   128: 127, 123
//     256: 172, 162   384: 224, 202   512: 248, 257   4096: 1486, 1716;
//     2048 rows, 512 x 512, 16 experts (two rounds of items): 35, 33
//   g, which the rows do not decide (61: 179, 190; 512: 324, 418) but the items
//     do: 36: 23.5, 15.4   64: 98, 64   128: 41, 28   256: 44, 42   384: 55, 64   768: 105, 123.
constexpr int64_t kLargeRows = 448;    // mean rows of an expert from which d_x takes large tiles
constexpr int64_t kLargeItemsX = 512;  // and of those tiles
constexpr int64_t kLargeItemsW = 320;  // large tiles from which g takes them
// Tiles that the dims leave part-empty count as full ones here; layers narrower than 256 with
// many experts, where that matters, were not measured.

// Where all items of smaller tiles run at once, each on a CU of its own, d_x takes those of
// 64 x 128, or of 128 x 128 with a third slot instead of a second workgroup (us with 128,
// two or three slots, and with 64): 3387 rows, 1024 -> 192, 9 experts: 20, 16, 12; 1024
// rows, 2048 -> 1024, 8 experts (160 items of 64): -, 25.5, 21.0; 2048 rows (288): -, 26,
// 33.  Experts of few rows leave most of a tile empty, and what counts is how many loads
// are in flight: 64 x 128 with four slots (mean rows 32: 93, 85; 50: 93, 84; 61: 95, 95;
// 80: 98, 105; 32 experts, 2048 -> 1024, 64: 55, 45; 128: 53, 59).
constexpr int64_t kFewItems = 256;
constexpr int64_t kShortRows = 64;

int launch_expert_dx(const moonep_shape &s, const int32_t *plan, const int32_t *wslot, int32_t B,
                     int32_t in_dim, int32_t out_dim, const uint16_t *d_y, const uint16_t *w_home,
                     const uint16_t *pool, int64_t w_stride, int64_t w_offset, uint16_t *d_x,
                     hipStream_t st)
{
    if ((int64_t)s.R * s.S * s.K == 0)
        return MOONEP_OK;
    const DxArgs a{seg_tables(s, plan, wslot, B), in_dim, out_dim, d_y, w_home, pool,
                   w_stride, w_offset, d_x};
    const int64_t rows = (int64_t)s.R * s.S * s.K;
    const int64_t items = ((rows + 255) / 256 + s.E / 2) * ((in_dim + 255) / 256);
    if (rows >= kLargeRows * s.E && items >= kLargeItemsX)
        return run_dx<256, 256, 128, 64, 32, 4>(a, st);
    const int64_t blocks = (in_dim + 127) / 128;
    if (((rows + 63) / 64 + s.E / 2) * blocks <= kFewItems)
        return run_dx<64, 128, 32, 64, 64, 3>(a, st);
    if (rows <= kShortRows * s.E)
        return run_dx<64, 128, 32, 64, 64, 4>(a, st);
    if (((rows + 127) / 128 + s.E / 2) * blocks <= kFewItems)
        return run_dx<128, 128, 64, 64, 64, 3>(a, st);
    return run_dx<128, 128, 64, 64, 64, 2>(a, st);
}

int launch_expert_dw(const moonep_shape &s, const int32_t *plan, int32_t in_dim, int32_t out_dim,
                     const uint16_t *x, const uint16_t *d_y, int accumulate, int64_t G,
                     int64_t g_offset, float *home, float *rep, hipStream_t st)
{
    if (accumulate && (int64_t)s.R * s.S * s.K == 0)
        return MOONEP_OK;
    const DwArgs a{seg_tables(s, plan, nullptr, 0), in_dim, out_dim, accumulate, x, d_y, G, g_offset,
                   home, rep};
    const int64_t items = (int64_t)s.E * ((in_dim + 255) / 256) * ((out_dim + 255) / 256);
    if (items >= kLargeItemsW)
        return run_dw<256, 256, 128, 64, 32, 4>(a, st);
    return run_dw<128, 128, 64, 64, 64, 3>(a, st);
}

}  // namespace moonep
