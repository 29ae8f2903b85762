// gemm_quant.hip -- the experts' products in 8 bits over the expert-grouped
// buffer: one projection with a bf16 output, or gate and up with the activation
// and an 8-bit output.
//
// Both operands are e4m3 codes with an E8M0 scale for each block of 128 along k
// (weights: of 128 x 128).  gfx950's scaled matrix instruction multiplies by
// E8M0 scales itself, one byte per lane and operand, so all blocks accumulate
// into one fp32 accumulator and the scales cost no vector work:
//   v_mfma_scale_f32_32x32x64_f8f6f4: lane l of A holds row l % 32, of B column
//   l % 32, 32 k values each (which 32 is free, as long as A and B agree), and
//   the byte that scales them; the 32 x 32 result as in the bf16 kernel: lane
//   l, register q holds row (q / 4) * 8 + (l / 32) * 4 + q % 4, column l % 32.
// The weights are the first operand, so that a lane holds one token row.
//
// Rounding: the accumulators are fp32, but the instruction adds its 64 products in
// groups of 8 (8 consecutive bytes of a lane, so of k) and first cuts each product,
// towards zero, to a multiple of 2^-13 of the group's largest power of two,
// 2^(ea + eb) of the codes' exponents (subnormal codes: -6); the groups and the
// accumulator are then added within 2^-24 of the largest.  (Found by one large and one
// small product at every pair of positions; a model of it gives the instruction's
// results on random codes, to fp32's rounding.)  Products of codes have
// eight bits, so those within 2^-7 of the largest are whole.  On normal codes that is
// an rms of 2^-19 (k = 128) to 2^-21 (k = 2048) of sum |a| |b|, 2^-14.5 at most, and
// 2^-18.5 towards zero where all products are positive; on codes of every size alike
// 2^-11 at most.  All 8-bit forms do this (scaled or not, both shapes), bf16 ones do
// not and take twice the time; the outputs' half steps are 2^-4 of an e4m3 code and
// 2^-8 of a bf16 value, so it is accepted.
//
// Structure: persistent workgroups walk (row tile, column block) items; K
// advances 128 at a time (one scale block) through a ring of S LDS stages
// filled by LDS-DMA, rows of 128 bytes with their 16-byte chunks XOR-swizzled
// so that 16 consecutive rows' reads fall on different banks; scales go through a
// ring of their own, a dword for four blocks.  The rings run on from one item to
// the next, under the epilogue.
//
// What bounds it, gate and up of 262144 rows, 2048 -> 2 x 1408 (1424-1441 us, 2.1
// PFLOP/s; a library product in 8 bits without block scales and segments takes
// 1264): the tile's loads (12.3 GB; alone 1259 us) and the matrix products (without
// loads 987 us), which overlap but share the power: 1.9-2.0 GHz with both, 2.13 without
// the loads.  The loads' limit is no bandwidth.  19% of the L2's requests miss, 3.3 GB
// come from beyond it (2.3 TB/s; rows and weights once are 0.95 GB), and with all of
// them made to hit the loads alone take 736 us, 16.7 TB/s, where LDS-DMA of resident
// data reaches 38: it is a stage's round trip, with one stage in flight, and half
// of it the misses'.  Deeper rings of smaller stages (the loads alone 1323 us with 96
// KB in flight), other schedules of the LDS reads and tiles of 128 rows (two
// workgroups per CU) were all no faster; an item order with fewer misses is untried.  At 4 rows an expert (77 us) it is bound by the weights' bytes, 5.6
// TB/s of them.  One projection of 32576 rows, 1408 -> 2048 (141-148 us, its products
// 64): 20% of the tiles' rows are empty, the bf16 stores take 25 us that the next
// item's loads, which return in order behind them, do not hide, and an item is
// eleven k-steps with one stage in flight.
//
// Gate and up: the column tile interleaves 32 gate and 32 up columns, so one
// wave holds both products of an output, and 128 output columns -- one block of
// the 8-bit output -- stay in one workgroup.
#include "quant.hpp"
#include "segments.hpp"

namespace moonep {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// What rows and chunks past the ends read: codes of 0.
__device__ __align__(16) const uint8_t kZeros[16] = {};

constexpr int kCuLds = 160 * 1024;
constexpr int kSegBytesMax = (2 * kMaxExperts + kMaxRanks + 1) * 4;  // seg_start of the largest shape
constexpr int kTileGroup = 8;  // row tiles per item group, as in the bf16 product

template <int BM, int BN, int WM, int WN, int BK, int S, bool GLU>
struct QCfg {
    static constexpr int kBK = BK;                    // k per stage, in bytes
    static constexpr int kCpr = BK / 16;              // 16-byte chunks of a row
    static constexpr int kRpi = 64 / kCpr;            // rows (1 KiB) per LDS-DMA load
    static constexpr int kTM = WM / 32, kTN = WN / 32;
    static constexpr int kWM = BM / WM, kWN = BN / WN;
    static constexpr int kWavesG = kWM * kWN;
    static constexpr int kThreads = kWavesG * 64;
    static constexpr int kAInstr = BM / kRpi / kWavesG;
    static constexpr int kBInstr = BN / kRpi / kWavesG;
    static constexpr int kPerStage = kAInstr + kBInstr;
    static constexpr int kStageBytes = (BM + BN) * BK;
    // Scales: a dword holds four blocks of a row, so a slot of a ring of its own
    // serves 4 * 128 / BK stages of an item: [BM] rows, then the weights' blocks.
    // At most S stages are loading or in use, so S slots do.
    static constexpr int kBBlocks = GLU ? 2 : (BN + kQuantBlock - 1) / kQuantBlock;
    static constexpr int kScaleStages = 4 * kQuantBlock / BK;
    static constexpr int kScaleWaves = (BM + kBBlocks + 63) / 64;
    static constexpr int kScaleBytes = kScaleWaves * 256;
    static constexpr int kScaleAt = S * kStageBytes;
    static constexpr int kOutCols = GLU ? BN / 2 : BN;
    // Epilogue, apart from the ring, which is loading the next item: for an 8-bit
    // output the waves' row maxima, for bf16 a band of 32 rows on its way out.
    static constexpr int kOutBytes = GLU ? 1 : 2;
    static constexpr int kBands = BM / 32, kBandRowBytes = BN * 2 + 16;
    static constexpr int kBandStores = 32 * (BN / 8) / kThreads;
    static constexpr int kOutAt = kScaleAt + S * kScaleBytes;
    static constexpr int kSegAt = kOutAt + (GLU ? BM * kWN * 4 : 32 * kBandRowBytes);
    static_assert(BK == 64 || BK == 128, "one or two matrix instructions, one scale");
    static_assert(BM % (kRpi * kWavesG) == 0 && BN % (kRpi * kWavesG) == 0, "rows per DMA round");
    static_assert(kScaleWaves <= kWavesG, "a thread for every scale");
    static constexpr int kStores = GLU ? kTM : kBands * kBandStores;  // of rows, per wave and item
    static_assert((S - 1) * kPerStage + kStores <= 63, "outstanding accesses must fit vmcnt");
    static_assert(GLU || (kBandStores >= 1 && 32 * (BN / 8) % kThreads == 0), "whole stores of a band");
    static_assert(!GLU || (kOutCols == kQuantBlock && kTN == 2), "gate and up in one wave, one block");
    static_assert(kSegAt + kSegBytesMax <= kCuLds, "LDS");
    // rows whose chunks share the banks: two of 128 bytes, four of 64
    __device__ static constexpr int swz(int r) { return BK == 128 ? (r >> 1) & 7 : (r >> 2) & 3; }
};

struct QuantGemmArgs {
    SegTables seg;
    int32_t in_dim, out_dim;
    const uint8_t *x8, *xs, *w_home, *pool;
    int64_t w_stride;
    int64_t code[2], scale[2];  // windows: the matrix, or gate and up
    void *out;
    uint8_t *out_scales;
};

// s_waitcnt vmcnt(n), the other counters left alone
template <int n>
__device__ __forceinline__ void wait_vm()
{
    __builtin_amdgcn_s_waitcnt(0x0F70 | (n & 15) | ((n >> 4) << 14));
}

// A value that every lane holds alike, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t v)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// Lanes 32 .. 63 of `a` for lanes 0 .. 31 of `b`.
__device__ __forceinline__ void swap_halves(uint32_t &a, uint32_t &b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// One LDS-DMA load: kBytes of each lane to dst + lane * kBytes.
template <int kBytes>
__device__ __forceinline__ void dma(const uint8_t *src, char *dst)
{
    auto *to = (__attribute__((address_space(3))) void *)dst;
    if constexpr (kBytes == 16)
        __builtin_amdgcn_global_load_lds((const void *)src, to, 16, 0, 0);
    else
        __builtin_amdgcn_global_load_lds((const void *)src, to, 4, 0, 0);
}

}  // namespace

template <int BM, int BN, int WM, int WN, int BK, int S, bool GLU, bool TAIL>
__global__ __launch_bounds__((QCfg<BM, BN, WM, WN, BK, S, GLU>::kThreads)) void expert_quant_kernel(
    QuantGemmArgs a)
{
    using G = QCfg<BM, BN, WM, WN, BK, S, GLU>;
    extern __shared__ __align__(16) char lds_b[];
    int32_t *seg_start = (int32_t *)(lds_b + G::kSegAt);
    __shared__ int scan_tmp[G::kWavesG];

    const int tid = (int)threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / G::kWN, wn = wave % G::kWN;
    const int32_t nseg = a.seg.E + a.seg.n_rep();
    const int32_t tiles = scan_tiles<BM, G::kWavesG>(a.seg, nseg, seg_start, scan_tmp);
    const int32_t nbn = (a.out_dim + G::kOutCols - 1) / G::kOutCols;
    // Items of whole tiles; those of the last round are halves of a tile's rows where
    // that still makes one round.  (32 bits: 2^31 items of 32 x 128 values at
    // least would be over 8 TB of output.)
    const uint32_t tile_items = (uint32_t)tiles * (uint32_t)nbn, rest = tile_items % gridDim.x;
    const uint32_t halves = G::kWM == 2 && 2 * rest <= gridDim.x ? rest : 0;
    const uint32_t whole = tile_items - halves, items = tile_items + halves;
    const int32_t nk = (a.in_dim + G::kBK - 1) / G::kBK;
    const int32_t SB = scale_row_bytes(a.in_dim), SO = scale_row_bytes(a.out_dim);

    // ---- the loads: items and their k-steps in one sequence ------------------
    // LDS-DMA: lane i of a load brings chunk (i % kCpr) ^ swz(row) of row kRpi g +
    // i / kCpr to byte 16 i of the load's KiB.  Row r of the B tile is column r of the
    // block, or for gate and up column (r / 64) * 32 + r % 32 of gate (r / 32
    // even) or up, which one load never mixes.
    struct Load {
        uint32_t it;
        int64_t m0;
        int32_t kt, mrows, n0;
        const uint8_t *a_base, *b_base[2];  // the item's first row; first column, of each matrix
        const uint8_t *scale;  // this thread's
        uint32_t a_off[G::kAInstr], b_off[G::kBInstr];
    };
    Load ld;
    const uint32_t first = (uint32_t)xcd_slot((int)blockIdx.x, (int)gridDim.x);
    if (first >= items)
        return;
    ld.it = first;
    const int dma_row = lane / G::kCpr, dma_pos = lane % G::kCpr;
    auto a_row = [&](int v) { return (v * G::kWavesG + wave) * G::kRpi + dma_row; };
    auto b_mat = [&](int v) { return GLU ? (v * G::kWavesG + wave) * G::kRpi / 32 % 2 : 0; };
    auto chunk = [&](int v) { return (dma_pos ^ G::swz(a_row(v))) << 4; };
    // First row and column of an item, its rows and its weights.
    auto locate = [&](uint32_t it, int64_t *m0, int32_t *mrows, int32_t *n0) -> const uint8_t * {
        int32_t t, nb, n, row0 = 0, most = BM;
        if (it >= whole) {
            row0 = (it - whole) % 2 * (BM / 2);
            most = BM / 2;
            it = whole + (it - whole) / 2;
        }
        item_of<kTileGroup>(it, tiles, nbn, &t, &nb);
        const int32_t s = find_segment(seg_start, nseg, t);
        const int32_t mt = t - __builtin_amdgcn_readfirstlane(seg_start[s]);
        int64_t wrow;
        bool pooled;
        *m0 = a.seg.segment(s, &n, &wrow, &pooled) + (int64_t)mt * BM;
        const int32_t left = n - mt * BM - row0;
        *mrows = left < 0 ? 0 : left < most ? left : most;  // 0: a short tile's second half
        *m0 += left > 0 ? row0 : 0;
        *n0 = nb * G::kOutCols;
        return (pooled ? a.pool : a.w_home) + wrow * a.w_stride;
    };
    auto begin_item = [&]() {
        const uint8_t *w = locate(ld.it, &ld.m0, &ld.mrows, &ld.n0);
        ld.a_base = a.x8 + ld.m0 * a.in_dim;
#pragma unroll
        for (int m = 0; m < 2; ++m)
            ld.b_base[m] = w + a.code[m] + (int64_t)ld.n0 * a.in_dim;
#pragma unroll
        for (int v = 0; v < G::kAInstr; ++v)
            ld.a_off[v] = (uint32_t)((a_row(v) < ld.mrows ? a_row(v) : 0) * a.in_dim + chunk(v));
#pragma unroll
        for (int v = 0; v < G::kBInstr; ++v) {
            const int r = a_row(v), c = GLU ? (r >> 6) * 32 + (r & 31) : r;
            // columns past the end are not stored: the block's first serves them
            ld.b_off[v] = (uint32_t)((ld.n0 + c < a.out_dim ? c : 0) * a.in_dim + chunk(v));
        }
        if (tid < BM) {
            ld.scale = a.xs + (ld.m0 + (tid < ld.mrows ? tid : 0)) * SB;
        } else {
            // weights: block q of the tile's columns, or gate's and up's block
            const int q = tid - BM < G::kBBlocks ? tid - BM : 0;
            const int32_t last_block = (a.out_dim - 1) / kQuantBlock;
            const int32_t block = ld.n0 / kQuantBlock + (GLU ? 0 : q);
            ld.scale = w + a.scale[GLU ? q : 0] +
                       (int64_t)(block < last_block ? block : last_block) * SB;
        }
    };
    // Issues the next stage into slot `to`; an item's every kScaleStages-th with the
    // scales of as many.  After the last item the loads go on with its first
    // stages again, which nobody computes: so every stage is followed by as many.
    int scale_to = 0;
    auto issue = [&](int to) {
        if (ld.kt == nk) {
            ld.kt = 0;
            ld.it += gridDim.x;
            if (ld.it < items)
                begin_item();
        }
        char *dst = lds_b + to * G::kStageBytes;
        const int64_t k0 = (int64_t)ld.kt * G::kBK;
        if (ld.kt % G::kScaleStages == 0) {
            if (wave < G::kScaleWaves)
                dma<4>(ld.scale + ld.kt / G::kScaleStages * 4,
                       lds_b + G::kScaleAt + scale_to * G::kScaleBytes + wave * 256);
            scale_to = scale_to + 1 == S ? 0 : scale_to + 1;
        }
#pragma unroll
        for (int v = 0; v < G::kPerStage; ++v) {
            const bool rows = v < G::kAInstr;
            const int w = rows ? v : v - G::kAInstr;
            const uint8_t *src = rows ? ld.a_base + k0 + ld.a_off[w]
                                      : (b_mat(w) ? ld.b_base[1] : ld.b_base[0]) + k0 + ld.b_off[w];
            if (TAIL)
                src = chunk(w) < a.in_dim - (int32_t)k0 ? src : kZeros;
            dma<16>(src, dst + (rows ? 0 : BM * G::kBK) + (w * G::kWavesG + wave) * 1024);
        }
        ++ld.kt;
    };

    // ---- the products ---------------------------------------------------------
    const int fr = lane & 31, fsw = G::swz(lane & 31), fhalf = lane >> 5;
    auto frag = [&](const char *base, int row0, int ks) -> i32x8 {
        const char *p = base + (row0 + fr) * G::kBK;
        const u32x4 lo = *(const u32x4 *)(p + (((4 * ks + fhalf) ^ fsw) << 4));
        const u32x4 hi = *(const u32x4 *)(p + (((4 * ks + 2 + fhalf) ^ fsw) << 4));
        i32x8 r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[j] = (int)lo[j];
            r[4 + j] = (int)hi[j];
        }
        return r;
    };
    ld.kt = 0;
    begin_item();
    int slot = 0, scale_slot = 0;  // of the stage computed next; the rings run on across items
#pragma unroll
    for (int st = 0; st < S; ++st)
        issue(st);

    for (uint32_t it = first; it < items; it += gridDim.x) {
        int64_t m0 = ld.m0;
        int32_t mrows = ld.mrows, n0 = ld.n0;
        if (ld.it != it)
            locate(it, &m0, &mrows, &n0);  // few k-steps: the loads are at a later item already
        m0 = uniform(m0);
        mrows = __builtin_amdgcn_readfirstlane(mrows);
        n0 = __builtin_amdgcn_readfirstlane(n0);
        f32x16 acc[G::kTM][G::kTN];
#pragma unroll
        for (int i = 0; i < G::kTM; ++i)
#pragma unroll
            for (int j = 0; j < G::kTN; ++j)
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    acc[i][j][q] = 0.0f;

        for (int32_t kt = 0; kt < nk; ++kt) {
            // This stage's loads have landed once only what was issued after them is
            // outstanding: S - 2 stages, S - 1 at an item's start (the slot of the
            // item before's last stage is loading already).  The first S stages
            // were issued ahead of the stores of the item before, which so need
            // not be waited for; scales and their stores come on top, if any.
            if (kt >= S || it == first)
                kt == 0 ? wait_vm<(S - 1) * G::kPerStage>() : wait_vm<(S - 2) * G::kPerStage>();
            else
                kt == 0 ? wait_vm<(S - 1) * G::kPerStage + G::kStores>()
                        : wait_vm<(S - 2) * G::kPerStage + G::kStores>();
            lds_barrier();  // every wave's part of the stage is there, and the one before is free
            const int cur = slot;
            slot = slot + 1 == S ? 0 : slot + 1;
            if (kt)
                issue(cur == 0 ? S - 1 : cur - 1);
            const char *sa = lds_b + cur * G::kStageBytes;
            const char *sb = sa + BM * G::kBK;
            const uint32_t *sc = (const uint32_t *)(lds_b + G::kScaleAt + scale_slot * G::kScaleBytes);
            const int shift = (kt * G::kBK / kQuantBlock & 3) * 8;
            if (kt % G::kScaleStages == G::kScaleStages - 1 || kt == nk - 1)
                scale_slot = scale_slot + 1 == S ? 0 : scale_slot + 1;
            if (G::kWM > 1 && wm * WM >= mrows)
                continue;  // none of this wave's rows
            int sca[G::kTM], scb[G::kTN];
#pragma unroll
            for (int i = 0; i < G::kTM; ++i)
                sca[i] = (int)(sc[wm * WM + i * 32 + fr] >> shift);
#pragma unroll
            for (int j = 0; j < G::kTN; ++j)
                scb[j] = (int)(sc[BM + (GLU ? j : (wn * WN + j * 32) / kQuantBlock)] >> shift);
            // Steps of one row tile and 64 k: each reads the next step's rows under its
            // own matrix instructions.
            constexpr int kSteps = G::kBK / 64 * G::kTM;
            i32x8 fa[2], fb[2][G::kTN];
#pragma unroll
            for (int j = 0; j < G::kTN; ++j)
                fb[0][j] = frag(sb, wn * WN + j * 32, 0);
            fa[0] = frag(sa, wm * WM, 0);
#pragma unroll
            for (int n = 0; n < kSteps; ++n) {
                const int i = n % G::kTM, ks = n / G::kTM, p = n + 1;
                if (p < kSteps) {
                    fa[p & 1] = frag(sa, wm * WM + p % G::kTM * 32, p / G::kTM);
                    if (p % G::kTM == 0)
#pragma unroll
                        for (int j = 0; j < G::kTN; ++j)
                            fb[(ks + 1) & 1][j] = frag(sb, wn * WN + j * 32, ks + 1);
                }
#pragma unroll
                for (int j = 0; j < G::kTN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        fb[ks & 1][j], fa[n & 1], acc[i][j], 0, 0, 0, scb[j], 0, sca[i]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        lds_barrier();  // the stage computed last is free
        issue(slot == 0 ? S - 1 : slot - 1);

        // ---- epilogue: lane l holds row l % 32 of tile i, and of each column tile
        // the columns 8 (q / 4) + 4 (l / 32) + q % 4 ------------------------------
        // the tile's rows, from its first column to the end of its last row
        const auto out = __builtin_amdgcn_make_buffer_rsrc(
            (char *)a.out + (m0 * a.out_dim + n0) * G::kOutBytes, 0,
            mrows ? (int)((uint32_t)(mrows * a.out_dim - n0) * G::kOutBytes) : 0, 0x00020000);
        // Offset of row `row` and column `col` of the item.  A buffer store drops what
        // is out of bounds, so every wave issues the same number: rows past the tile
        // end behind the buffer, and columns past the row are sent there.
        auto place = [&](int row, int col) -> int {
            const bool in = n0 + col < a.out_dim;
            return (int)(in ? (uint32_t)(row * a.out_dim) * G::kOutBytes + col * G::kOutBytes : 0xFFFFFFF0u);
        };
        if constexpr (GLU) {
            float *row_max = (float *)(lds_b + G::kOutAt);  // [BM][kWN]
#pragma unroll
            for (int i = 0; i < G::kTM; ++i) {
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const float g = acc[i][0][q], u = acc[i][G::kTN - 1][q];
                    // the exponential's argument is rounded once, |g| 2^-24 of its value: far
                    // below a code's half step of 2^-4
                    acc[i][0][q] = g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
                }
                if (n0 + G::kOutCols > a.out_dim) {
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        if (n0 + wn * 32 + (q >> 2) * 8 + fhalf * 4 >= a.out_dim)
                            acc[i][0][q] = 0.0f;
                }
                uint32_t m = 0;
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    m = max(m, abs_bits(acc[i][0][q]));
                m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
                if (fhalf == 0)
                    row_max[(wm * WM + i * 32 + fr) * G::kWN + wn] = __uint_as_float(m);
            }
            lds_barrier();
#pragma unroll
            for (int i = 0; i < G::kTM; ++i) {
                const int row = wm * WM + i * 32 + fr;
                uint32_t m = 0;
#pragma unroll
                for (int q = 0; q < G::kWN; ++q)
                    m = max(m, __float_as_uint(row_max[row * G::kWN + q]));
                const uint32_t byte = scale_byte(m);
                const float inv = inverse_scale(byte);
                uint32_t d[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    d[q] = pack_e4m3(acc[i][0][4 * q], acc[i][0][4 * q + 1], acc[i][0][4 * q + 2],
                                     acc[i][0][4 * q + 3], inv, byte);
                // the lower lanes take the row's columns 0 .. 15, the upper 16 .. 31
                swap_halves(d[0], d[2]);
                swap_halves(d[1], d[3]);
                __builtin_amdgcn_raw_buffer_store_b128(u32x4{d[0], d[2], d[1], d[3]}, out,
                                                       place(row, wn * 32 + fhalf * 16), 0, 0);
                if (wn == 0 && fhalf == 0 && row < mrows) {
                    uint8_t *dst = a.out_scales + (m0 + row) * SO;
                    const int32_t nb = n0 / kQuantBlock;
                    dst[nb] = (uint8_t)byte;
                    if (nb == nbn - 1)
                        for (int32_t p = nbn; p < SO; ++p)
                            dst[p] = 127;
                }
            }
        } else {
            char *so = lds_b + G::kOutAt;
#pragma unroll
            for (int band = 0; band < G::kBands; ++band) {
                if (band)
                    lds_barrier();  // the band before has been read
#pragma unroll
                for (int i = 0; i < G::kTM; ++i) {
                    if (wm * G::kTM + i != band)
                        continue;
#pragma unroll
                    for (int j = 0; j < G::kTN; ++j)
#pragma unroll
                        for (int q = 0; q < 16; q += 4)
                            *(u32x2 *)(so + fr * G::kBandRowBytes + (wn * WN + j * 32 + q * 2 + fhalf * 4) * 2) =
                                u32x2{pack_bf16(acc[i][j][q], acc[i][j][q + 1]),
                                      pack_bf16(acc[i][j][q + 2], acc[i][j][q + 3])};
                }
                lds_barrier();
#pragma unroll
                for (int v = 0; v < G::kBandStores; ++v) {
                    const int idx = tid + v * G::kThreads, row = idx / (BN / 8), c = idx % (BN / 8);
                    __builtin_amdgcn_raw_buffer_store_b128(
                        *(const u32x4 *)(so + row * G::kBandRowBytes + c * 16), out,
                        place(band * 32 + row, c * 8), 0, 0);
                }
            }
        }
    }
    wait_vm<0>();  // the loads that nobody computes, before the LDS goes to another workgroup
}

namespace {

template <int BM, int BN, int WM, int WN, int BK, int S, bool GLU, bool TAIL>
int run_quant(const QuantGemmArgs &a, hipStream_t st)
{
    using G = QCfg<BM, BN, WM, WN, BK, S, GLU>;
    const auto kernel = expert_quant_kernel<BM, BN, WM, WN, BK, S, GLU, TAIL>;
    const size_t lds = G::kSegAt + (size_t)(a.seg.E + a.seg.pl.cap + 1) * 4;
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
        return MOONEP_ERR_HIP;
    // Raised once per device, to what the largest allowed E and R need.
    static bool raised[64] = {};
    if (dev < 0 || dev >= 64 || !raised[dev]) {
        if (hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                G::kSegAt + kSegBytesMax) != hipSuccess)
            return MOONEP_ERR_HIP;
        if (dev >= 0 && dev < 64)
            raised[dev] = true;
    }
    const int per_cu = 2 * lds <= kCuLds ? 2 : 1;
    hipLaunchKernelGGL(kernel, dim3(cus * per_cu), dim3(G::kThreads), lds, st, a);
    return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_ERR_HIP;
}

// TAIL: the last k-step is part of one.
template <int BM, int BN, int WM, int WN, int BK, int S, bool GLU>
int run_tail(const QuantGemmArgs &a, bool tail, hipStream_t st)
{
    return tail ? run_quant<BM, BN, WM, WN, BK, S, GLU, true>(a, st)
                : run_quant<BM, BN, WM, WN, BK, S, GLU, false>(a, st);
}

}  // namespace

int launch_expert_quant(const moonep_shape &s, const int32_t *plan, const int32_t *wslot, int32_t B,
                        int32_t in_dim, int32_t out_dim, const uint8_t *x8, const uint8_t *xs,
                        const uint8_t *w_home, const uint8_t *pool, int64_t w_stride,
                        const int64_t *code, const int64_t *scale, void *out, uint8_t *out_scales,
                        hipStream_t st)
{
    const int64_t rows = (int64_t)s.R * s.S * s.K;
    if (rows == 0)
        return MOONEP_OK;
    QuantGemmArgs a;
    a.seg = seg_tables(s, plan, wslot, B);
    a.in_dim = in_dim;
    a.out_dim = out_dim;
    a.x8 = x8;
    a.xs = xs;
    a.w_home = w_home;
    a.pool = pool;
    a.w_stride = w_stride;
    const bool glu = out_scales != nullptr;
    for (int m = 0; m < 2; ++m) {
        a.code[m] = code[glu ? m : 0];
        a.scale[m] = scale[glu ? m : 0];
    }
    a.out = out;
    a.out_scales = out_scales;
    const bool tail = in_dim % kQuantBlock != 0;
    // Tiles by the mean rows of an expert: few rows want few wasted ones and a deep
    // ring of weights, many want the bytes that a large tile saves.  Measured at
    // R = 8, E = 64, K = 8, us by mean rows:
    //   gate and up, tiles of 32 / 64 / 256 rows, 2048 -> 1408: 4: 77 / 78 / 101, 12:
    //   86 / 89 / 111, 16: 96 / 87 / 111, 64: 147 / 117 / 131, 80: 166 / 127 / 132,
    //   96: 178 / 133 / 131, 128: 219 / 159 / 135, 512: 624 / 412 / 246;
    //   4096 -> 4096: 64: 565 / 466 / 490, 96: 700 / 544 / 529;
    //   one projection, 32 x 128 / 128 x 128 / 256 x 256, 1408 -> 2048: 4: 41 / 45 / 55,
    //   16: 48 / 52 / 70, 24: 53 / 53 / 70, 64: 74 / 59 / 74, 128: 115 / 74 / 78, 192:
    //   155 / 93 / 86, 512: 365 / 192 / 149; 4096 -> 4096: 96: 385 / 283 / 282, 128:
    //   482 / 316 / 297.
    // With other experts and skews the tile chosen is within 6% of the best (one
    // projection of skewed short segments, the last line: 10-14%): E = 128, K = 4, gate and up 2048 -> 1408: 8: 148 / 152 / 206, 12: 166 /
    //   154 / 207, 64: 267 / 221 / 232, 88: 325 / 249 / 238; one projection 1408 -> 2048:
    //   24: 99 / 102 / 125, 128: 218 / 144 / 144, 200: 316 / 181 / 164;
    //   E = 32, 4096 -> 4096: 24: 224 / 224 / 256 and 115 / 116 / 155, 88: 344 / 269 / 270
    //   and 191 / 142 / 164, 128: 430 / 331 / 282 and 245 / 163 / 166;
    //   E = 256, skewed, 2048 -> 768: 8: 118 / 111 / 147, 88: 326 / 241 / 230; 768 -> 2048:
    //   8: 57 / 70 / 81, 24: 83 / 91 / 101, 88: 182 / 143 / 130, 144: 269 / 179 / 157.
    const int64_t mean = rows / s.E;
    if (glu) {
        if (mean <= 12)
            return run_tail<32, 256, 32, 64, 128, 3, true>(a, tail, st);
        if (mean <= 88)
            return run_tail<64, 256, 64, 64, 128, 3, true>(a, tail, st);
        return run_tail<256, 256, 128, 64, 128, 2, true>(a, tail, st);
    }
    if (mean <= 24)
        return run_tail<32, 128, 32, 32, 128, 6, false>(a, tail, st);
    if (mean <= 144)
        return run_tail<128, 128, 64, 32, 128, 3, false>(a, tail, st);
    return run_tail<256, 256, 128, 64, 128, 2, false>(a, tail, st);
}

}  // namespace moonep
