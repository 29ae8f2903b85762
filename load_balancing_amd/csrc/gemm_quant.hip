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
//
// Structure: persistent workgroups walk (row tile, column block) items; K
// advances 128 at a time (one scale block) through a ring of S LDS stages
// filled by LDS-DMA, rows of 128 bytes with their 16-byte chunks XOR-swizzled
// so that 16 consecutive rows' reads fall on different banks; each stage also
// carries the dword of A scales that its block's byte is taken from.
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

constexpr int kTileGroup = 8;  // row tiles per item group, as in the bf16 product

template <int BM, int BN, int WM, int WN, int S, bool GLU>
struct QCfg {
    static constexpr int kBK = 128;
    static constexpr int kTM = WM / 32, kTN = WN / 32;
    static constexpr int kWM = BM / WM, kWN = BN / WN;
    static constexpr int kWavesG = kWM * kWN;
    static constexpr int kThreads = kWavesG * 64;
    static constexpr int kAInstr = BM / 8 / kWavesG;  // 8 rows (1 KiB) per LDS-DMA load
    static constexpr int kBInstr = BN / 8 / kWavesG;
    static constexpr int kPerStage = kAInstr + kBInstr + 1;
    static constexpr int kScaleAt = (BM + BN) * kBK;
    static constexpr int kStageBytes = kScaleAt + kThreads * 4;
    static constexpr int kOutCols = GLU ? BN / 2 : BN;
    static constexpr int kLdo = GLU ? kOutCols + 4 : kOutCols + 8;  // epilogue row, elements
    static constexpr int kOutBytes = GLU ? 4 : 2;
    static constexpr int kOutVec = 8;                     // columns per thread of the epilogue
    static constexpr int kOIter = WM * kOutCols / kOutVec / kThreads;
    static_assert(BM % (8 * kWavesG) == 0 && BN % (8 * kWavesG) == 0, "rows per DMA round");
    static_assert(BM <= kThreads, "one scale dword per thread");
    static_assert(WM * kLdo * kOutBytes <= S * kStageBytes, "an epilogue band must fit the ring");
    static_assert((S - 2) * kPerStage <= 63, "outstanding loads must fit vmcnt");
    static_assert(!GLU || (kOutCols == kQuantBlock && kTN == 2), "gate and up in one wave, one block");
    static_assert(kOIter >= 1 && WM * kOutCols % (kOutVec * kThreads) == 0, "epilogue split");
    __device__ static constexpr int swz(int r) { return (r >> 1) & 7; }
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

}  // namespace

template <int BM, int BN, int WM, int WN, int S, bool GLU>
__global__ __launch_bounds__((QCfg<BM, BN, WM, WN, S, GLU>::kThreads)) void expert_quant_kernel(
    QuantGemmArgs a)
{
    using G = QCfg<BM, BN, WM, WN, S, GLU>;
    extern __shared__ __align__(16) char lds_b[];
    int32_t *seg_start = (int32_t *)(lds_b + S * G::kStageBytes);
    __shared__ int scan_tmp[G::kWavesG];

    const int tid = (int)threadIdx.x, lane = lane_id(), wave = tid >> 6;
    const int wm = wave / G::kWN, wn = wave % G::kWN;
    const int32_t nseg = a.seg.E + a.seg.n_rep();
    const int32_t tiles = scan_tiles<BM, G::kWavesG>(a.seg, nseg, seg_start, scan_tmp);
    const int32_t nbn = (a.out_dim + G::kOutCols - 1) / G::kOutCols;
    const int64_t items = (int64_t)tiles * nbn;
    const int32_t nk = (a.in_dim + G::kBK - 1) / G::kBK;
    const int32_t SB = scale_row_bytes(a.in_dim), SO = scale_row_bytes(a.out_dim);
    const bool k_tail = a.in_dim % G::kBK != 0;

    for (int64_t it = xcd_slot((int)blockIdx.x, (int)gridDim.x); it < items; it += gridDim.x) {
        int32_t t, nb;
        item_of<kTileGroup>(it, tiles, nbn, &t, &nb);
        const int32_t s = find_segment(seg_start, nseg, t);
        int64_t wrow;
        bool pooled;
        const int32_t mt = t - seg_start[s];
        const int64_t m0 = a.seg.first_row(s, &wrow, &pooled) + (int64_t)mt * BM;
        const int32_t left = a.seg.rows(s) - mt * BM;
        const int32_t mrows = left < BM ? left : BM;
        const uint8_t *wbase = (pooled ? a.pool : a.w_home) + wrow * a.w_stride;
        const int32_t n0 = nb * G::kOutCols;

        // Row of the B tile -> matrix and column: for gate and up, 32 of one and
        // 32 of the other in turn.
        auto b_col = [&](int row) { return n0 + (GLU ? (row >> 6) * 32 + (row & 31) : row); };
        auto b_mat = [&](int row) { return GLU ? (row >> 5) & 1 : 0; };

        // LDS-DMA: lane i of a load brings chunk (i % 8) ^ swz(row) of row
        // 8 g + i / 8 to byte 16 i of the load's KiB.
        const int dma_row = lane >> 3, dma_pos = lane & 7;
        uint32_t a_off[G::kAInstr];
        const uint8_t *b_ptr[G::kBInstr];
#pragma unroll
        for (int v = 0; v < G::kAInstr; ++v) {
            const int row = (v * G::kWavesG + wave) * 8 + dma_row;
            a_off[v] = (uint32_t)((row < mrows ? row : 0) * a.in_dim + ((dma_pos ^ G::swz(row)) << 4));
        }
#pragma unroll
        for (int v = 0; v < G::kBInstr; ++v) {
            const int row = (v * G::kWavesG + wave) * 8 + dma_row;
            const int32_t col = b_col(row) < a.out_dim ? b_col(row) : n0;
            b_ptr[v] = wbase + a.code[b_mat(row)] + (int64_t)col * a.in_dim + ((dma_pos ^ G::swz(row)) << 4);
        }
        const uint8_t *a_base = a.x8 + m0 * a.in_dim;
        const int srow = tid % BM;
        const uint8_t *as_base = a.xs + (m0 + (srow < mrows ? srow : 0)) * SB;
        auto dma16 = [&](const uint8_t *src, char *dst) {
            __builtin_amdgcn_global_load_lds((const void *)src,
                                             (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
        };
        auto issue = [&](int32_t kt) {
            char *dst = lds_b + (kt % S) * G::kStageBytes;
            const int64_t k0 = (int64_t)kt * G::kBK;
            const bool tail = k_tail && kt == nk - 1;
#pragma unroll
            for (int v = 0; v < G::kAInstr; ++v) {
                const int row = (v * G::kWavesG + wave) * 8 + dma_row;
                const uint8_t *src = a_base + k0 + a_off[v];
                if (tail && k0 + ((dma_pos ^ G::swz(row)) << 4) >= a.in_dim)
                    src = kZeros;
                dma16(src, dst + (v * G::kWavesG + wave) * 1024);
            }
#pragma unroll
            for (int v = 0; v < G::kBInstr; ++v) {
                const int row = (v * G::kWavesG + wave) * 8 + dma_row;
                const uint8_t *src = b_ptr[v] + k0;
                if (tail && k0 + ((dma_pos ^ G::swz(row)) << 4) >= a.in_dim)
                    src = kZeros;
                dma16(src, dst + BM * G::kBK + (v * G::kWavesG + wave) * 1024);
            }
            __builtin_amdgcn_global_load_lds(
                (const void *)(as_base + (kt >> 2) * 4),
                (__attribute__((address_space(3))) void *)(dst + G::kScaleAt + wave * 256), 4, 0, 0);
        };
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
        // scale row of this wave's B columns (column tile j of gate and up: its
        // matrix); columns past the end are not stored, any row serves them
        auto b_scales = [&](int j) -> const uint32_t * {
            const int32_t last_block = (a.out_dim - 1) / kQuantBlock;
            const int32_t col = n0 + (GLU ? 0 : wn * WN + j * 32);
            const int32_t block = col / kQuantBlock < last_block ? col / kQuantBlock : last_block;
            return (const uint32_t *)(wbase + a.scale[GLU ? j & 1 : 0] + (int64_t)block * SB);
        };

        f32x16 acc[G::kTM][G::kTN];
#pragma unroll
        for (int i = 0; i < G::kTM; ++i)
#pragma unroll
            for (int j = 0; j < G::kTN; ++j)
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    acc[i][j][q] = 0.0f;

#pragma unroll
        for (int st = 0; st + 1 < S; ++st)
            if (st < nk)
                issue(st);
        for (int32_t kt = 0; kt < nk; ++kt) {
            if (kt + S - 2 < nk)
                wait_vm<(S - 2) * G::kPerStage>();
            else
                wait_vm<0>();
            __syncthreads();  // every wave's part of stage kt is there; slot (kt - 1) % S is free
            if (kt + S - 1 < nk)
                issue(kt + S - 1);
            const char *sa = lds_b + (kt % S) * G::kStageBytes;
            const char *sb = sa + BM * G::kBK;
            const int shift = (kt & 3) * 8;
            int sca[G::kTM], scb[G::kTN];
#pragma unroll
            for (int i = 0; i < G::kTM; ++i)
                sca[i] = (int)(*(const uint32_t *)(sa + G::kScaleAt + (wm * WM + i * 32 + fr) * 4) >> shift);
#pragma unroll
            for (int j = 0; j < G::kTN; ++j)
                scb[j] = (int)(b_scales(j)[kt >> 2] >> shift);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                i32x8 fa[G::kTM], fb[G::kTN];
#pragma unroll
                for (int i = 0; i < G::kTM; ++i)
                    fa[i] = frag(sa, wm * WM + i * 32, ks);
#pragma unroll
                for (int j = 0; j < G::kTN; ++j)
                    fb[j] = frag(sb, wn * WN + j * 32, ks);
#pragma unroll
                for (int i = 0; i < G::kTM; ++i)
#pragma unroll
                    for (int j = 0; j < G::kTN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                            fa[i], fb[j], acc[i][j], 0, 0, 0, sca[i], 0, scb[j]);
            }
        }
        __syncthreads();  // the ring is free for the epilogue

        // ---- epilogue, one band of wave rows at a time through LDS -------------
#pragma unroll
        for (int band = 0; band < G::kWM; ++band) {
            if (wm == band) {
#pragma unroll
                for (int i = 0; i < G::kTM; ++i)
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const int row = i * 32 + (q >> 2) * 8 + (lane >> 5) * 4 + (q & 3);
                        if (GLU) {
                            const float g = acc[i][0][q], u = acc[i][G::kTN - 1][q];
                            const float h = g / (1.0f + __expf(-g)) * u;
                            ((float *)lds_b)[row * G::kLdo + wn * 32 + fr] = h;
                        } else {
#pragma unroll
                            for (int j = 0; j < G::kTN; ++j)
                                ((uint16_t *)lds_b)[row * G::kLdo + wn * WN + j * 32 + fr] =
                                    (uint16_t)(pack_bf16(acc[i][j][q], 0.0f) & 0xFFFFu);
                        }
                    }
            }
            __syncthreads();
#pragma unroll
            for (int v = 0; v < G::kOIter; ++v) {
                const int idx = tid + v * G::kThreads;
                const int row = idx / (G::kOutCols / 8), c = idx % (G::kOutCols / 8) * 8;
                const int grow = band * WM + row;
                const bool in = grow < mrows && n0 + c < a.out_dim;
                const int64_t at = (m0 + grow) * a.out_dim + n0 + c;
                if (GLU) {
                    const float *src = (const float *)lds_b + row * G::kLdo + c;
                    float f[8];
                    uint32_t m = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        f[j] = src[j];
                        m = max(m, n0 + c < a.out_dim ? abs_bits(f[j]) : 0u);
                    }
                    const uint32_t byte = scale_byte(row16_max(m));
                    const float inv = inverse_scale(byte);
                    if (in)
                        *(u32x2 *)((uint8_t *)a.out + at) =
                            u32x2{pack_e4m3(f[0], f[1], f[2], f[3], inv, byte),
                                  pack_e4m3(f[4], f[5], f[6], f[7], inv, byte)};
                    if (grow < mrows && c == 0) {
                        uint8_t *dst = a.out_scales + (m0 + grow) * SO;
                        dst[nb] = (uint8_t)byte;
                        if (nb == nbn - 1)
                            for (int32_t p = nbn; p < SO; ++p)
                                dst[p] = 127;
                    }
                } else if (in) {
                    *(u32x4 *)((uint16_t *)a.out + at) =
                        *(const u32x4 *)((const uint16_t *)lds_b + row * G::kLdo + c);
                }
            }
            __syncthreads();
        }
    }
}

namespace {

template <int BM, int BN, int WM, int WN, int S, bool GLU>
int run_quant(const QuantGemmArgs &a, hipStream_t st)
{
    using G = QCfg<BM, BN, WM, WN, S, GLU>;
    const auto kernel = expert_quant_kernel<BM, BN, WM, WN, S, GLU>;
    const size_t ring = (size_t)S * G::kStageBytes;
    const size_t lds = ring + (size_t)(a.seg.E + a.seg.pl.cap + 1) * 4;
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
        return MOONEP_ERR_HIP;
    // Raised once per device, to what the largest allowed E and R need.
    static bool raised[64] = {};
    if (dev < 0 || dev >= 64 || !raised[dev]) {
        const size_t most = ring + (size_t)(2 * kMaxExperts + kMaxRanks + 1) * 4;
        if (hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                (int)most) != hipSuccess)
            return MOONEP_ERR_HIP;
        if (dev >= 0 && dev < 64)
            raised[dev] = true;
    }
    int per_cu = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, kernel, G::kThreads, lds) != hipSuccess)
        return MOONEP_ERR_HIP;
    hipLaunchKernelGGL(kernel, dim3(cus * (per_cu > 0 ? per_cu : 1)), dim3(G::kThreads), lds, st, a);
    return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_ERR_HIP;
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
    if (rows <= (int64_t)32 * s.E)
        return glu ? run_quant<32, 256, 32, 64, 3, true>(a, st)
                   : run_quant<32, 128, 32, 32, 4, false>(a, st);
    return glu ? run_quant<256, 256, 128, 64, 2, true>(a, st)
               : run_quant<256, 256, 128, 64, 2, false>(a, st);
}

}  // namespace moonep
