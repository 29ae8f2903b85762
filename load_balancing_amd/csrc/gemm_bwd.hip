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
// stays as it is in memory in its stage, [kBK rows][columns], and
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
#include "segments.hpp"

namespace moonep {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

namespace {

constexpr int kBK = 64;  // contraction per LDS stage

// A lane's byte offset in a transposed stage of rows of RB bytes, for 32-column
// tile 0 and k-step 0; tile T is at offset ^ (T << 6), k-step ks at + ks 16 RB.
template <int RB>
__device__ __forceinline__ int tr_offset(int lane)
{
    const int row = (lane >> 5) * 8 + ((lane & 15) >> 2);
    return row * RB + ((row & 3) << 6) + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
}

template <int RB>
__device__ __forceinline__ bf16x8 tr_frag(const char *p)
{
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(void *)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(void *)(p + 4 * RB));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ void dma16(const char *src, char *dst)
{
    __builtin_amdgcn_global_load_lds((const void *)src,
                                     (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
}

// Waits until at most N vector-memory operations of this wave are outstanding.
template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N >= 0 && N <= 63, "vmcnt");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

// ---------------------------------------------------------------------------
// d_x: rows of d_y against W, contracted over W's rows
// ---------------------------------------------------------------------------

template <int BM, int BN, int WM, int WN, int S>
struct DxCfg {
    static constexpr int kTM = WM / 32, kTN = WN / 32;
    static constexpr int kWM = BM / WM, kWN = BN / WN;
    static constexpr int kWavesG = kWM * kWN;
    static constexpr int kThreads = kWavesG * 64;
    static constexpr int kRowA = kBK * 2, kRowB = BN * 2;  // bytes of a stage row
    static constexpr int kStageA = BM * kRowA, kStageB = kBK * kRowB;
    static constexpr int kStageBytes = kStageA + kStageB;
    static constexpr int kAInstr = kStageA / 1024 / kWavesG, kBInstr = kStageB / 1024 / kWavesG;
    static constexpr int kPerStage = kAInstr + kBInstr;
    static constexpr int kLdo = BN + 8;
    static constexpr int kOVec = WM * BN / 8 / kThreads;
    static_assert(WM * kLdo * 2 <= S * kStageBytes, "an epilogue band must fit the ring");
    static_assert(kStageA % (1024 * kWavesG) == 0 && kStageB % (1024 * kWavesG) == 0, "DMA rounds");
    static_assert((S - 2) * kPerStage <= 63, "outstanding loads must fit vmcnt");
    // 16-byte chunk c of row r of the A part sits at c ^ swz(r), as in gemm.hip
    __device__ static constexpr int swz(int r) { return (r / 2) % 8; }
};

struct DxArgs {
    SegTables seg;
    int32_t in_dim, out_dim;
    const uint16_t *d_y, *w_home, *pool;
    int64_t w_stride, w_offset;
    uint16_t *d_x;
};

constexpr int kGroupM = 8;  // row tiles per item group, as in gemm.hip

template <int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__((DxCfg<BM, BN, WM, WN, S>::kThreads)) void expert_dx_kernel(DxArgs a)
{
    using G = DxCfg<BM, BN, WM, WN, S>;
    extern __shared__ __align__(16) uint16_t lds[];
    char *ring = (char *)lds;
    int32_t *seg_start = (int32_t *)(ring + S * G::kStageBytes);  // [E + cap + 1]
    __shared__ int scan_tmp[G::kWavesG];

    const int tid = (int)threadIdx.x, lane = lane_id(), wave = tid >> 6;
    const int32_t nseg = a.seg.E + a.seg.n_rep();
    const int32_t total_tiles = scan_tiles<BM, G::kWavesG>(a.seg, nseg, seg_start, scan_tmp);
    const int32_t nbn = (a.in_dim + BN - 1) / BN;  // the last block may be part-empty
    const int64_t items = (int64_t)total_tiles * nbn;
    const int P = (int)gridDim.x;
    const int slot = xcd_slot((int)blockIdx.x, P);
    const int32_t nk = a.out_dim / kBK;
    const int wm = wave / G::kWN, wn = wave % G::kWN;

    for (int64_t it = slot; it < items; it += P) {
        int32_t t, nb;
        item_of<kGroupM>(it, total_tiles, nbn, &t, &nb);
        const int32_t s = find_segment(seg_start, nseg, t);
        const int32_t mt = t - seg_start[s];
        int64_t wrow;
        bool pooled;
        int32_t len;
        const int64_t row0 = a.seg.segment(s, &len, &wrow, &pooled);
        const uint16_t *wbase = (pooled ? a.pool : a.w_home) + wrow * a.w_stride + a.w_offset;
        const int64_t m0 = row0 + (int64_t)mt * BM;
        const int32_t mrows = len - mt * BM < BM ? len - mt * BM : BM;
        const int32_t n0 = nb * BN;

        uint32_t a_off[G::kAInstr], b_off[G::kBInstr];
#pragma unroll
        for (int v = 0; v < G::kAInstr; ++v) {
            const int row = (v * G::kWavesG + wave) * 8 + lane / 8;
            const int chunk = (lane % 8) ^ G::swz(row);
            a_off[v] = (uint32_t)(row < mrows ? row : 0) * (uint32_t)a.out_dim * 2 + chunk * 16;
        }
#pragma unroll
        for (int v = 0; v < G::kBInstr; ++v) {
            constexpr int kCpr = G::kRowB / 16;
            const int at = (v * G::kWavesG + wave) * 64 + lane;
            const int row = at / kCpr, chunk = (at % kCpr) ^ ((row & 3) << 2);
            const int32_t col = n0 + chunk * 8;
            b_off[v] = (uint32_t)row * (uint32_t)a.in_dim * 2 + (uint32_t)(col < a.in_dim ? col : 0) * 2;
        }
        const char *a_base = (const char *)(a.d_y + m0 * a.out_dim);
        const char *b_base = (const char *)wbase;
        const int64_t b_step = (int64_t)kBK * a.in_dim * 2;
        auto issue = [&](int32_t kt, int st) {
            char *dst = ring + st * G::kStageBytes + wave * 1024;
            const char *ap = a_base + (int64_t)kt * G::kRowA;
            const char *bp = b_base + kt * b_step;
#pragma unroll
            for (int v = 0; v < G::kAInstr; ++v)
                dma16(ap + a_off[v], dst + v * G::kWavesG * 1024);
#pragma unroll
            for (int v = 0; v < G::kBInstr; ++v)
                dma16(bp + b_off[v], dst + G::kStageA + v * G::kWavesG * 1024);
        };
        const int fr = lane & 31, fsw = G::swz(lane & 31), fhalf = lane >> 5;
        auto frag_a = [&](const char *base, int row0, int ks) -> bf16x8 {
            return *(const bf16x8 *)(base + (row0 + fr) * G::kRowA + (((2 * ks + fhalf) ^ fsw) << 4));
        };
        const int tr0 = tr_offset<G::kRowB>(lane);
        auto frag_b = [&](const char *base, int tile, int ks) -> bf16x8 {
            return tr_frag<G::kRowB>(base + (tr0 ^ (tile << 6)) + ks * 16 * G::kRowB);
        };

        f32x16 acc[G::kTM][G::kTN];
#pragma unroll
        for (int i = 0; i < G::kTM; ++i)
#pragma unroll
            for (int j = 0; j < G::kTN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[i][j][r] = 0.0f;

#pragma unroll
        for (int st = 0; st + 1 < S; ++st)
            if (st < nk)
                issue(st, st);
        for (int32_t kt = 0; kt < nk; ++kt) {
            // this wave's loads of stage kt have landed once at most the later
            // stages' loads are outstanding
            if (kt + S - 2 < nk)
                wait_vm<(S - 2) * G::kPerStage>();
            else
                wait_vm<0>();
            __syncthreads();  // stage kt is visible to all; slot (kt - 1) % S is free
            if (kt + S - 1 < nk)
                issue(kt + S - 1, (kt + S - 1) % S);
            const char *sa = ring + (kt % S) * G::kStageBytes;
            const char *sb = sa + G::kStageA;
            bf16x8 fa[2][G::kTM], fb[2][G::kTN];
#pragma unroll
            for (int i = 0; i < G::kTM; ++i)
                fa[0][i] = frag_a(sa, wm * WM + i * 32, 0);
#pragma unroll
            for (int j = 0; j < G::kTN; ++j)
                fb[0][j] = frag_b(sb, wn * G::kTN + j, 0);
#pragma unroll
            for (int ks = 0; ks < kBK / 16; ++ks) {
                const int cur = ks & 1, nxt = cur ^ 1;
                if (ks + 1 < kBK / 16) {
#pragma unroll
                    for (int i = 0; i < G::kTM; ++i)
                        fa[nxt][i] = frag_a(sa, wm * WM + i * 32, ks + 1);
#pragma unroll
                    for (int j = 0; j < G::kTN; ++j)
                        fb[nxt][j] = frag_b(sb, wn * G::kTN + j, ks + 1);
                }
#pragma unroll
                for (int i = 0; i < G::kTM; ++i)
#pragma unroll
                    for (int j = 0; j < G::kTN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[cur][i], fb[cur][j],
                                                                            acc[i][j], 0, 0, 0);
            }
        }
        __syncthreads();  // every wave is done with the ring before the epilogue reuses it

        // epilogue: one band of wave rows at a time through LDS, as in gemm.hip
        uint16_t *so = lds;
#pragma unroll
        for (int band = 0; band < G::kWM; ++band) {
            if (wm == band) {
#pragma unroll
                for (int i = 0; i < G::kTM; ++i)
#pragma unroll
                    for (int j = 0; j < G::kTN; ++j)
#pragma unroll
                        for (int r = 0; r < 16; r += 2) {
                            const int row = i * 32 + (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3);
                            const int col = wn * WN + j * 32 + (lane & 31);
                            const uint32_t p = pack_bf16(acc[i][j][r], acc[i][j][r + 1]);
                            so[row * G::kLdo + col] = (uint16_t)(p & 0xFFFFu);
                            so[(row + 1) * G::kLdo + col] = (uint16_t)(p >> 16);
                        }
            }
            __syncthreads();
#pragma unroll
            for (int v = 0; v < G::kOVec; ++v) {
                const int idx = tid + v * G::kThreads;
                const int row = idx / (BN / 8), c = idx % (BN / 8);
                const int grow = band * WM + row;
                if (grow < mrows && n0 + c * 8 < a.in_dim)
                    *(u32x4 *)(a.d_x + (m0 + grow) * a.in_dim + n0 + c * 8) =
                        *(const u32x4 *)(so + row * G::kLdo + c * 8);
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------------------
// g: both operands contracted over the segment's rows
// ---------------------------------------------------------------------------

template <int BM, int BN, int WM, int WN, int S>
struct DwCfg {
    static constexpr int kTM = WM / 32, kTN = WN / 32;
    static constexpr int kWM = BM / WM, kWN = BN / WN;
    static constexpr int kWavesG = kWM * kWN;
    static constexpr int kThreads = kWavesG * 64;
    static constexpr int kRowA = BM * 2, kRowB = BN * 2;
    static constexpr int kStageA = kBK * kRowA, kStageB = kBK * kRowB;
    static constexpr int kStageBytes = kStageA + kStageB;
    static constexpr int kAInstr = kStageA / 1024 / kWavesG, kBInstr = kStageB / 1024 / kWavesG;
    static constexpr int kPerStage = kAInstr + kBInstr;
    static_assert(kStageA % (1024 * kWavesG) == 0 && kStageB % (1024 * kWavesG) == 0, "DMA rounds");
    static_assert((S - 2) * kPerStage <= 63, "outstanding loads must fit vmcnt");
};

struct DwArgs {
    SegTables seg;
    int32_t in_dim, out_dim, accumulate;
    const uint16_t *x, *d_y;
    int64_t G, g_offset;
    float *home, *rep;
};

// What the rows behind a segment's last are read as: zeros, so that they add
// nothing whatever the buffer holds there.
__device__ const uint32_t g_zero_row[4] = {0, 0, 0, 0};

template <int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__((DwCfg<BM, BN, WM, WN, S>::kThreads)) void expert_dw_kernel(DwArgs a)
{
    using G = DwCfg<BM, BN, WM, WN, S>;
    extern __shared__ __align__(16) uint16_t lds[];
    char *ring = (char *)lds;
    const int tid = (int)threadIdx.x, lane = lane_id(), wave = tid >> 6;
    const int32_t nseg = a.seg.E + a.seg.n_rep();
    const int32_t nbm = (a.out_dim + BM - 1) / BM, nbn = (a.in_dim + BN - 1) / BN;
    const int64_t per = (int64_t)nbm * nbn, items = nseg * per;
    const int P = (int)gridDim.x;
    const int wm = wave / G::kWN, wn = wave % G::kWN;

    for (int64_t it = xcd_slot((int)blockIdx.x, P); it < items; it += P) {
        const int32_t s = (int32_t)(it / per), within = (int32_t)(it - s * per);
        const int32_t mb = within % nbm, nb = within / nbm;
        const int32_t m0 = mb * BM, n0 = nb * BN;
        const int32_t len = __builtin_amdgcn_readfirstlane(a.seg.rows(s));
        const int64_t row0 = len ? a.seg.first_row(s) : 0;
        float *out = s < a.seg.E ? a.home + s * a.G : a.rep + (int64_t)(s - a.seg.E) * a.G;
        out += a.g_offset;

        uint32_t a_off[G::kAInstr], b_off[G::kBInstr];
        int a_row[G::kAInstr], b_row[G::kBInstr];
#pragma unroll
        for (int v = 0; v < G::kAInstr; ++v) {
            constexpr int kCpr = G::kRowA / 16;
            const int at = (v * G::kWavesG + wave) * 64 + lane;
            const int row = at / kCpr, chunk = (at % kCpr) ^ ((row & 3) << 2);
            const int32_t col = m0 + chunk * 8;
            a_row[v] = row;
            a_off[v] = (uint32_t)row * (uint32_t)a.out_dim * 2 + (uint32_t)(col < a.out_dim ? col : 0) * 2;
        }
#pragma unroll
        for (int v = 0; v < G::kBInstr; ++v) {
            constexpr int kCpr = G::kRowB / 16;
            const int at = (v * G::kWavesG + wave) * 64 + lane;
            const int row = at / kCpr, chunk = (at % kCpr) ^ ((row & 3) << 2);
            const int32_t col = n0 + chunk * 8;
            b_row[v] = row;
            b_off[v] = (uint32_t)row * (uint32_t)a.in_dim * 2 + (uint32_t)(col < a.in_dim ? col : 0) * 2;
        }
        const char *a_base = (const char *)(a.d_y + row0 * a.out_dim);
        const char *b_base = (const char *)(a.x + row0 * a.in_dim);
        const int64_t a_step = (int64_t)kBK * a.out_dim * 2, b_step = (int64_t)kBK * a.in_dim * 2;
        const char *zero = (const char *)g_zero_row;
        auto issue = [&](int32_t kt, int st) {
            char *dst = ring + st * G::kStageBytes + wave * 1024;
            const char *ap = a_base + kt * a_step;
            const char *bp = b_base + kt * b_step;
            const int32_t left = len - kt * kBK;
#pragma unroll
            for (int v = 0; v < G::kAInstr; ++v)
                dma16(a_row[v] < left ? ap + a_off[v] : zero, dst + v * G::kWavesG * 1024);
#pragma unroll
            for (int v = 0; v < G::kBInstr; ++v)
                dma16(b_row[v] < left ? bp + b_off[v] : zero, dst + G::kStageA + v * G::kWavesG * 1024);
        };
        const int tra = tr_offset<G::kRowA>(lane), trb = tr_offset<G::kRowB>(lane);
        auto frag_a = [&](const char *base, int tile, int ks) -> bf16x8 {
            return tr_frag<G::kRowA>(base + (tra ^ (tile << 6)) + ks * 16 * G::kRowA);
        };
        auto frag_b = [&](const char *base, int tile, int ks) -> bf16x8 {
            return tr_frag<G::kRowB>(base + (trb ^ (tile << 6)) + ks * 16 * G::kRowB);
        };

        f32x16 acc[G::kTM][G::kTN];
#pragma unroll
        for (int i = 0; i < G::kTM; ++i)
#pragma unroll
            for (int j = 0; j < G::kTN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[i][j][r] = 0.0f;

        const int32_t nk = (len + kBK - 1) / kBK;
        __syncthreads();  // the item before is done with the ring
#pragma unroll
        for (int st = 0; st + 1 < S; ++st)
            if (st < nk)
                issue(st, st);
        for (int32_t kt = 0; kt < nk; ++kt) {
            if (kt + S - 2 < nk)
                wait_vm<(S - 2) * G::kPerStage>();
            else
                wait_vm<0>();
            __syncthreads();
            if (kt + S - 1 < nk)
                issue(kt + S - 1, (kt + S - 1) % S);
            const char *sa = ring + (kt % S) * G::kStageBytes;
            const char *sb = sa + G::kStageA;
            bf16x8 fa[2][G::kTM], fb[2][G::kTN];
#pragma unroll
            for (int i = 0; i < G::kTM; ++i)
                fa[0][i] = frag_a(sa, wm * G::kTM + i, 0);
#pragma unroll
            for (int j = 0; j < G::kTN; ++j)
                fb[0][j] = frag_b(sb, wn * G::kTN + j, 0);
#pragma unroll
            for (int ks = 0; ks < kBK / 16; ++ks) {
                const int cur = ks & 1, nxt = cur ^ 1;
                if (ks + 1 < kBK / 16) {
#pragma unroll
                    for (int i = 0; i < G::kTM; ++i)
                        fa[nxt][i] = frag_a(sa, wm * G::kTM + i, ks + 1);
#pragma unroll
                    for (int j = 0; j < G::kTN; ++j)
                        fb[nxt][j] = frag_b(sb, wn * G::kTN + j, ks + 1);
                }
#pragma unroll
                for (int i = 0; i < G::kTM; ++i)
#pragma unroll
                    for (int j = 0; j < G::kTN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[cur][i], fb[cur][j],
                                                                            acc[i][j], 0, 0, 0);
            }
        }
        // a register's 32 lanes hold 32 consecutive columns: whole 128-byte lines
#pragma unroll
        for (int i = 0; i < G::kTM; ++i)
#pragma unroll
            for (int j = 0; j < G::kTN; ++j) {
                const int32_t row = m0 + wm * WM + i * 32 + (lane >> 5) * 4;
                const int32_t col = n0 + wn * WN + j * 32 + (lane & 31);
                if (m0 + wm * WM + i * 32 < a.out_dim && n0 + wn * WN + j * 32 < a.in_dim) {
                    float *p = out + (int64_t)row * a.in_dim + col;
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
                        p[(int64_t)((r >> 2) * 8 + (r & 3)) * a.in_dim] = acc[i][j][r];
                }
            }
    }
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

template <int BM, int BN, int WM, int WN, int S>
int run_dx(const DxArgs &a, hipStream_t st)
{
    using G = DxCfg<BM, BN, WM, WN, S>;
    constexpr size_t kRing = (size_t)S * G::kStageBytes;
    static bool raised[64] = {};
    int cus = 0;
    const int rc = prepare_launch(expert_dx_kernel<BM, BN, WM, WN, S>,
                                  kRing + (size_t)(2 * kMaxExperts + kMaxRanks + 1) * 4, raised, &cus);
    if (rc != MOONEP_OK)
        return rc;
    const size_t bytes = kRing + (size_t)(a.seg.E + a.seg.pl.cap + 1) * 4;
    const int per_cu = (int)((160u << 10) / bytes);
    hipLaunchKernelGGL((expert_dx_kernel<BM, BN, WM, WN, S>), dim3(cus * (per_cu > 1 ? 2 : 1)),
                       dim3(G::kThreads), bytes, st, a);
    return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_ERR_HIP;
}

template <int BM, int BN, int WM, int WN, int S>
int run_dw(const DwArgs &a, hipStream_t st)
{
    using G = DwCfg<BM, BN, WM, WN, S>;
    constexpr size_t kRing = (size_t)S * G::kStageBytes;
    static bool raised[64] = {};
    int cus = 0;
    const int rc = prepare_launch(expert_dw_kernel<BM, BN, WM, WN, S>, kRing, raised, &cus);
    if (rc != MOONEP_OK)
        return rc;
    const int per_cu = (int)((160u << 10) / kRing);
    hipLaunchKernelGGL((expert_dw_kernel<BM, BN, WM, WN, S>), dim3(cus * (per_cu > 1 ? 2 : 1)),
                       dim3(G::kThreads), kRing, st, a);
    return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_ERR_HIP;
}

}  // namespace

int launch_expert_dx(const moonep_shape &s, const int32_t *plan, const int32_t *wslot, int32_t B,
                     int32_t in_dim, int32_t out_dim, const uint16_t *d_y, const uint16_t *w_home,
                     const uint16_t *pool, int64_t w_stride, int64_t w_offset, uint16_t *d_x,
                     hipStream_t st)
{
    if ((int64_t)s.R * s.S * s.K == 0)
        return MOONEP_OK;
    const DxArgs a{seg_tables(s, plan, wslot, B), in_dim, out_dim, d_y, w_home, pool,
                   w_stride, w_offset, d_x};
    return run_dx<256, 256, 128, 64, 2>(a, st);
}

int launch_expert_dw(const moonep_shape &s, const int32_t *plan, int32_t in_dim, int32_t out_dim,
                     const uint16_t *x, const uint16_t *d_y, int accumulate, int64_t G,
                     int64_t g_offset, float *home, float *rep, hipStream_t st)
{
    if (accumulate && (int64_t)s.R * s.S * s.K == 0)
        return MOONEP_OK;
    const DwArgs a{seg_tables(s, plan, nullptr, 0), in_dim, out_dim, accumulate, x, d_y, G, g_offset,
                   home, rep};
    return run_dw<256, 256, 128, 64, 2>(a, st);
}

}  // namespace moonep
