// quant.hip -- 8-bit rows: the residual's addition with the RMS norm and its
// 8-bit output, the dispatch of 8-bit rows, and expert weights in 8 bits.
//
// All three are HBM-bound streams.  Eight consecutive columns per lane make 16
// lanes (one DPP row) cover a block of 128 columns and a wave cover 512, so a
// block's largest magnitude is four DPP steps and a wave's four scale bytes
// leave as one dword.
#include "quant.hpp"

namespace moonep {

namespace {

// Largest grid, in workgroups; rows beyond it are walked grid-stride.
constexpr int64_t kRowGrid = (int64_t)1 << 20;

__device__ __forceinline__ void unpack8(const u32x4 &w, float (&f)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16_lo(w[j]);
        f[2 * j + 1] = bf16_hi(w[j]);
    }
}

// Eight scaled values as codes.  Non-temporal, as every other store here: in the
// norm of 131072 x 4096 rows write-back stores of the codes alone cost 835 us
// against 808.
__device__ __forceinline__ void store_codes(void *to, const float (&f)[8], float inv, uint32_t byte)
{
    __builtin_nontemporal_store(u32x2{pack_e4m3(f[0], f[1], f[2], f[3], inv, byte),
                                      pack_e4m3(f[4], f[5], f[6], f[7], inv, byte)},
                                (u32x2 *)to);
}

__device__ __forceinline__ float wave_sum(float v)
{
    v = row16_sum(v);
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

}  // namespace

// One row per team of kTeam threads (a wave, or the whole workgroup), kIter
// groups of eight columns per thread in registers: every input is read once.
// Sum of squares in fp32 per thread, then over the wave and the waves; 64 bits
// there change no more codes than the rounding of y does (1e-4 of the output's
// norm either way).  131072 x 4096 with residual and bf16 output: 4.8 GB in 809 us,
// 6.0 TB/s, what a stream of reads and writes reaches.
template <int kTeam, int kIter>
__global__ __launch_bounds__((kTeam == 64 ? kBlock : kTeam)) void rmsnorm_quant_kernel(
    const u32x4 *x, const u32x4 *res, const u32x4 *__restrict__ weight, float eps,
    u32x4 *res_out, u32x4 *__restrict__ y_out, u32x2 *__restrict__ y8, uint32_t *__restrict__ ys,
    int64_t N, int32_t V, int32_t H)
{
    constexpr int kThreads = kTeam == 64 ? kBlock : kTeam;  // several waves of one row each
    constexpr int kTeams = kThreads / kTeam, kTeamWaves = kTeam / 64;
    __shared__ float part[2][kTeamWaves];
    const int t = (int)threadIdx.x % kTeam, lane = lane_id();
    const int32_t SD = scale_row_bytes(H) / 4;
    constexpr bool kKeepWeight = kIter <= 4;  // else read again each row, from the L2
    u32x4 w[kIter];
#pragma unroll
    for (int i = 0; i < kIter && kKeepWeight; ++i) {
        const int32_t v = i * kTeam + t;
        w[i] = v < V ? weight[v] : u32x4{0, 0, 0, 0};
    }
    int flip = 0;
    for (int64_t row = (int64_t)blockIdx.x * kTeams + (int)threadIdx.x / kTeam; row < N;
         row += (int64_t)gridDim.x * kTeams) {
        u32x4 r[kIter], a[kIter];
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const int32_t v = i * kTeam + t;
            r[i] = v < V ? load_nt(x + row * V + v) : u32x4{0, 0, 0, 0};
            if (res)
                a[i] = v < V ? load_nt(res + row * V + v) : u32x4{0, 0, 0, 0};
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            float f[8];
            unpack8(r[i], f);
            if (res) {
                float g[8];
                unpack8(a[i], g);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    r[i][j] = pack_bf16(f[2 * j] + g[2 * j], f[2 * j + 1] + g[2 * j + 1]);
                const int32_t v = i * kTeam + t;
                if (v < V)
                    store_nt(res_out + row * V + v, r[i]);
                unpack8(r[i], f);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                ss = __builtin_fmaf(f[j], f[j], ss);
        }
        ss = wave_sum(ss);
        if (kTeamWaves > 1) {
            // two buffers in turn, so one barrier a row is enough
            if (lane == 0)
                part[flip][t >> 6] = ss;
            __syncthreads();
            ss = 0.0f;
#pragma unroll
            for (int q = 0; q < kTeamWaves; ++q)
                ss += part[flip][q];
            flip ^= 1;
        }
        const float rstd = 1.0f / sqrtf(ss / (float)H + eps);
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const int32_t v = i * kTeam + t;
            float f[8], g[8];
            unpack8(r[i], f);
            if (!kKeepWeight)
                w[i] = v < V ? weight[v] : u32x4{0, 0, 0, 0};
            unpack8(w[i], g);
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f[j] = f[j] * rstd * g[j];
                m = max(m, v < V ? abs_bits(f[j]) : 0u);
            }
            const uint32_t byte = scale_byte(row16_max(m));
            const float inv = inverse_scale(byte);
            const uint32_t dword = gather_scale_dword(byte);
            if (v < V) {
                store_codes(y8 + row * V + v, f, inv, byte);
                if (y_out)
                    store_nt(y_out + row * V + v,
                             u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                   pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])});
            }
            const int32_t q = v >> 6;  // the wave's 512 columns
            if (lane == 0 && q < SD)
                ys[row * SD + q] = dword;
        }
    }
}

// One wave per (token, 1 KiB of codes): the codes, and with the first piece the
// token's scales, go to each of its K rows: every code is read once.  32768 tokens
// of 2048 codes to 8 rows each: 0.61 GB in 116 us, 5.25 TB/s; copies of rows to
// random places reach 5.28.
__global__ __launch_bounds__(kBlock) void dispatch_quant_kernel(
    const u32x4 *__restrict__ x8, const uint32_t *__restrict__ xs, const int32_t *slot_of,
    u32x4 *buf8, uint32_t *bufs, int64_t N, int32_t V, int32_t pieces, int32_t SD, int32_t K,
    uint32_t nrows)
{
    const int lane = lane_id();
    const int64_t total = N * pieces;
    for (int64_t w = (int64_t)blockIdx.x * kWaves + ((int)threadIdx.x >> 6); w < total;
         w += (int64_t)gridDim.x * kWaves) {
        const int64_t tok = w / pieces;
        const int32_t piece = (int32_t)(w - tok * pieces);
        const int32_t v = piece * 64 + lane;
        const int32_t *so = slot_of + tok * K;
        u32x4 val = {0, 0, 0, 0};
        if (v < V)
            val = load_nt(x8 + tok * V + v);
        for (int32_t k = 0; k < K; ++k) {
            const uint32_t sk = (uint32_t)so[k];
            if (sk < nrows && v < V)
                store_nt(buf8 + (int64_t)sk * V + v, val);
        }
        if (piece == 0)
            for (int32_t c = lane; c < SD; c += 64) {
                const uint32_t s = xs[tok * SD + c];
                for (int32_t k = 0; k < K; ++k) {
                    const uint32_t sk = (uint32_t)so[k];
                    if (sk < nrows)
                        bufs[(int64_t)sk * SD + c] = s;
                }
            }
    }
}

// An item is 128 rows x 512 columns (four blocks): wave w holds rows w, w + 16,
// .. of it in registers between the blocks' magnitudes and their codes, and the
// next item's rows are on their way meanwhile (the barrier waits for LDS alone).
// On 64 experts of 1408 x 2048: 112-114 us, 4.9 TB/s; without the next item's
// loads 124, one block of 128 x 128 per workgroup (256-byte row pieces) 177,
// write-back code stores 131.
constexpr int kWqWaves = 16, kWqRows = kQuantBlock / kWqWaves;
constexpr int64_t kWqGrid = 512;

__global__ __launch_bounds__(kWqWaves * 64) void quant_weights_kernel(
    const uint16_t *__restrict__ w, int64_t w_stride, int64_t w_offset, uint8_t *__restrict__ w8,
    int64_t w8_stride, int64_t code_offset, int64_t scale_offset, int64_t items, int32_t out_dim,
    int32_t in_dim, int32_t nrb, int32_t ncb)
{
    __shared__ uint32_t part[2][kWqWaves][4];
    const int lane = lane_id(), wave = (int)threadIdx.x >> 6;
    int flip = 0;
    // Rows of item `it` into r; rows and columns past the matrix are 0.
    auto load = [&](int64_t it, u32x4 (&r)[kWqRows]) {
        const int32_t cb = (int32_t)(it % ncb), rb = (int32_t)(it / ncb % nrb);
        const int32_t col = cb * 512 + lane * 8, row0 = rb * kQuantBlock + wave;
        const uint16_t *src = w + it / ncb / nrb * w_stride + w_offset + (int64_t)row0 * in_dim + col;
#pragma unroll
        for (int i = 0; i < kWqRows; ++i) {
            r[i] = u32x4{0, 0, 0, 0};
            if (row0 + i * kWqWaves < out_dim && col < in_dim)
                r[i] = load_nt((const u32x4 *)(src + (int64_t)(i * kWqWaves) * in_dim));
        }
    };
    u32x4 nxt[kWqRows];
    load(blockIdx.x, nxt);
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int32_t cb = (int32_t)(it % ncb), rb = (int32_t)(it / ncb % nrb);
        const int32_t col = cb * 512 + lane * 8, row0 = rb * kQuantBlock + wave;
        uint8_t *dst = w8 + it / ncb / nrb * w8_stride;
        uint8_t *code = dst + code_offset + (int64_t)row0 * in_dim + col;
        u32x4 r[kWqRows];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kWqRows; ++i) {
            r[i] = nxt[i];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                m = max(m, max((r[i][j] << 16) & 0x7FFF0000u, r[i][j] & 0x7FFF0000u));
        }
        if (it + gridDim.x < items)
            load(it + gridDim.x, nxt);
        m = row16_max(m);
        if ((lane & 15) == 0)
            part[flip][wave][lane >> 4] = m;
        lds_barrier();
#pragma unroll
        for (int q = 0; q < kWqWaves; ++q)
            m = max(m, part[flip][q][lane >> 4]);
        flip ^= 1;
        const uint32_t byte = scale_byte(m);
        const float inv = inverse_scale(byte);
        const uint32_t dword = gather_scale_dword(byte);
        if (threadIdx.x == 0)
            *(uint32_t *)(dst + scale_offset + ((int64_t)rb * ncb + cb) * 4) = dword;
#pragma unroll
        for (int i = 0; i < kWqRows; ++i) {
            float f[8];
            unpack8(r[i], f);
            if (row0 + i * kWqWaves < out_dim && col < in_dim)
                store_codes(code + (int64_t)(i * kWqWaves) * in_dim, f, inv, byte);
        }
    }
}

namespace {

int last() { return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_ERR_HIP; }

template <int kTeam, int kIter>
int run_rmsnorm(const moonep_shape &s, const uint16_t *x, const uint16_t *res,
                const uint16_t *weight, float eps, uint16_t *res_out, uint16_t *y_out, uint8_t *y8,
                uint8_t *ys, hipStream_t st)
{
    constexpr int kThreads = kTeam == 64 ? kBlock : kTeam;
    const int64_t N = (int64_t)s.R * s.S, per = kThreads / kTeam;
    const int64_t blocks = (N + per - 1) / per;
    const dim3 grid((uint32_t)(blocks < kRowGrid ? blocks : kRowGrid));
    hipLaunchKernelGGL((rmsnorm_quant_kernel<kTeam, kIter>), grid, dim3(kThreads), 0, st,
                       (const u32x4 *)x, (const u32x4 *)res, (const u32x4 *)weight, eps,
                       (u32x4 *)res_out, (u32x4 *)y_out, (u32x2 *)y8, (uint32_t *)ys, N, s.H / 8,
                       s.H);
    return last();
}

}  // namespace

int launch_rmsnorm_quant(const moonep_shape &s, const uint16_t *x, const uint16_t *res,
                         const uint16_t *weight, float eps, uint16_t *res_out, uint16_t *y_out,
                         uint8_t *y8, uint8_t *ys, hipStream_t st)
{
    if ((int64_t)s.R * s.S == 0)
        return MOONEP_OK;
    // Threads of a row, and groups of eight columns of each: a wave without a
    // barrier up to 1024 columns, then two to four groups a thread.  Measured with
    // residual and bf16 output, TB/s: H = 1024 6.0 (256 threads, one group: 5.5),
    // 2048 6.1 (256 x 1: 5.9), 4096 6.0 (512 x 1: 6.1, 512 x 2: 5.6), 7168 6.0
    // (512 x 2: 5.9, 1024 x 1: 6.0).
    if (s.H <= 512)
        return run_rmsnorm<64, 1>(s, x, res, weight, eps, res_out, y_out, y8, ys, st);
    if (s.H <= 1024)
        return run_rmsnorm<64, 2>(s, x, res, weight, eps, res_out, y_out, y8, ys, st);
    if (s.H <= 2048)
        return run_rmsnorm<128, 2>(s, x, res, weight, eps, res_out, y_out, y8, ys, st);
    if (s.H <= 4096)
        return run_rmsnorm<256, 2>(s, x, res, weight, eps, res_out, y_out, y8, ys, st);
    if (s.H <= 8192)
        return run_rmsnorm<256, 4>(s, x, res, weight, eps, res_out, y_out, y8, ys, st);
    if (s.H <= 16384)
        return run_rmsnorm<1024, 2>(s, x, res, weight, eps, res_out, y_out, y8, ys, st);
    if (s.H <= 32768)  // 512 threads: twice the registers a thread
        return run_rmsnorm<512, 8>(s, x, res, weight, eps, res_out, y_out, y8, ys, st);
    return run_rmsnorm<1024, 8>(s, x, res, weight, eps, res_out, y_out, y8, ys, st);
}

int launch_dispatch_quant(const moonep_shape &s, const uint8_t *x8, const uint8_t *xs,
                          const int32_t *slot_of, uint8_t *buf8, uint8_t *bufs, hipStream_t st)
{
    const int64_t N = (int64_t)s.R * s.S;
    if (N == 0)
        return MOONEP_OK;
    const int32_t V = s.H / 16, pieces = (V + 63) / 64, SD = scale_row_bytes(s.H) / 4;
    const int64_t blocks = (N * pieces + kWaves - 1) / kWaves;
    const dim3 grid((uint32_t)(blocks < kRowGrid ? blocks : kRowGrid));
    hipLaunchKernelGGL(dispatch_quant_kernel, grid, dim3(kBlock), 0, st, (const u32x4 *)x8,
                       (const uint32_t *)xs, slot_of, (u32x4 *)buf8, (uint32_t *)bufs, N, V, pieces,
                       SD, s.K, (uint32_t)(N * s.K));
    return last();
}

int launch_quant_weights(const moonep_shape &s, int32_t in_dim, int32_t out_dim, const uint16_t *w,
                         int64_t w_stride, int64_t w_offset, uint8_t *w8, int64_t w8_stride,
                         int64_t code_offset, int64_t scale_offset, hipStream_t st)
{
    const int32_t nrb = (out_dim - 1) / kQuantBlock + 1;
    const int32_t ncb = scale_row_bytes(in_dim) / 4;
    const int64_t items = (int64_t)s.E * nrb * ncb;
    const dim3 grid((uint32_t)(items < kWqGrid ? items : kWqGrid));
    hipLaunchKernelGGL(quant_weights_kernel, grid, dim3(kWqWaves * 64), 0, st, w, w_stride,
                       w_offset, w8, w8_stride, code_offset, scale_offset, items, out_dim, in_dim,
                       nrb, ncb);
    return last();
}

}  // namespace moonep
