// grads.hip -- the norm over many gradient tensors and their clipping.
//
//   norm = sqrt(sum over every element of g^2),
//   out  = g * (max_norm / norm if norm > max_norm and finite, else 1).
//
// The tensors are a device table of runs (address, address of the output,
// elements, type), so that one launch covers any number of them.  Squares of
// fp32 values are exact in fp64 and cannot overflow there; every thread sums
// its own in fp64, a workgroup joins its threads', and the workgroups' sums are
// joined in a fixed order: the same table gives the same bits on the same
// device.
//
// Two passes over the gradients are needed, the factor being known only after
// the first; the second walks the runs from the last to the first, so that what
// the first read last is still in the 256 MiB memory-side cache.  Its loads and its
// stores are non-temporal: it is the last to read the gradients, and written lines
// that stay in the caches have to leave them while the next kernel reads
// (192 tensors of 2.9e6 fp32: 1244 -> 1179 us; 448 of 3e4 to 7e4: 55.7 -> 46.2).
#include "moonep_internal.hpp"

namespace moonep {

namespace {

constexpr int kGradBlock = 256;
constexpr int kGradWaves = kGradBlock / 64;
constexpr int kGradGrid = 2048;  // workgroups, and so sums in the workspace, at most
constexpr int kUnroll = 8;       // 16-byte loads in flight per thread

struct GradRun {
    uint64_t src, dst;
    int64_t count, type;
};
static_assert(sizeof(GradRun) == 32, "four words");

// Addresses out of the table are global memory: told so, the compiler makes
// global accesses of them, not flat ones.
#define MOONEP_GLOBAL __attribute__((address_space(1)))
typedef const MOONEP_GLOBAL char *gsrc;
typedef MOONEP_GLOBAL char *gdst;

// Sixteen bytes at an address that is a multiple of the element size only.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ u32x4 load16(gsrc p) { return *(const MOONEP_GLOBAL u32x4_any *)p; }
__device__ __forceinline__ u32x4 load16_nt(gsrc p)
{
    return __builtin_nontemporal_load((const MOONEP_GLOBAL u32x4_any *)p);
}
__device__ __forceinline__ void store16_nt(gdst p, u32x4 v)
{
    __builtin_nontemporal_store(v, (MOONEP_GLOBAL u32x4_any *)p);
}

__device__ __forceinline__ float load1(gsrc p, bool bf16)
{
    return bf16 ? bf16_lo(*(const MOONEP_GLOBAL uint16_t *)p) : *(const MOONEP_GLOBAL float *)p;
}

// Sum of one value per thread over the workgroup, in every thread.
__device__ __forceinline__ double block_sum(double v, double *tmp)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v += __shfl_xor(v, d, 64);
    if (lane_id() == 0)
        tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < kGradWaves; ++w)
        sum += tmp[w];
    __syncthreads();
    return sum;
}

template <bool kBf16>
__device__ __forceinline__ double square_sum(u32x4 v)
{
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kBf16) {
            const double a = bf16_lo(v[i]), b = bf16_hi(v[i]);
            s = __builtin_fma(a, a, s);
            s = __builtin_fma(b, b, s);
        } else {
            const double a = __uint_as_float(v[i]);
            s = __builtin_fma(a, a, s);
        }
    }
    return s;
}

template <bool kBf16>
__device__ __forceinline__ double run_sum(const GradRun &r)
{
    constexpr int kSize = kBf16 ? 2 : 4, kPer = 16 / kSize;
    gsrc src = (gsrc)r.src;
    const int64_t vecs = r.count / kPer;
    double s = 0.0;
    int64_t i = threadIdx.x;
    for (; i + (kUnroll - 1) * kGradBlock < vecs; i += kUnroll * kGradBlock) {
        u32x4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            v[u] = load16(src + (i + u * kGradBlock) * 16);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            s += square_sum<kBf16>(v[u]);
    }
    for (; i < vecs; i += kGradBlock)
        s += square_sum<kBf16>(load16(src + i * 16));
    for (int64_t e = vecs * kPer + threadIdx.x; e < r.count; e += kGradBlock) {
        const double a = load1(src + e * kSize, kBf16);
        s = __builtin_fma(a, a, s);
    }
    return s;
}

__global__ __launch_bounds__(kGradBlock) void grad_sum_kernel(const GradRun *runs, int64_t n,
                                                              double *sums)
{
    __shared__ double tmp[kGradWaves];
    double s = 0.0;
    for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
        const GradRun r = runs[i];
        s += r.type == MOONEP_BF16 ? run_sum<true>(r) : run_sum<false>(r);
    }
    s = block_sum(s, tmp);
    if (threadIdx.x == 0)
        sums[blockIdx.x] = s;
}

// The sum of the workgroups' sums, in an order that their number fixes.
__device__ __forceinline__ double join_sums(const double *sums, int n, double *tmp)
{
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kGradBlock)
        s += sums[i];
    return block_sum(s, tmp);
}

__global__ __launch_bounds__(kGradBlock) void grad_norm_kernel(const double *sums, int n,
                                                               double *sumsq, float *norm)
{
    __shared__ double tmp[kGradWaves];
    const double s = join_sums(sums, n, tmp);
    if (threadIdx.x == 0) {
        *norm = (float)__builtin_sqrt(s);
        if (sumsq)
            *sumsq = s;
    }
}

// A product of bf16 by f has up to 32 bits.  Rounded to fp32 and then to bf16 it is off
// where the first rounding makes a tie for the second: that takes 2^-16 of all pairs, so that
// one factor in 500 does it for one of bf16's 128 significands.  Those, and what is a tie
// by itself, are rounded again from the exact product, which fp64 holds (291 tensors of 63
// to 2097152, the scaling alone: 45.8 us without the question, 46.0 with it, and with such a
// factor 46.6 and 49.6).
__device__ __forceinline__ bool bf16_tie(float p) { return (uint16_t)__float_as_uint(p) == 0x8000; }
__device__ __forceinline__ uint32_t scaled_exactly(float g, float f)
{
    return bf16_of_double((double)g * (double)f);
}

template <bool kBf16>
__device__ __forceinline__ u32x4 scaled(u32x4 v, float f)
{
    u32x4 o;
    bool tie = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kBf16) {
            const float a = bf16_lo(v[i]) * f, b = bf16_hi(v[i]) * f;
            o[i] = pack_bf16(a, b);
            tie |= bf16_tie(a);
            tie |= bf16_tie(b);
        } else {
            o[i] = __float_as_uint(__uint_as_float(v[i]) * f);
        }
    }
    if (kBf16 && tie) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = scaled_exactly(bf16_lo(v[i]), f) | scaled_exactly(bf16_hi(v[i]), f) << 16;
    }
    return o;
}

template <bool kBf16>
__device__ __forceinline__ void run_scale(const GradRun &r, float f)
{
    constexpr int kSize = kBf16 ? 2 : 4, kPer = 16 / kSize;
    gsrc src = (gsrc)r.src;
    gdst dst = (gdst)r.dst;
    const int64_t vecs = r.count / kPer;
    int64_t i = threadIdx.x;
    for (; i + (kUnroll - 1) * kGradBlock < vecs; i += kUnroll * kGradBlock) {
        u32x4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            v[u] = load16_nt(src + (i + u * kGradBlock) * 16);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            store16_nt(dst + (i + u * kGradBlock) * 16, scaled<kBf16>(v[u], f));
    }
    for (; i < vecs; i += kGradBlock)
        store16_nt(dst + i * 16, scaled<kBf16>(load16_nt(src + i * 16), f));
    for (int64_t e = vecs * kPer + threadIdx.x; e < r.count; e += kGradBlock) {
        const float g = load1(src + e * kSize, kBf16);
        if (kBf16)
            *(MOONEP_GLOBAL uint16_t *)(dst + e * kSize) = (uint16_t)scaled_exactly(g, f);
        else
            *(MOONEP_GLOBAL float *)(dst + e * kSize) = g * f;
    }
}

__global__ __launch_bounds__(kGradBlock) void grad_scale_kernel(const GradRun *runs, int64_t n,
                                                                double max_norm, const double *sums,
                                                                int nsums, float *norm)
{
    __shared__ double tmp[kGradWaves];
    const double total = __builtin_sqrt(join_sums(sums, nsums, tmp));
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *norm = (float)total;
    const bool clip = total > max_norm && total < __builtin_inf();
    const float f = clip ? (float)(max_norm / total) : 1.0f;
    for (int64_t i = n - 1 - blockIdx.x; i >= 0; i -= gridDim.x) {
        const GradRun r = runs[i];
        if (!clip && r.src == r.dst)
            continue;
        if (r.type == MOONEP_BF16)
            run_scale<true>(r, f);
        else
            run_scale<false>(r, f);
    }
}

int grad_grid(int64_t n) { return (int)(n < 1 ? 1 : (n < kGradGrid ? n : kGradGrid)); }

}  // namespace

size_t grad_workspace() { return kGradGrid * sizeof(double); }

int launch_grad_norm(const void *table, int64_t n, double *sumsq, float *norm, void *ws,
                     hipStream_t st)
{
    const int grid = grad_grid(n);
    hipLaunchKernelGGL(grad_sum_kernel, dim3(grid), dim3(kGradBlock), 0, st, (const GradRun *)table,
                       n, (double *)ws);
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kGradBlock), 0, st, (const double *)ws, grid,
                       sumsq, norm);
    return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_ERR_HIP;
}

int launch_grad_clip(const void *table, int64_t n, double max_norm, const double *sumsq, float *norm,
                     void *ws, hipStream_t st)
{
    const int grid = grad_grid(n);
    if (!sumsq)
        hipLaunchKernelGGL(grad_sum_kernel, dim3(grid), dim3(kGradBlock), 0, st,
                           (const GradRun *)table, n, (double *)ws);
    hipLaunchKernelGGL(grad_scale_kernel, dim3(grid), dim3(kGradBlock), 0, st, (const GradRun *)table,
                       n, max_norm, sumsq ? sumsq : (const double *)ws, sumsq ? 1 : grid, norm);
    return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_ERR_HIP;
}

}  // namespace moonep
