// router.hip -- scores, the K experts and gates of every token, the balance
// loss, and the gradient of gates and loss with respect to the logits.
//
// A token's E logits are held by the 16 lanes of one DPP row (four tokens per
// wave), kV per lane: chunk i of 64 experts gives lane c the experts
// 64 i + 4 c .. + 3, so that rows of E % 4 == 0 are read as whole vectors.  Sums
// and maxima over a token are four DPP steps for four tokens at once.
//
// Choosing: K rounds of the row's largest key below the last one.  A key is one
// word, the leading bits of the logit in integer order above the expert id
// (counted down, so that ties go to the lower id): unique, so a round is one
// addition and half a three-way minimum per element.  bf16 logits fit whole; where
// two of the K + 1 largest fp32 logits share their leading bits, or the row holds
// a NaN, that row is chosen again on whole keys, over all 64 lanes of its wave.
//
// The shares of a workgroup's tokens are summed in registers (each lane keeps
// its experts), then over its rows and waves, into one partial row of E sums
// per workgroup; a second kernel joins the partials in fp64 in a fixed order, and
// a third the loss.  Counts are integer atomics in LDS.
//
// Measured: 131072 x 256 fp32, sigmoid, K = 8, with the loss: 57 us, of which the
// first kernel 47, the joins 5 each; its vector instructions (some 700 for four
// tokens, the exponentials and reciprocals at a quarter of the rate) alone take
// about 43 us, its bytes 24; bf16 46 us, its bytes 13.  131072 x 128 bf16, softmax,
// backward: 21 us, its bytes 13 (normalised sigmoid 24: its slope has an exponential
// of its own); 64 tokens of 64 experts: 3.4 us, a launch.  Sixteen lanes a token are a
// balance: fewer would not hold 1024 experts in registers, more would spend the
// reductions' steps on fewer tokens.
#include "quant.hpp"

namespace moonep {

namespace {

constexpr int kRowLanes = 16, kRowsPerWave = 64 / kRowLanes;
constexpr int kRowsPerBlock = kWaves * kRowsPerWave;
constexpr int32_t kNoKey = INT32_MIN, kNanKey = INT32_MIN + 1;  // nothing; a NaN, below -inf

// Workgroups of the backward: about what is on the chip at once (2048 of kV = 4, 1024
// to 1792 of kV = 8 and 16, fewer above).  131072 tokens, us at 1024 / 2048, bf16 and
// fp32: E = 32 16.7 / 15.0 and 16.7 / 15.1, 64 16.2 / 15.2 and 16.0 / 15.7, 96 21.3 /
// 21.9 and 27.4 / 30.7, 128 21.0 / 22.2 and 33.5 / 37.5, 256 37.1 / 43.2 and 63.3 /
// 62.9, 512 78.3 / 92.0 and 122 / 124; 65536 of 1024 133 / 170 and 147 / 204.
int64_t bwd_blocks(int32_t E) { return E <= 64 ? 2048 : 1024; }

// Workgroups of the loss's first pass: enough to fill the chip, few enough that
// their partial rows stay small beside the logits; and no more tokens for one than
// that each lane adds 128 shares in fp32 (shares that are all alike, so that every
// addition rounds the same way, then are 2e-6 off at most; without the limit 2^24
// tokens of 3 experts were 1.5e-5 off).
constexpr int64_t kLossBlocks = 1024, kLossTokens = 2048;
constexpr int kJoinThreads = 1024, kJoinExperts = 64, kJoinRows = kJoinThreads / kJoinExperts;

// Workgroups of one group of n tokens, and the tokens of each: about `blocks` in
// all, two rounds of rows each at least.
struct Split {
    int64_t per_group, tokens;
};

Split split_tokens(int64_t n, int64_t groups, int64_t blocks)
{
    int64_t per = blocks / groups;
    const int64_t most = (n + 2 * kRowsPerBlock - 1) / (2 * kRowsPerBlock);
    per = per < most ? per : most;
    per = per < 1 ? 1 : per;
    Split s;
    s.tokens = (n + per - 1) / per;
    s.per_group = s.tokens ? (n + s.tokens - 1) / s.tokens : 1;
    return s;
}

struct RouterLayout {
    Split split;
    size_t count_off, loss_off, bytes;  // the shares' partial rows come first
};

RouterLayout router_layout(const moonep_shape &s, int32_t groups)
{
    RouterLayout l{};
    const int64_t n = (int64_t)s.R * s.S / groups, least = groups * ((n + kLossTokens - 1) / kLossTokens);
    l.split = split_tokens(n, groups, least < kLossBlocks ? kLossBlocks : least);
    const size_t rows = (size_t)l.split.per_group * groups * s.E * 4;
    const size_t nchunk = (size_t)(s.E + kJoinExperts - 1) / kJoinExperts;
    l.count_off = rows;
    l.loss_off = (2 * rows + 15) & ~(size_t)15;
    l.bytes = l.loss_off + nchunk * groups * 8;
    return l;
}

// 2^(x log2 e) with the product rounded once: (1.25 |x| + 2) 2^-24 relative (the
// constant's rounding is the quarter), 1.6e-6 at |x| = 20; for fp32 logits under
// softmax the rounding of their difference costs |x| 2^-24 as well, for sigmoid and
// bf16 logits there is nothing else.  The choice does not go through it.  With the
// product's dropped part taken along, as four more operations an element, 131072 x 256
// forward takes 63.8 us instead of 59.8 and the backward of x 128 bf16 24.0 instead of
// 22.1, so it is left out.  0 and infinity at the ends; results below 2^-126 are 0.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// v_rcp is good to one unit in the last place; 0 below 2^-126 (logits under -87.3).
__device__ __forceinline__ float sigmoid_of(float l) { return __builtin_amdgcn_rcpf(1.0f + exp_of(-l)); }

__device__ __forceinline__ int32_t key_of(float l)
{
    const int32_t b = __float_as_int(l + 0.0f);  // -0 -> +0
    return l != l ? kNanKey : b ^ ((b >> 31) & 0x7FFFFFFF);
}

// One word per element for the rounds: leading bits of the logit in unsigned
// order, then the id counted down in kIdBits.  The lane's part of the id, 4 c, is
// left to be subtracted, so that element i's part is a constant.  Elements past E
// hold -inf and the highest ids, so every expert comes before them.
template <int kIdBits>
__device__ __forceinline__ uint32_t packed_key(float l, int i)
{
    constexpr uint32_t kIds = (1u << kIdBits) - 1u;
    const uint32_t b = __float_as_uint(l + 0.0f);  // -0 -> +0
    const uint32_t u = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return (u & ~kIds) | (kIds - (uint32_t)((i >> 2) * 64 + (i & 3)));
}

// Expert of element i in the row's lane c.
__device__ __forceinline__ int32_t expert_of(int i, int c) { return (i >> 2) * 64 + c * 4 + (i & 3); }

// Four tokens' logits in fp32, one per row of lanes, from `rows` (uniform) on; a
// row past the last reads the first.  Experts past E are -inf (score 0): their
// lanes read the row's last experts and drop them, so that no branch splits the
// loads.
template <int kV, bool kBf16>
__device__ __forceinline__ void load_rows(const char *rows, int32_t row, int32_t E, int c, bool vec,
                                          float (&l)[kV])
{
    constexpr int kSize = kBf16 ? 2 : 4;
    constexpr float kNone = -__builtin_huge_valf();
    // Offsets and bounds are cheaper to compute again than to keep across the
    // rows: as loop invariants they take a register or a mask each.
    asm volatile("" : "+v"(c));
    if (vec) {
#pragma unroll
        for (int i = 0; i < kV; i += 4) {
            const int32_t e = expert_of(i, c), from = e < E ? e : E - 4;
            const char *p = rows + (uint32_t)((row * E + from) * kSize);
            if (kBf16) {
                const u32x2 w = *(const u32x2 *)p;
                l[i] = bf16_lo(w[0]);
                l[i + 1] = bf16_hi(w[0]);
                l[i + 2] = bf16_lo(w[1]);
                l[i + 3] = bf16_hi(w[1]);
            } else {
                const f32x4 w = *(const f32x4 *)p;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    l[i + j] = w[j];
            }
        }
        if (E == kV * kRowLanes)
            return;
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int32_t e = expert_of(i, c), from = e < E ? e : E - 1;
            const char *p = rows + (uint32_t)((row * E + from) * kSize);
            l[i] = kBf16 ? bf16_lo(*(const uint16_t *)p) : *(const float *)p;
        }
    }
#pragma unroll
    for (int i = 0; i < kV; ++i)
        l[i] = expert_of(i, c) < E ? l[i] : kNone;
}

// Scores of the row in place of the logits, and 1 / Z (0 for a row with no
// expert: every score is 0 there).  top: the largest logit (softmax only).
template <int kV>
__device__ __forceinline__ float scores(float (&l)[kV], int32_t score, float top)
{
    float z = 0.0f;
    if (score == MOONEP_SCORE_SOFTMAX) {
        // all masked: subtract 0, every exponential is 0
        const float base = top == -__builtin_huge_valf() ? 0.0f : top;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            l[i] = exp_of(l[i] - base);
            z += l[i];
        }
        z = row16_sum(z);
        return z == 0.0f ? 0.0f : 1.0f / z;
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        l[i] = sigmoid_of(l[i]);
        z += l[i];
    }
    return 1.0f / (row16_sum(z) + 1e-20f);
}

template <int kV>
__device__ __forceinline__ float row_top(const float (&l)[kV])
{
    // fmaxf drops a NaN; it comes back through its own exponential
    float m = l[0];
#pragma unroll
    for (int i = 1; i < kV; ++i)
        m = fmaxf(m, l[i]);
    m = fmaxf(m, __uint_as_float(dpp<kDppRowRor8>(__float_as_uint(m))));
    m = fmaxf(m, __uint_as_float(dpp<kDppRowRor4>(__float_as_uint(m))));
    m = fmaxf(m, __uint_as_float(dpp<kDppRowRor2>(__float_as_uint(m))));
    return fmaxf(m, __uint_as_float(dpp<kDppRowRor1>(__float_as_uint(m))));
}

__device__ __forceinline__ int32_t row16_imax(int32_t v)
{
    v = max(v, (int32_t)dpp<kDppRowRor8>((uint32_t)v));
    v = max(v, (int32_t)dpp<kDppRowRor4>((uint32_t)v));
    v = max(v, (int32_t)dpp<kDppRowRor2>((uint32_t)v));
    return max(v, (int32_t)dpp<kDppRowRor1>((uint32_t)v));
}

struct RouterArgs {
    const void *logits;
    int32_t *topk_idx;
    float *gates;
    float *prob_part;      // [blocks, E]
    int32_t *count_part;   // [blocks, E]
    int64_t N, n, per_group, tokens;
    int32_t E, K, score, normalize, vec;
    float scale;
};

}  // namespace

// Workgroup b takes `tokens` consecutive tokens of group b / per_group.
// Four waves per SIMD up to 256 experts: without the bound 16 experts a lane take
// more registers than that, and the loads of fewer waves are waited for.
template <int kV, bool kBf16, bool kLoss>
__global__ __launch_bounds__(kBlock, (kV <= 16 ? 4 : 1)) void router_kernel(RouterArgs a)
{
    extern __shared__ __align__(16) uint32_t lds[];
    int32_t *hist = (int32_t *)lds;        // [E]
    float *sums = (float *)(lds + a.E);    // [kWaves][E]
    const int lane = lane_id(), wave = (int)threadIdx.x >> 6;
    const int c = lane % kRowLanes, r = lane / kRowLanes;
    const int64_t g = (int64_t)blockIdx.x / a.per_group;
    const int64_t first = g * a.n + ((int64_t)blockIdx.x - g * a.per_group) * a.tokens;
    const int64_t end = first + a.tokens < (g + 1) * a.n ? first + a.tokens : (g + 1) * a.n;
    constexpr int kIdBits = kV == 4 ? 6 : kV == 8 ? 7 : kV == 16 ? 8 : kV == 32 ? 9 : 10;
    // Expert e of round k0 + c in lane c: its id, its score for the gates.  (Keys of
    // a row with a NaN may have run out, before it is chosen again.)
    auto put = [&](int64_t tok, bool on, int32_t k0, int32_t kn, int c, int32_t e, float base, float *mine,
                   float *wsum) {
        const bool in = on && c < kn;
        e = e < a.E ? e : a.E - 1;
        float v = 0.0f;
        if (in)
            v = kBf16 ? bf16_lo(((const uint16_t *)a.logits)[tok * a.E + e])
                      : ((const float *)a.logits)[tok * a.E + e];
        *mine = !in ? 0.0f : a.score == MOONEP_SCORE_SOFTMAX ? exp_of(v - base) : sigmoid_of(v);
        *wsum += *mine;
        if (in) {
            a.topk_idx[tok * a.K + k0 + c] = e;
            if (a.K > kRowLanes)
                a.gates[tok * a.K + k0 + c] = *mine;
        }
        return e;
    };
    float acc[kV];
    if (kLoss) {
        for (int32_t e = (int32_t)threadIdx.x; e < a.E; e += kBlock)
            hist[e] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kV; ++i)
            acc[i] = 0.0f;
    }
    const char *logits = (const char *)a.logits;
    constexpr int kSize = kBf16 ? 2 : 4;
    float nxt[kV];  // the next tokens' logits, on their way
    int64_t t0 = first + wave * kRowsPerWave;
    if (t0 < end)
        load_rows<kV, kBf16>(logits + t0 * a.E * kSize, t0 + r < end ? r : 0, a.E, c, a.vec != 0, nxt);
    for (; t0 < end; t0 += kRowsPerBlock) {
        const int64_t tok = t0 + r;
        const bool on = tok < end;
        float l[kV];
        uint32_t key[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            l[i] = nxt[i];
            key[i] = packed_key<kIdBits>(l[i], i);
        }
        const int64_t t2 = t0 + kRowsPerBlock < end ? t0 + kRowsPerBlock : t0;
        load_rows<kV, kBf16>(logits + t2 * a.E * kSize, t2 + r < end ? r : 0, a.E, c, a.vec != 0, nxt);
        const float top = a.score == MOONEP_SCORE_SOFTMAX ? row_top(l) : 0.0f;
        const float rz = scores(l, a.score, top);
        if (kLoss) {
#pragma unroll
            for (int i = 0; i < kV; ++i)
                acc[i] = __builtin_fmaf(l[i], on ? rz : 0.0f, acc[i]);
        }
        // K rounds; lane k % 16 keeps round k's expert and score, and a chunk of
        // 16 rounds is written at once
        const float base = top == -__builtin_huge_valf() ? 0.0f : top;
        float wsum = 0.0f, mine = 0.0f;
        bool again = rz != rz;  // a NaN in the row
        int32_t chosen = 0;     // the last chunk's expert of this lane
        auto next_key = [&](uint32_t last) {
            // last - 1 - (key - 4 c) wraps above last for the keys chosen already,
            // and is least for the largest of the others
            const uint32_t mine_last = last + (uint32_t)c * 4;
            uint32_t d = 0xFFFFFFFFu;
#pragma unroll
            for (int i = 0; i < kV; ++i)
                d = min(d, mine_last + ~key[i]);
            return last - 1u - row16_min(d);
        };
        uint32_t least = 0xFFFFFFFFu;  // difference of two keys in turn, bit by bit
        uint32_t m = 0xFFFFFF00u;  // the last round's key: those at it and above are chosen
        for (int32_t k0 = 0; k0 < a.K; k0 += kRowLanes) {
            const int32_t kn = a.K - k0 < kRowLanes ? a.K - k0 : kRowLanes;
            uint32_t my_key = 0;
            for (int32_t k = 0; k < kn; ++k) {
                const uint32_t was = m;
                m = next_key(was);
                if (!kBf16 && k0 + k)
                    least = min(least, m ^ was);
                my_key = c == k ? m : my_key;
            }
            if (!kBf16 && k0 + kn == a.K && a.K < a.E)
                least = min(least, next_key(m) ^ m);
            chosen = put(tok, on, k0, kn, c,
                         (int32_t)((1u << kIdBits) - 1u - (my_key & ((1u << kIdBits) - 1u))), base,
                         &mine, &wsum);
        }
        again |= least >> kIdBits == 0;
        // Whole keys, for one token at a time over all lanes (rare: so that it takes
        // few registers from the other rows): the largest, and the least id that
        // has it.
        const uint64_t tied = ballot(again && on);
        for (int q = 0; q < kRowsPerWave && tied; ++q) {
            if (!((tied >> (q * kRowLanes)) & 1))
                continue;
            const char *row = logits + (t0 + q) * a.E * kSize;
            int32_t whole[kV / 4];
#pragma unroll
            for (int i = 0; i < kV / 4; ++i) {
                const int32_t e = i * 64 + lane, from = e < a.E ? e : 0;
                const int32_t w = key_of(kBf16 ? bf16_lo(((const uint16_t *)row)[from])
                                               : ((const float *)row)[from]);
                whole[i] = e < a.E ? w : kNoKey;
            }
            wsum = r == q ? 0.0f : wsum;
            for (int32_t k0 = 0; k0 < a.K; k0 += kRowLanes) {
                const int32_t kn = a.K - k0 < kRowLanes ? a.K - k0 : kRowLanes;
                int32_t my_e = 0;
                for (int32_t k = 0; k < kn; ++k) {
                    int32_t w = whole[0];
#pragma unroll
                    for (int i = 1; i < kV / 4; ++i)
                        w = max(w, whole[i]);
                    w = row16_imax(w);
                    w = max(w, __shfl_xor(w, 16, 64));
                    w = max(w, __shfl_xor(w, 32, 64));
                    uint32_t e = 0xFFFFu;
#pragma unroll
                    for (int i = kV / 4 - 1; i >= 0; --i)
                        e = whole[i] == w ? (uint32_t)(i * 64 + lane) : e;
                    e = row16_min(e);
                    e = min(e, (uint32_t)__shfl_xor((int)e, 16, 64));
                    e = min(e, (uint32_t)__shfl_xor((int)e, 32, 64));
#pragma unroll
                    for (int i = 0; i < kV / 4; ++i)
                        whole[i] = e == (uint32_t)(i * 64 + lane) ? kNoKey : whole[i];
                    my_e = c == k ? (int32_t)e : my_e;
                }
                if (r == q)
                    chosen = put(tok, on, k0, kn, c, my_e, base, &mine, &wsum);
            }
        }
        if (kLoss && on) {
            if (a.K > kRowLanes)
                for (int32_t k = c; k < a.K; k += kRowLanes)
                    atomicAdd(hist + a.topk_idx[tok * a.K + k], 1);
            else if (c < a.K)
                atomicAdd(hist + chosen, 1);
        }
        float f = a.scale;
        if (a.normalize) {
            const float w = row16_sum(wsum) + (a.score == MOONEP_SCORE_SIGMOID ? 1e-20f : 0.0f);
            f = w == 0.0f ? 0.0f : a.scale / w;
        } else if (a.score == MOONEP_SCORE_SOFTMAX) {
            f = a.scale * rz;
        }
        if (a.K <= kRowLanes) {
            if (on && c < a.K)
                a.gates[tok * a.K + c] = mine * f;
        } else if (on) {
            // each lane scales what it wrote itself
            for (int32_t k = c; k < a.K; k += kRowLanes)
                a.gates[tok * a.K + k] *= f;
        }
    }
    if (kLoss) {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            acc[i] += __shfl_xor(acc[i], 16, 64);
            acc[i] += __shfl_xor(acc[i], 32, 64);
            if (r == 0 && expert_of(i, c) < a.E)
                sums[wave * a.E + expert_of(i, c)] = acc[i];
        }
        __syncthreads();
        for (int32_t e = (int32_t)threadIdx.x; e < a.E; e += kBlock) {
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < kWaves; ++q)
                s += sums[q * a.E + e];
            a.prob_part[(int64_t)blockIdx.x * a.E + e] = s;
            a.count_part[(int64_t)blockIdx.x * a.E + e] = hist[e];
        }
    }
}

// Joins the partial rows of one group and 64 experts: 16 rows at a time, then
// over the 16 in LDS.
__global__ __launch_bounds__(kJoinThreads) void router_join_kernel(
    const float *__restrict__ prob_part, const int32_t *__restrict__ count_part, int64_t per_group,
    int32_t E, int32_t nchunk, int32_t *__restrict__ counts, float *__restrict__ prob_sum,
    double *__restrict__ losses)
{
    __shared__ double prob[kJoinThreads];
    __shared__ int32_t cnt[kJoinThreads];
    const int t = (int)threadIdx.x;
    const int64_t g = (int64_t)blockIdx.x / nchunk;
    const int32_t e = (int32_t)((int64_t)blockIdx.x - g * nchunk) * kJoinExperts + t % kJoinExperts;
    double p = 0.0;
    int32_t n = 0;
    if (e < E) {
#pragma unroll 8
        for (int64_t b = t / kJoinExperts; b < per_group; b += kJoinRows) {
            const int64_t at = (g * per_group + b) * E + e;
            p += (double)prob_part[at];
            n += count_part[at];
        }
    }
    prob[t] = p;
    cnt[t] = n;
    __syncthreads();
    if (t < kJoinExperts) {
#pragma unroll
        for (int q = 1; q < kJoinRows; ++q) {
            p += prob[t + q * kJoinExperts];
            n += cnt[t + q * kJoinExperts];
        }
        if (e < E) {
            counts[g * E + e] = n;
            prob_sum[g * E + e] = (float)p;
        }
        double s = e < E ? (double)n * p : 0.0;
#pragma unroll
        for (int d = 32; d > 0; d >>= 1)
            s += __shfl_xor(s, d, 64);
        if (t == 0)
            losses[blockIdx.x] = s;
    }
}

// The loss: the (group, chunk) sums, in an order of their number alone.
__global__ __launch_bounds__(kJoinThreads) void router_loss_kernel(const double *__restrict__ losses,
                                                                   int64_t total, double factor,
                                                                   float *__restrict__ loss)
{
    __shared__ double part[kJoinThreads / 64];
    const int t = (int)threadIdx.x;
    double s = 0.0;
    for (int64_t i = t; i < total; i += kJoinThreads)
        s += losses[i];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        s += __shfl_xor(s, d, 64);
    if (t % 64 == 0)
        part[t / 64] = s;
    __syncthreads();
    if (t == 0) {
        s = 0.0;
        for (int q = 0; q < kJoinThreads / 64; ++q)
            s += part[q];
        loss[0] = (float)(s * factor);
    }
}

namespace {

struct RouterBwdArgs {
    const void *logits;
    const int32_t *topk_idx, *counts;
    const float *d_gates, *d_loss;
    void *d_logits;
    int64_t n, per_group, tokens;
    int32_t E, K, score, normalize, vec;
    int32_t mean;  // of a group's counts, to the nearest integer
    float scale, factor;
};

}  // namespace

// Four tokens per wave.  What passes between a token's K entries (a lane each)
// and its E experts goes through LDS, E floats for each row of lanes: the
// scores, read at the chosen experts, and the gates' gradients, added up there.
template <int kV, bool kBf16>
__global__ __launch_bounds__(kBlock) void router_bwd_kernel(RouterBwdArgs a)
{
    extern __shared__ __align__(16) uint32_t lds[];
    const int lane = lane_id(), wave = (int)threadIdx.x >> 6;
    const int c = lane % kRowLanes, r = lane / kRowLanes;
    float *own = (float *)lds + (wave * kRowsPerWave + r) * (kV * kRowLanes);
    const float tiny = a.score == MOONEP_SCORE_SIGMOID ? 1e-20f : 0.0f;
    const int64_t g = (int64_t)blockIdx.x / a.per_group;
    const int64_t first = g * a.n + ((int64_t)blockIdx.x - g * a.per_group) * a.tokens;
    const int64_t end = first + a.tokens < (g + 1) * a.n ? first + a.tokens : (g + 1) * a.n;
    // The loss's gradient at p_e, less that of a mean count: a_e - sum_j a_j p_j takes no
    // constant into account but for a tiny / Z of it (as sum_j p_j = 1 - tiny / Z), and
    // counts near their mean, where the loss drives them, would cancel to rounding.
    float la[kV], la_tiny = 0.0f;
    if (a.counts) {
        const float dl = a.d_loss[0] * a.factor;
        la_tiny = dl * (float)a.mean * tiny;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int32_t e = expert_of(i, c);
            la[i] = e < a.E ? dl * (float)(a.counts[g * a.E + e] - a.mean) : 0.0f;
        }
    }
    const char *logits = (const char *)a.logits;
    constexpr int kSize = kBf16 ? 2 : 4;
    float nxt[kV];  // the next tokens' logits, on their way
    int64_t t0 = first + wave * kRowsPerWave;
    if (t0 < end)
        load_rows<kV, kBf16>(logits + t0 * a.E * kSize, t0 + r < end ? r : 0, a.E, c, a.vec != 0, nxt);
    for (; t0 < end; t0 += kRowsPerBlock) {
        const int64_t tok = t0 + r;
        const bool on = tok < end;
        // the first 16 entries of the token, one a lane; others are read again
        uint32_t e0 = 0xFFFFFFFFu;
        float d0 = 0.0f;
        if (a.d_gates && on && c < a.K) {
            e0 = (uint32_t)a.topk_idx[tok * a.K + c];
            d0 = a.d_gates[tok * a.K + c];
        }
        float l[kV], s[kV], part[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i)
            l[i] = nxt[i];
        const int64_t t2 = t0 + kRowsPerBlock < end ? t0 + kRowsPerBlock : t0;
        load_rows<kV, kBf16>(logits + t2 * a.E * kSize, t2 + r < end ? r : 0, a.E, c, a.vec != 0, nxt);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            s[i] = l[i];
            part[i] = 0.0f;
        }
        const float rz = scores(s, a.score, a.score == MOONEP_SCORE_SOFTMAX ? row_top(l) : 0.0f);
        float all = 0.0f;  // what every expert's ds loses to the gates
        if (a.d_gates) {
#pragma unroll
            for (int i = 0; i < kV; i += 4)
                *(f32x4 *)(own + expert_of(i, c)) = f32x4{s[i], s[i + 1], s[i + 2], s[i + 3]};
            wave_sync();
            // dg_k - sum_j dg_j s_j / W (normalised) takes no constant into account but
            // for a tiny / W of it.  The first entry's comes off, that of the largest
            // score: with one expert chosen nothing is left, and where one dominates
            // its own term is the others' small ones, not what is left of two equal ones.
            const float d_first = a.normalize ? row16_first(e0 < (uint32_t)a.E ? d0 : 0.0f) : 0.0f;
            float w = 0.0f, gs = 0.0f;
            auto chosen = [&](uint32_t e, float d) {
                if (e < (uint32_t)a.E) {
                    w += own[e];
                    gs = __builtin_fmaf(d - d_first, own[e], gs);
                }
            };
            chosen(e0, d0);
            if (a.K > kRowLanes && on)
                for (int32_t k = c + kRowLanes; k < a.K; k += kRowLanes)
                    chosen((uint32_t)a.topk_idx[tok * a.K + k], a.d_gates[tok * a.K + k]);
            w = row16_sum(w) + tiny;
            gs = row16_sum(gs);
            float mul = a.scale, sub = 0.0f;
            if (a.normalize) {
                const float rw = w == 0.0f ? 0.0f : 1.0f / w;
                mul = a.scale * rw;
                sub = (gs - d_first * tiny) * rw;
            } else if (a.score == MOONEP_SCORE_SOFTMAX) {
                mul = a.scale * rz;
                all = mul * gs * rz;
            }
            wave_sync();
#pragma unroll
            for (int i = 0; i < kV; i += 4)
                *(f32x4 *)(own + expert_of(i, c)) = f32x4{0, 0, 0, 0};
            wave_sync();
            auto spread = [&](uint32_t e, float d) {
                if (e < (uint32_t)a.E)
                    atomicAdd(own + e, mul * (d - d_first - sub));
            };
            spread(e0, d0);
            if (a.K > kRowLanes && on)
                for (int32_t k = c + kRowLanes; k < a.K; k += kRowLanes)
                    spread((uint32_t)a.topk_idx[tok * a.K + k], a.d_gates[tok * a.K + k]);
            wave_sync();
#pragma unroll
            for (int i = 0; i < kV; i += 4) {
                const f32x4 v = *(const f32x4 *)(own + expert_of(i, c));
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    part[i + j] = v[j];
            }
            wave_sync();
        }
        if (a.counts) {
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < kV; ++i)
                dot = __builtin_fmaf(la[i], s[i], dot);
            dot = (row16_sum(dot) - la_tiny) * rz;
#pragma unroll
            for (int i = 0; i < kV; ++i)
                part[i] += (la[i] - dot) * rz;
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            float slope = s[i];
            if (a.score == MOONEP_SCORE_SIGMOID) {
                // s (1 - s) without the difference, which loses the digits of s near 1
                const float d = exp_of(-__builtin_fabsf(l[i])), q = __builtin_amdgcn_rcpf(1.0f + d);
                slope = d * q * q;
            }
            s[i] = (part[i] - all) * slope;
        }
        if (!on)
            continue;
#pragma unroll
        for (int i = 0; i < kV; i += 4) {
            const int32_t e = expert_of(i, c);
            const int64_t at = tok * a.E + e;
            if (a.vec && e < a.E) {
                if (kBf16)
                    *(u32x2 *)((uint16_t *)a.d_logits + at) =
                        u32x2{pack_bf16(s[i], s[i + 1]), pack_bf16(s[i + 2], s[i + 3])};
                else
                    *(f32x4 *)((float *)a.d_logits + at) = f32x4{s[i], s[i + 1], s[i + 2], s[i + 3]};
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (e + j < a.E) {
                        if (kBf16)
                            ((uint16_t *)a.d_logits)[at + j] = (uint16_t)(pack_bf16(s[i + j], 0.0f) & 0xFFFFu);
                        else
                            ((float *)a.d_logits)[at + j] = s[i + j];
                    }
            }
        }
    }
}

namespace {

int last() { return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_ERR_HIP; }

// Rows can be read as vectors of four: every row starts on one.
bool row_vectors(const void *a, const void *b, int32_t E, bool bf16)
{
    const uintptr_t m = bf16 ? 7 : 15;
    return E % 4 == 0 && (((uintptr_t)a | (uintptr_t)b) & m) == 0;
}

// f<kV>() for the fewest experts per lane that hold E.
template <template <int> class F, class... Args>
int by_experts(int32_t E, Args... args)
{
    if (E <= 64)
        return F<4>::run(args...);
    if (E <= 128)
        return F<8>::run(args...);
    if (E <= 256)
        return F<16>::run(args...);
    if (E <= 512)
        return F<32>::run(args...);
    return F<64>::run(args...);
}

template <int kV>
struct RunRouter {
    static int run(const RouterArgs &a, bool bf16, bool with_loss, int64_t blocks, hipStream_t st)
    {
        const size_t lds = with_loss ? (size_t)(1 + kWaves) * a.E * 4 : 0;
        const dim3 grid((uint32_t)blocks), block(kBlock);
        if (bf16 && with_loss)
            hipLaunchKernelGGL((router_kernel<kV, true, true>), grid, block, lds, st, a);
        else if (bf16)
            hipLaunchKernelGGL((router_kernel<kV, true, false>), grid, block, lds, st, a);
        else if (with_loss)
            hipLaunchKernelGGL((router_kernel<kV, false, true>), grid, block, lds, st, a);
        else
            hipLaunchKernelGGL((router_kernel<kV, false, false>), grid, block, lds, st, a);
        return last();
    }
};

template <int kV>
struct RunRouterBwd {
    static int run(const RouterBwdArgs &a, bool bf16, int64_t blocks, hipStream_t st)
    {
        const size_t lds = a.d_gates ? (size_t)kRowsPerBlock * kV * kRowLanes * 4 : 0;
        const dim3 grid((uint32_t)blocks), block(kBlock);
        if (bf16)
            hipLaunchKernelGGL((router_bwd_kernel<kV, true>), grid, block, lds, st, a);
        else
            hipLaunchKernelGGL((router_bwd_kernel<kV, false>), grid, block, lds, st, a);
        return last();
    }
};

}  // namespace

size_t router_workspace(const moonep_shape &s, int32_t groups) { return router_layout(s, groups).bytes; }

int launch_router(const moonep_shape &s, const moonep_router_opts &o, const void *logits,
                  int32_t *topk_idx, float *gates, int32_t *counts, float *prob_sum, float *loss,
                  void *ws, hipStream_t st)
{
    const RouterLayout lay = router_layout(s, o.groups);
    const bool with_loss = loss != nullptr, bf16 = o.logits_type == MOONEP_BF16;
    char *base = (char *)ws;
    RouterArgs a;
    a.logits = logits;
    a.topk_idx = topk_idx;
    a.gates = gates;
    a.prob_part = with_loss ? (float *)base : nullptr;
    a.count_part = with_loss ? (int32_t *)(base + lay.count_off) : nullptr;
    a.N = (int64_t)s.R * s.S;
    a.E = s.E;
    a.K = s.K;
    a.score = o.score;
    a.normalize = o.normalize;
    a.vec = row_vectors(logits, nullptr, s.E, bf16);
    a.scale = o.scale;
    if (!with_loss) {
        // one workgroup per 16 tokens, more where that would be over 2^20 workgroups
        if (a.N == 0)
            return MOONEP_OK;
        a.n = a.N;
        a.tokens = kRowsPerBlock * (1 + a.N / ((int64_t)kRowsPerBlock << 20));
        a.per_group = (a.N + a.tokens - 1) / a.tokens;
        return by_experts<RunRouter>(s.E, a, bf16, false, a.per_group, st);
    }
    a.n = a.N / o.groups;
    a.tokens = lay.split.tokens;
    a.per_group = lay.split.per_group;
    const int rc = by_experts<RunRouter>(s.E, a, bf16, true, a.per_group * o.groups, st);
    if (rc != MOONEP_OK)
        return rc;
    const int32_t nchunk = (s.E + kJoinExperts - 1) / kJoinExperts;
    const double n = (double)a.n;
    const double factor = a.n ? (double)s.E / ((double)s.K * n * n * o.groups) : 0.0;
    double *losses = (double *)(base + lay.loss_off);
    const int64_t parts = (int64_t)nchunk * o.groups;
    hipLaunchKernelGGL(router_join_kernel, dim3((uint32_t)parts), dim3(kJoinThreads), 0, st,
                       a.prob_part, a.count_part, a.per_group, s.E, nchunk, counts, prob_sum, losses);
    hipLaunchKernelGGL(router_loss_kernel, dim3(1), dim3(kJoinThreads), 0, st, losses, parts, factor,
                       loss);
    return last();
}

int launch_router_bwd(const moonep_shape &s, const moonep_router_opts &o, const void *logits,
                      const int32_t *topk_idx, const int32_t *counts, const float *d_gates,
                      const float *d_loss, void *d_logits, hipStream_t st)
{
    RouterBwdArgs a;
    a.logits = logits;
    a.topk_idx = topk_idx;
    a.counts = counts;
    a.d_gates = d_gates;
    a.d_loss = d_loss;
    a.d_logits = d_logits;
    const int64_t N = (int64_t)s.R * s.S;
    if (N == 0)
        return MOONEP_OK;
    // without the loss no group matters
    const int64_t groups = counts ? o.groups : 1;
    const Split split = split_tokens(N / groups, groups, bwd_blocks(s.E));
    a.n = N / groups;
    a.per_group = split.per_group;
    a.tokens = split.tokens;
    a.E = s.E;
    a.K = s.K;
    a.score = o.score;
    a.normalize = o.normalize;
    const bool bf16 = o.logits_type == MOONEP_BF16;
    a.vec = row_vectors(logits, d_logits, s.E, bf16);
    a.scale = o.scale;
    a.mean = (int32_t)((a.n * s.K + s.E / 2) / s.E);
    a.factor = (float)((double)s.E / ((double)s.K * (double)a.n * (double)a.n * o.groups));
    return by_experts<RunRouterBwd>(s.E, a, bf16, split.per_group * groups, st);
}

}  // namespace moonep
