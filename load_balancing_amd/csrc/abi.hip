// abi.hip -- the extern "C" entry points of libmoonep: argument validation on
// the host, then the launches.  Every call is asynchronous on the caller's
// stream except moonep_read_error.  The operations each call performs are
// described, with the pages that define them, in include/moonep.h.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <mutex>

#include "quant.hpp"

namespace moonep {
int launch_route_stats(const moonep_shape &s, const int32_t *topk, int32_t *counts, float *maxvio,
                       void *ws, hipStream_t st);
int launch_plan(const moonep_shape &s, const int32_t *topk, const int32_t *counts, void *ws,
                int32_t *plan, int32_t *slot_of, int32_t *src_of_slot, hipStream_t st,
                int32_t policy);
size_t plan_lds_bytes(int32_t E, int32_t R);
int launch_dispatch(const moonep_shape &s, const uint16_t *x, const int32_t *slot_of, uint16_t *buf,
                    hipStream_t st);
int launch_combine(const moonep_shape &s, const uint16_t *out, const float *gates,
                   const int32_t *slot_of, uint16_t *y, hipStream_t st);
int launch_dispatch_bwd(const moonep_shape &s, const uint16_t *d_buf, const int32_t *slot_of,
                        uint16_t *dx, hipStream_t st);
int launch_combine_bwd(const moonep_shape &s, const uint16_t *dy, const uint16_t *out,
                       const float *gates, const int32_t *slot_of, uint16_t *d_out, float *d_gates,
                       hipStream_t st);
int launch_replica_reduce(const moonep_shape &s, const int32_t *plan, int64_t G, float *home,
                          float *rep, int grid, hipStream_t st);
int launch_weight_slots(const moonep_shape &s, const int32_t *plan, int32_t B, int32_t *wslot,
                        hipStream_t st);
int launch_prefetch(const moonep_shape &s, const int32_t *plan, const int32_t *wslot, int32_t B,
                    int64_t wbytes, const void *w_home, void *pool, int grid, hipStream_t st);
int gemm_out_align();
int launch_expert_gemm(const moonep_shape &s, const int32_t *plan, const int32_t *wslot, int32_t B,
                       int32_t in_dim, int32_t out_dim, const uint16_t *x, const uint16_t *w_home,
                       const uint16_t *pool, int64_t w_stride, int64_t w_offset, uint16_t *y,
                       hipStream_t st);
size_t router_workspace(const moonep_shape &s, int32_t groups);
int launch_router(const moonep_shape &s, const moonep_router_opts &o, const void *logits,
                  int32_t *topk_idx, float *gates, int32_t *counts, float *prob_sum, float *loss,
                  void *ws, hipStream_t st);
int launch_router_bwd(const moonep_shape &s, const moonep_router_opts &o, const void *logits,
                      const int32_t *topk_idx, const int32_t *counts, const float *d_gates,
                      const float *d_loss, void *d_logits, hipStream_t st);
int launch_rmsnorm_quant(const moonep_shape &s, const uint16_t *x, const uint16_t *res,
                         const uint16_t *weight, float eps, uint16_t *res_out, uint16_t *y_out,
                         uint8_t *y8, uint8_t *ys, hipStream_t st);
int launch_dispatch_quant(const moonep_shape &s, const uint8_t *x8, const uint8_t *xs,
                          const int32_t *slot_of, uint8_t *buf8, uint8_t *bufs, hipStream_t st);
int launch_quant_weights(const moonep_shape &s, int32_t in_dim, int32_t out_dim, const uint16_t *w,
                         int64_t w_stride, int64_t w_offset, uint8_t *w8, int64_t w8_stride,
                         int64_t code_offset, int64_t scale_offset, hipStream_t st);
int launch_expert_quant(const moonep_shape &s, const int32_t *plan, const int32_t *wslot, int32_t B,
                        int32_t in_dim, int32_t out_dim, const uint8_t *x8, const uint8_t *xs,
                        const uint8_t *w_home, const uint8_t *pool, int64_t w_stride,
                        const int64_t *code, const int64_t *scale, void *out, uint8_t *out_scales,
                        hipStream_t st);
}  // namespace moonep

using namespace moonep;

// Scratch of moonep_plan_noalloc: the route_stats -> plan workspace of any
// valid shape (the 256-byte control block plus E x nseg int32 counts, with
// E <= 1024 and at most 2048 wave segments), one copy per device, held until
// the process ends.  In host code this name is not a device address: the
// address comes from hipGetSymbolAddress, once per device (static_scratch).
constexpr size_t kStaticScratchBytes = kCtlBytes + (size_t)4 * kMaxExperts * kMaxSegments;
static_assert(kStaticScratchBytes == (size_t)MOONEP_NOALLOC_SCRATCH_BYTES, "scratch size");
static __device__ __align__(256) uint8_t scratch[kStaticScratchBytes];

namespace {

constexpr int kMaxDevices = 64;
std::mutex scratch_mu;
void *scratch_ptr[kMaxDevices] = {};

// Device address of the current device's copy of `scratch`.
int static_scratch(void **out)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices)
        return MOONEP_ERR_HIP;
    std::lock_guard<std::mutex> lock(scratch_mu);
    if (!scratch_ptr[dev]) {
        void *p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p)
            return MOONEP_ERR_HIP;
        scratch_ptr[dev] = p;
    }
    *out = scratch_ptr[dev];
    return MOONEP_OK;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return na && nb && x < y + nb && y < x + na;
}

int shape_status(const moonep_shape *s)
{
    if (!s)
        return MOONEP_ERR_NULL_PTR;
    if (s->R < 1 || s->E < 1 || s->S < 0 || s->K < 1 || s->H < 8)
        return MOONEP_ERR_INVALID_SHAPE;
    if (s->E % s->R != 0 || s->K > s->E || s->H % 8 != 0)
        return MOONEP_ERR_INVALID_SHAPE;
    if (s->E > kMaxExperts || s->R > kMaxRanks)
        return MOONEP_ERR_INVALID_SHAPE;
    if ((int64_t)s->R * s->S * s->K >= ((int64_t)1 << 31))
        return MOONEP_ERR_INVALID_SHAPE;
    return MOONEP_OK;
}

int64_t n_entries(const moonep_shape *s) { return (int64_t)s->R * s->S * s->K; }
int64_t n_tokens(const moonep_shape *s) { return (int64_t)s->R * s->S; }

struct Range {
    const void *p;
    size_t n;
};

// An output shares bytes with an input, or with another output.
template <int NO, int NI>
bool aliased(const Range (&out)[NO], const Range (&in)[NI])
{
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i)
            if (overlap(out[o].p, out[o].n, in[i].p, in[i].n))
                return true;
        for (int q = 0; q < o; ++q)
            if (overlap(out[o].p, out[o].n, out[q].p, out[q].n))
                return true;
    }
    return false;
}

// Pointers may be NULL only when the array they name is empty.
bool present(const void *p, int64_t n) { return p != nullptr || n == 0; }

}  // namespace

extern "C" {

int moonep_check_shape(const moonep_shape *shape) { return shape_status(shape); }

size_t moonep_workspace_bytes(const moonep_shape *shape)
{
    if (shape_status(shape) != MOONEP_OK)
        return 0;
    return ws_layout(*shape).bytes;
}

int moonep_plan_layout_of(const moonep_shape *shape, moonep_plan_layout *layout)
{
    const int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    if (!layout)
        return MOONEP_ERR_NULL_PTR;
    const PlanLayout p = plan_layout(shape->E, shape->R);
    layout->words = p.words;
    layout->cap = p.cap;
    layout->header = p.header;
    layout->rep_expert = p.rep_expert;
    layout->rep_host = p.rep_host;
    layout->rep_count = p.rep_count;
    layout->rep_spill_off = p.rep_spill_off;
    layout->rep_row_off = p.rep_row_off;
    layout->spill = p.spill;
    layout->keep = p.keep;
    layout->home_row_off = p.home_row_off;
    layout->rep_first = p.rep_first;
    layout->rep_cnt = p.rep_cnt;
    layout->exp_rep_list = p.exp_rep_list;
    layout->load = p.load;
    layout->rank_rep_first = p.rank_rep_first;
    layout->rank_rep_cnt = p.rank_rep_cnt;
    return MOONEP_OK;
}

size_t moonep_plan_bytes(const moonep_shape *shape)
{
    if (shape_status(shape) != MOONEP_OK)
        return 0;
    return (size_t)plan_layout(shape->E, shape->R).words * 4;
}

int moonep_route_stats(const moonep_shape *shape, const int32_t *topk_idx, int32_t *expert_counts,
                       float *maxvio, void *workspace, size_t workspace_bytes, void *stream)
{
    int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    const int64_t nk = n_entries(shape);
    if (!present(topk_idx, nk) || !expert_counts || !maxvio || !workspace)
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(topk_idx, 4) || !aligned(expert_counts, 4) || !aligned(maxvio, 4) ||
        !aligned(workspace, 16))
        return MOONEP_ERR_MISALIGNED;
    if (workspace_bytes < ws_layout(*shape).bytes)
        return MOONEP_ERR_WORKSPACE;
    return launch_route_stats(*shape, topk_idx, expert_counts, maxvio, workspace,
                              (hipStream_t)stream);
}

namespace {

int plan_with_policy(const moonep_shape *shape, const int32_t *topk_idx,
                     const int32_t *expert_counts, void *workspace, size_t workspace_bytes,
                     int32_t *plan, int32_t *slot_of, int32_t *src_of_slot, void *stream,
                     int32_t policy)
{
    int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    const int64_t nk = n_entries(shape);
    if (!present(topk_idx, nk) || !expert_counts || !workspace || !plan ||
        !present(slot_of, nk) || !present(src_of_slot, nk))
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(topk_idx, 4) || !aligned(expert_counts, 4) || !aligned(plan, 4) ||
        !aligned(slot_of, 4) || !aligned(src_of_slot, 4) || !aligned(workspace, 16))
        return MOONEP_ERR_MISALIGNED;
    if (workspace_bytes < ws_layout(*shape).bytes)
        return MOONEP_ERR_WORKSPACE;
    if (overlap(slot_of, nk * 4, src_of_slot, nk * 4))
        return MOONEP_ERR_ALIAS;
    return launch_plan(*shape, topk_idx, expert_counts, workspace, plan, slot_of, src_of_slot,
                       (hipStream_t)stream, policy);
}

}  // namespace

int moonep_plan(const moonep_shape *shape, const int32_t *topk_idx, const int32_t *expert_counts,
                void *workspace, size_t workspace_bytes, int32_t *plan, int32_t *slot_of,
                int32_t *src_of_slot, void *stream)
{
    return plan_with_policy(shape, topk_idx, expert_counts, workspace, workspace_bytes, plan,
                            slot_of, src_of_slot, stream, 0);
}

int moonep_plan_largest_first(const moonep_shape *shape, const int32_t *topk_idx,
                              const int32_t *expert_counts, void *workspace,
                              size_t workspace_bytes, int32_t *plan, int32_t *slot_of,
                              int32_t *src_of_slot, void *stream)
{
    return plan_with_policy(shape, topk_idx, expert_counts, workspace, workspace_bytes, plan,
                            slot_of, src_of_slot, stream, 1);
}

int moonep_plan_noalloc(const moonep_shape *shape, const int32_t *topk_idx, int32_t *expert_counts,
                        float *maxvio, int32_t *plan, int32_t *slot_of, int32_t *src_of_slot,
                        void *stream)
{
    int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    const int64_t nk = n_entries(shape);
    if (!present(topk_idx, nk) || !expert_counts || !maxvio || !plan || !present(slot_of, nk) ||
        !present(src_of_slot, nk))
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(topk_idx, 4) || !aligned(expert_counts, 4) || !aligned(maxvio, 4) ||
        !aligned(plan, 4) || !aligned(slot_of, 4) || !aligned(src_of_slot, 4))
        return MOONEP_ERR_MISALIGNED;
    if (overlap(slot_of, nk * 4, src_of_slot, nk * 4))
        return MOONEP_ERR_ALIAS;
    if (ws_layout(*shape).bytes > kStaticScratchBytes)
        return MOONEP_ERR_WORKSPACE;
    void *ws = nullptr;
    if ((rc = static_scratch(&ws)) != MOONEP_OK)
        return rc;
    const hipStream_t st = (hipStream_t)stream;
    if ((rc = launch_route_stats(*shape, topk_idx, expert_counts, maxvio, ws, st)) != MOONEP_OK)
        return rc;
    return launch_plan(*shape, topk_idx, expert_counts, ws, plan, slot_of, src_of_slot, st, 0);
}

int moonep_dispatch(const moonep_shape *shape, const uint16_t *x, const int32_t *slot_of,
                    uint16_t *buf, void *stream)
{
    int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    const int64_t nk = n_entries(shape), nt = n_tokens(shape);
    if (!present(x, nt) || !present(slot_of, nk) || !present(buf, nk))
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(x, 16) || !aligned(buf, 16) || !aligned(slot_of, 4))
        return MOONEP_ERR_MISALIGNED;
    const size_t row = (size_t)shape->H * 2;
    if (overlap(x, nt * row, buf, nk * row))
        return MOONEP_ERR_ALIAS;
    return launch_dispatch(*shape, x, slot_of, buf, (hipStream_t)stream);
}

int moonep_combine(const moonep_shape *shape, const uint16_t *expert_out, const float *gates,
                   const int32_t *slot_of, uint16_t *y, void *stream)
{
    int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    const int64_t nk = n_entries(shape), nt = n_tokens(shape);
    if (!present(expert_out, nk) || !present(gates, nk) || !present(slot_of, nk) ||
        !present(y, nt))
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(expert_out, 16) || !aligned(y, 16) || !aligned(gates, 4) || !aligned(slot_of, 4))
        return MOONEP_ERR_MISALIGNED;
    const size_t row = (size_t)shape->H * 2;
    if (overlap(expert_out, nk * row, y, nt * row))
        return MOONEP_ERR_ALIAS;
    return launch_combine(*shape, expert_out, gates, slot_of, y, (hipStream_t)stream);
}

int moonep_combine_bwd(const moonep_shape *shape, const uint16_t *dy, const uint16_t *expert_out,
                       const float *gates, const int32_t *slot_of, uint16_t *d_out,
                       float *d_gates, void *stream)
{
    int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    const int64_t nk = n_entries(shape), nt = n_tokens(shape);
    if (!present(dy, nt) || !present(expert_out, nk) || !present(gates, nk) ||
        !present(slot_of, nk) || !present(d_out, nk) || !present(d_gates, nk))
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(dy, 16) || !aligned(expert_out, 16) || !aligned(d_out, 16) || !aligned(gates, 4) ||
        !aligned(slot_of, 4) || !aligned(d_gates, 4))
        return MOONEP_ERR_MISALIGNED;
    const size_t row = (size_t)shape->H * 2;
    if (overlap(d_out, nk * row, dy, nt * row) || overlap(d_out, nk * row, expert_out, nk * row))
        return MOONEP_ERR_ALIAS;
    return launch_combine_bwd(*shape, dy, expert_out, gates, slot_of, d_out, d_gates,
                              (hipStream_t)stream);
}

int moonep_dispatch_bwd(const moonep_shape *shape, const uint16_t *d_buf, const int32_t *slot_of,
                        uint16_t *dx, void *stream)
{
    int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    const int64_t nk = n_entries(shape), nt = n_tokens(shape);
    if (!present(d_buf, nk) || !present(slot_of, nk) || !present(dx, nt))
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(d_buf, 16) || !aligned(dx, 16) || !aligned(slot_of, 4))
        return MOONEP_ERR_MISALIGNED;
    const size_t row = (size_t)shape->H * 2;
    if (overlap(d_buf, nk * row, dx, nt * row))
        return MOONEP_ERR_ALIAS;
    return launch_dispatch_bwd(*shape, d_buf, slot_of, dx, (hipStream_t)stream);
}

int moonep_replica_grad_reduce(const moonep_shape *shape, const int32_t *plan, int64_t G,
                               float *home_grads, float *replica_grads, void *stream)
{
    int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    if (G < 0)
        return MOONEP_ERR_ARG;
    if (!plan || !present(home_grads, G) || !present(replica_grads, G))
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(plan, 4) || !aligned(home_grads, 4) || !aligned(replica_grads, 4))
        return MOONEP_ERR_MISALIGNED;
    const size_t hb = (size_t)shape->E * (size_t)G * 4;
    const size_t rb = (size_t)(shape->E + shape->R) * (size_t)G * 4;
    if (overlap(home_grads, hb, replica_grads, rb))
        return MOONEP_ERR_ALIAS;
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
        return MOONEP_ERR_HIP;
    return launch_replica_reduce(*shape, plan, G, home_grads, replica_grads, cus * 4,
                                 (hipStream_t)stream);
}

int moonep_weight_slots(const moonep_shape *shape, const int32_t *plan, int32_t B, int32_t *wslot,
                        void *stream)
{
    int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    if (B < 0 || (int64_t)shape->R * B >= ((int64_t)1 << 31))
        return MOONEP_ERR_ARG;
    if (!plan || !wslot)
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(plan, 4) || !aligned(wslot, 4))
        return MOONEP_ERR_MISALIGNED;
    return launch_weight_slots(*shape, plan, B, wslot, (hipStream_t)stream);
}

int moonep_prefetch_weights(const moonep_shape *shape, const int32_t *plan, const int32_t *wslot,
                            int32_t B, int64_t wbytes, const void *w_home, void *pool, void *stream)
{
    int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    if (B < 0 || (int64_t)shape->R * B >= ((int64_t)1 << 31) || wbytes < 0 || wbytes % 16 != 0)
        return MOONEP_ERR_ARG;
    const int64_t pool_rows = (int64_t)shape->R * B;
    if (!plan || !wslot || !present(w_home, wbytes) || !present(pool, pool_rows * wbytes))
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(plan, 4) || !aligned(wslot, 4) || !aligned(w_home, 16) || !aligned(pool, 16))
        return MOONEP_ERR_MISALIGNED;
    if (overlap(w_home, (size_t)shape->E * (size_t)wbytes, pool, (size_t)pool_rows * (size_t)wbytes))
        return MOONEP_ERR_ALIAS;
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
        return MOONEP_ERR_HIP;
    return launch_prefetch(*shape, plan, wslot, B, wbytes, w_home, pool, cus * 4,
                           (hipStream_t)stream);
}

int moonep_expert_gemm(const moonep_shape *shape, const int32_t *plan, const int32_t *wslot,
                       int32_t B, int32_t in_dim, int32_t out_dim, const uint16_t *x,
                       const uint16_t *w_home, const uint16_t *pool, int64_t w_stride,
                       int64_t w_offset, uint16_t *y, void *stream)
{
    int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    // the kernel addresses a row of a tile by a 32-bit byte offset: 256 rows of in_dim bf16
    constexpr int32_t kMaxInDim = 1 << 22;
    if (B < 0 || (int64_t)shape->R * B >= ((int64_t)1 << 31) || in_dim <= 0 || in_dim % 64 != 0 ||
        in_dim > kMaxInDim || out_dim <= 0 || out_dim % gemm_out_align() != 0 ||
        w_stride % 8 != 0 || w_offset < 0 || w_offset % 8 != 0 ||
        w_offset + (int64_t)out_dim * in_dim > w_stride)
        return MOONEP_ERR_ARG;
    const int64_t rows = n_entries(shape);
    const int64_t pool_rows = (int64_t)shape->R * B;
    if (!plan || !wslot || !w_home || !present(x, rows) || !present(y, rows) ||
        !present(pool, pool_rows))
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(plan, 4) || !aligned(wslot, 4) || !aligned(x, 16) || !aligned(y, 16) ||
        !aligned(w_home, 16) || !aligned(pool, 16))
        return MOONEP_ERR_MISALIGNED;
    const size_t yb = (size_t)rows * out_dim * 2;
    if (overlap(y, yb, x, (size_t)rows * in_dim * 2) ||
        overlap(y, yb, w_home, (size_t)shape->E * (size_t)w_stride * 2) ||
        overlap(y, yb, pool, (size_t)pool_rows * (size_t)w_stride * 2))
        return MOONEP_ERR_ALIAS;
    return launch_expert_gemm(*shape, plan, wslot, B, in_dim, out_dim, x, w_home, pool, w_stride,
                              w_offset, y, (hipStream_t)stream);
}

namespace {

// The rules of moonep_router_opts.
int router_status(const moonep_shape *s, const moonep_router_opts *o)
{
    if (!o)
        return MOONEP_ERR_NULL_PTR;
    if ((o->score != MOONEP_SCORE_SOFTMAX && o->score != MOONEP_SCORE_SIGMOID) ||
        (o->logits_type != MOONEP_F32 && o->logits_type != MOONEP_BF16) || !isfinite(o->scale) ||
        o->groups < 1 || o->groups > (1 << 20) || n_tokens(s) % o->groups != 0 ||
        (int64_t)o->groups * s->E > (1 << 24))
        return MOONEP_ERR_ARG;
    return MOONEP_OK;
}

// A matrix of out_dim x in_dim codes and its scales inside a weight row of
// `stride` bytes.
struct Window {
    int64_t code, scale, code_bytes, scale_bytes;

    Window(int64_t c, int64_t sc, int32_t in_dim, int32_t out_dim)
        : code(c), scale(sc), code_bytes((int64_t)out_dim * in_dim),
          scale_bytes((int64_t)((out_dim - 1) / kQuantBlock + 1) * scale_row_bytes(in_dim))
    {
    }
    bool inside(int64_t stride) const
    {
        return code >= 0 && code % 16 == 0 && scale >= 0 && scale % 4 == 0 &&
               code_bytes <= stride && code <= stride - code_bytes && scale_bytes <= stride &&
               scale <= stride - scale_bytes &&
               (code + code_bytes <= scale || scale + scale_bytes <= code);
    }
};

int expert_quant(const moonep_shape *shape, const int32_t *plan, const int32_t *wslot, int32_t B,
                 int32_t in_dim, int32_t out_dim, const uint8_t *x8, const uint8_t *xs,
                 const uint8_t *w_home, const uint8_t *pool, int64_t w_stride, int nmat,
                 const int64_t *code, const int64_t *scale, void *out, int64_t out_row,
                 uint8_t *out_scales, void *stream)
{
    const int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    // the kernel addresses a row of a tile, in and out, by a 32-bit byte offset
    constexpr int32_t kMaxDim = 1 << 22;
    if (B < 0 || (int64_t)shape->R * B >= ((int64_t)1 << 31) || in_dim <= 0 || in_dim % 16 != 0 ||
        in_dim > kMaxDim || out_dim <= 0 || out_dim % 16 != 0 || out_dim > kMaxDim ||
        w_stride <= 0 || w_stride % 16 != 0)
        return MOONEP_ERR_ARG;
    for (int m = 0; m < nmat; ++m)
        if (!Window(code[m], scale[m], in_dim, out_dim).inside(w_stride))
            return MOONEP_ERR_ARG;
    const int64_t rows = n_entries(shape), pool_rows = (int64_t)shape->R * B;
    if (!plan || !wslot || !w_home || !present(x8, rows) || !present(xs, rows) ||
        !present(out, rows) || (nmat == 2 && !present(out_scales, rows)) || !present(pool, pool_rows))
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(plan, 4) || !aligned(wslot, 4) || !aligned(x8, 16) || !aligned(xs, 4) ||
        !aligned(out, 16) || !aligned(out_scales, 4) || !aligned(w_home, 16) || !aligned(pool, 16))
        return MOONEP_ERR_MISALIGNED;
    const Range out_r[] = {{out, (size_t)rows * (size_t)out_row},
                           {out_scales, out_scales ? (size_t)rows * scale_row_bytes(out_dim) : 0}};
    const Range in_r[] = {{x8, (size_t)rows * in_dim},
                          {xs, (size_t)rows * scale_row_bytes(in_dim)},
                          {w_home, (size_t)shape->E * (size_t)w_stride},
                          {pool, (size_t)pool_rows * (size_t)w_stride},
                          {plan, moonep_plan_bytes(shape)},
                          {wslot, (size_t)(shape->E + shape->R) * 4}};
    if (aliased(out_r, in_r))
        return MOONEP_ERR_ALIAS;
    if (rows == 0)
        return MOONEP_OK;
    return launch_expert_quant(*shape, plan, wslot, B, in_dim, out_dim, x8, xs, w_home, pool,
                               w_stride, code, scale, out, out_scales, (hipStream_t)stream);
}

}  // namespace

size_t moonep_router_workspace_bytes(const moonep_shape *shape, const moonep_router_opts *opts)
{
    if (shape_status(shape) != MOONEP_OK || router_status(shape, opts) != MOONEP_OK)
        return 0;
    return router_workspace(*shape, opts->groups);
}

int moonep_router(const moonep_shape *shape, const moonep_router_opts *opts, const void *logits,
                  int32_t *topk_idx, float *gates, int32_t *counts, float *prob_sum, float *loss,
                  void *workspace, size_t workspace_bytes, void *stream)
{
    int rc = shape_status(shape);
    if (rc != MOONEP_OK || (rc = router_status(shape, opts)) != MOONEP_OK)
        return rc;
    const int64_t nk = n_entries(shape);
    const bool some = counts || prob_sum || loss || workspace;
    if (!present(logits, nk) || !present(topk_idx, nk) || !present(gates, nk) ||
        (some && !(counts && prob_sum && loss && workspace)))
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(logits, opts->logits_type == MOONEP_BF16 ? 2 : 4) || !aligned(topk_idx, 4) ||
        !aligned(gates, 4) || !aligned(counts, 4) || !aligned(prob_sum, 4) || !aligned(loss, 4) ||
        !aligned(workspace, 16))
        return MOONEP_ERR_MISALIGNED;
    if (some && workspace_bytes < router_workspace(*shape, opts->groups))
        return MOONEP_ERR_WORKSPACE;
    const size_t table = some ? (size_t)opts->groups * shape->E * 4 : 0;
    const Range in[] = {{logits, (size_t)n_tokens(shape) * shape->E *
                                     (opts->logits_type == MOONEP_BF16 ? 2 : 4)}};
    const Range out[] = {{topk_idx, (size_t)nk * 4}, {gates, (size_t)nk * 4}, {counts, table},
                         {prob_sum, table}, {loss, some ? (size_t)4 : 0},
                         {workspace, some ? router_workspace(*shape, opts->groups) : 0}};
    if (aliased(out, in))
        return MOONEP_ERR_ALIAS;
    return launch_router(*shape, *opts, logits, topk_idx, gates, counts, prob_sum, loss, workspace,
                         (hipStream_t)stream);
}

int moonep_router_bwd(const moonep_shape *shape, const moonep_router_opts *opts,
                      const void *logits, const int32_t *topk_idx, const int32_t *counts,
                      const float *d_gates, const float *d_loss, void *d_logits, void *stream)
{
    int rc = shape_status(shape);
    if (rc != MOONEP_OK || (rc = router_status(shape, opts)) != MOONEP_OK)
        return rc;
    const int64_t nk = n_entries(shape);
    if (!present(logits, nk) || !present(topk_idx, nk) || !present(d_logits, nk) ||
        (counts != nullptr) != (d_loss != nullptr))
        return MOONEP_ERR_NULL_PTR;
    const size_t la = opts->logits_type == MOONEP_BF16 ? 2 : 4;
    if (!aligned(logits, la) || !aligned(d_logits, la) || !aligned(topk_idx, 4) ||
        !aligned(counts, 4) || !aligned(d_gates, 4) || !aligned(d_loss, 4))
        return MOONEP_ERR_MISALIGNED;
    const size_t lb = (size_t)n_tokens(shape) * shape->E * la;
    const Range in[] = {{logits, lb}, {topk_idx, (size_t)nk * 4},
                        {counts, counts ? (size_t)opts->groups * shape->E * 4 : 0},
                        {d_gates, d_gates ? (size_t)nk * 4 : 0}, {d_loss, d_loss ? (size_t)4 : 0}};
    const Range out[] = {{d_logits, lb}};
    if (aliased(out, in))
        return MOONEP_ERR_ALIAS;
    return launch_router_bwd(*shape, *opts, logits, topk_idx, counts, d_gates, d_loss, d_logits,
                             (hipStream_t)stream);
}

size_t moonep_scale_bytes(int32_t cols) { return cols < 1 ? 0 : (size_t)scale_row_bytes(cols); }

int moonep_rmsnorm_quant(const moonep_shape *shape, const uint16_t *x, const uint16_t *res,
                         const uint16_t *weight, float eps, uint16_t *res_out, uint16_t *y_out,
                         uint8_t *y8, uint8_t *ys, void *stream)
{
    const int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    if (shape->H % 16 != 0 || shape->H > 65536 || !isfinite(eps) || eps < 0.0f)
        return MOONEP_ERR_ARG;
    const int64_t n = n_tokens(shape);
    if (!present(x, n) || !weight || !present(y8, n) || !present(ys, n) ||
        (res != nullptr) != (res_out != nullptr))
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(x, 16) || !aligned(res, 16) || !aligned(weight, 16) || !aligned(res_out, 16) ||
        !aligned(y_out, 16) || !aligned(y8, 16) || !aligned(ys, 4))
        return MOONEP_ERR_MISALIGNED;
    const size_t row = (size_t)n * shape->H * 2, wb = (size_t)shape->H * 2;
    // the sum may go over x or res, whole rows over themselves
    const Range in[] = {{res_out == x ? nullptr : x, res_out == x ? 0 : row},
                        {res, res && res_out != res ? row : 0}, {weight, wb}};
    const Range out[] = {{res_out, res_out ? row : 0}, {y_out, y_out ? row : 0}, {y8, row / 2},
                         {ys, (size_t)n * scale_row_bytes(shape->H)}};
    if (aliased(out, in))
        return MOONEP_ERR_ALIAS;
    return launch_rmsnorm_quant(*shape, x, res, weight, eps, res_out, y_out, y8, ys,
                                (hipStream_t)stream);
}

int moonep_dispatch_quant(const moonep_shape *shape, const uint8_t *x8, const uint8_t *xs,
                          const int32_t *slot_of, uint8_t *buf8, uint8_t *bufs, void *stream)
{
    const int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    if (shape->H % 16 != 0)
        return MOONEP_ERR_ARG;
    const int64_t nk = n_entries(shape), nt = n_tokens(shape);
    if (!present(x8, nt) || !present(xs, nt) || !present(slot_of, nk) || !present(buf8, nk) ||
        !present(bufs, nk))
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(x8, 16) || !aligned(buf8, 16) || !aligned(xs, 4) || !aligned(bufs, 4) ||
        !aligned(slot_of, 4))
        return MOONEP_ERR_MISALIGNED;
    const size_t row = (size_t)shape->H, sr = (size_t)scale_row_bytes(shape->H);
    const Range in[] = {{x8, nt * row}, {xs, nt * sr}, {slot_of, (size_t)nk * 4}};
    const Range out[] = {{buf8, nk * row}, {bufs, nk * sr}};
    if (aliased(out, in))
        return MOONEP_ERR_ALIAS;
    return launch_dispatch_quant(*shape, x8, xs, slot_of, buf8, bufs, (hipStream_t)stream);
}

int moonep_quant_weights(const moonep_shape *shape, int32_t in_dim, int32_t out_dim,
                         const uint16_t *w, int64_t w_stride, int64_t w_offset, uint8_t *w8,
                         int64_t w8_stride, int64_t code_offset, int64_t scale_offset, void *stream)
{
    const int rc = shape_status(shape);
    if (rc != MOONEP_OK)
        return rc;
    constexpr int32_t kMaxDim = 1 << 30;
    if (in_dim <= 0 || in_dim % 16 != 0 || in_dim > kMaxDim || out_dim <= 0 || out_dim > kMaxDim ||
        w_stride <= 0 || w_stride % 8 != 0 || w_offset < 0 || w_offset % 8 != 0 || w8_stride <= 0 ||
        w8_stride % 16 != 0)
        return MOONEP_ERR_ARG;
    const Window win(code_offset, scale_offset, in_dim, out_dim);
    if (win.code_bytes > w_stride || w_offset > w_stride - win.code_bytes || !win.inside(w8_stride))
        return MOONEP_ERR_ARG;
    if (!w || !w8)
        return MOONEP_ERR_NULL_PTR;
    if (!aligned(w, 16) || !aligned(w8, 16))
        return MOONEP_ERR_MISALIGNED;
    if (overlap(w, (size_t)shape->E * (size_t)w_stride * 2, w8, (size_t)shape->E * (size_t)w8_stride))
        return MOONEP_ERR_ALIAS;
    return launch_quant_weights(*shape, in_dim, out_dim, w, w_stride, w_offset, w8, w8_stride,
                                code_offset, scale_offset, (hipStream_t)stream);
}

int moonep_expert_gemm_quant(const moonep_shape *shape, const int32_t *plan, const int32_t *wslot,
                             int32_t B, int32_t in_dim, int32_t out_dim, const uint8_t *x8,
                             const uint8_t *xs, const uint8_t *w_home, const uint8_t *pool,
                             int64_t w_stride, int64_t code_offset, int64_t scale_offset,
                             uint16_t *y, void *stream)
{
    return expert_quant(shape, plan, wslot, B, in_dim, out_dim, x8, xs, w_home, pool, w_stride, 1,
                        &code_offset, &scale_offset, y, (int64_t)out_dim * 2, nullptr, stream);
}

int moonep_expert_glu_quant(const moonep_shape *shape, const int32_t *plan, const int32_t *wslot,
                            int32_t B, int32_t in_dim, int32_t mid_dim, const uint8_t *x8,
                            const uint8_t *xs, const uint8_t *w_home, const uint8_t *pool,
                            int64_t w_stride, int64_t gate_code_offset, int64_t gate_scale_offset,
                            int64_t up_code_offset, int64_t up_scale_offset, uint8_t *h8,
                            uint8_t *hs, void *stream)
{
    const int64_t code[2] = {gate_code_offset, up_code_offset};
    const int64_t scale[2] = {gate_scale_offset, up_scale_offset};
    return expert_quant(shape, plan, wslot, B, in_dim, mid_dim, x8, xs, w_home, pool, w_stride, 2,
                        code, scale, h8, mid_dim, hs, stream);
}

int moonep_read_error(void *workspace, size_t workspace_bytes, int32_t *host_code, void *stream)
{
    if (!workspace || !host_code)
        return MOONEP_ERR_NULL_PTR;
    if (workspace_bytes < kCtlBytes)
        return MOONEP_ERR_WORKSPACE;
    hipStream_t st = (hipStream_t)stream;
    int32_t v = 0;
    if (hipMemcpyAsync(&v, (int32_t *)workspace + kCtlError, 4, hipMemcpyDeviceToHost, st) !=
            hipSuccess ||
        hipStreamSynchronize(st) != hipSuccess)
        return MOONEP_ERR_HIP;
    *host_code = v;
    if (v != 0) {
        if (hipMemsetAsync((int32_t *)workspace + kCtlError, 0, 4, st) != hipSuccess ||
            hipStreamSynchronize(st) != hipSuccess)
            return MOONEP_ERR_HIP;
    }
    return MOONEP_OK;
}

}  // extern "C"
