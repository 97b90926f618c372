// C ABI of the group norm: argument validation (before any HIP call) and launches on the
// caller's stream.  Declared in iabn.h.
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "checks.hpp"
#include "gnorm.hpp"
#include "iabn.h"

using namespace iabn;

namespace {

constexpr int64_t kGnMaxC = int64_t(1) << 26;
constexpr int64_t kGnMaxGroups = int64_t(1) << 24;  // a workgroup of 256 each: threads in 32 bits

iabn_status check_gn(const iabn_group_norm* l)
{
    if (!l || !dtype_ok(l->dtype) || l->n < 0 || l->hw < 0 || l->c < 0) return IABN_ERR_INVALID_ARG;
    if (l->groups < 1 || l->c % l->groups != 0) return IABN_ERR_INVALID_ARG;
    if (l->act < IABN_GN_SILU || l->act > IABN_GN_LEAKY_RELU) return IABN_ERR_INVALID_ARG;
    if (!isfinite(l->act_param) || !(l->eps >= 0.f) || !isfinite(l->eps)) return IABN_ERR_INVALID_ARG;
    IABN_TRY(check_vec(l->weight));
    IABN_TRY(check_vec(l->bias));
    if (l->c >= kGnMaxC || l->groups >= kGnMaxGroups || double(l->n) * double(l->hw) > double(kMaxExtent) || l->n > kMaxExtent ||
        l->hw > kMaxExtent)
        return IABN_ERR_UNSUPPORTED;
    return IABN_OK;
}

bool empty(const iabn_group_norm* l) { return l->n == 0 || l->hw == 0 || l->c == 0; }

GnArgs gn_args(const iabn_group_norm* l)
{
    GnArgs a{};
    a.N = l->n; a.HW = l->hw; a.C = l->c; a.G = l->groups;
    a.weight = l->weight; a.bias = l->bias;
    a.act = l->act; a.param = l->act_param; a.eps = l->eps;
    return a;
}

size_t gn_need(const iabn_group_norm* l)
{
    return empty(l) ? 0 : gn_workspace_bytes(l->n, l->hw, l->c, l->groups, device_cus());
}

}  // namespace

extern "C" {

size_t iabn_group_norm_workspace_size(const iabn_group_norm* l)
{
    return check_gn(l) == IABN_OK ? gn_need(l) : 0;
}

iabn_status iabn_group_norm_forward(const iabn_group_norm* l, const void* x, int64_t ldx, void* y,
                                    int64_t ldy, float* stats, void* workspace,
                                    size_t workspace_bytes, hipStream_t stream)
{
    IABN_TRY(check_gn(l));
    if (empty(l)) return IABN_OK;
    const int64_t T = l->n * l->hw, C = l->c, es = esize(l->dtype);
    const Rows in{x, ldx, T, C, es}, out{y, ldy, T, C, es};
    IABN_TRY(check_rows(in));
    IABN_TRY(check_rows(out));
    if (!aligned(stats, 8)) return IABN_ERR_MISALIGNED;
    const size_t need = gn_need(l);
    IABN_TRY(check_ws(workspace, workspace_bytes, need));
    const Rows outs[] = {out, vector_row(stats, 2 * l->n * l->groups),
                         vector_row(workspace, int64_t(need), 1)};
    const Rows vectors[] = {vector_row(l->weight, C), vector_row(l->bias, C)};
    IABN_TRY(check_distinct(outs));
    IABN_TRY(check_all_apart(outs, vectors));
    IABN_TRY(check_out(out, in));
    IABN_TRY(check_apart(outs[1], in));
    IABN_TRY(check_apart(outs[2], in));
    GnArgs a = gn_args(l);
    a.x = x; a.ldx = ldx;
    a.out = y; a.ldo = ldy;
    a.stats = stats;
    launch_gn_forward(a, l->dtype, device_cus(), workspace, stream);
    return launched();
}

iabn_status iabn_group_norm_backward(const iabn_group_norm* l, const void* x, int64_t ldx,
                                     const void* dy, int64_t lddy, void* dx, int64_t lddx,
                                     const float* stats, float* dweight, float* dbias,
                                     void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    IABN_TRY(check_gn(l));
    const int64_t T = l->n * l->hw, C = l->c, es = esize(l->dtype);
    if (C == 0 || (!dx && !dweight && !dbias)) return IABN_OK;
    const Rows in{x, ldx, T, C, es}, grad{dy, lddy, T, C, es}, out{dx, lddx, T, C, es};
    IABN_TRY(check_vec(dweight));
    IABN_TRY(check_vec(dbias));
    if (T > 0) {
        IABN_TRY(check_rows(in));
        IABN_TRY(check_rows(grad));
        if (dx) IABN_TRY(check_rows(out));
        if (!stats) return IABN_ERR_INVALID_ARG;
        if (!aligned(stats, 8)) return IABN_ERR_MISALIGNED;
    }
    const size_t need = gn_need(l);
    IABN_TRY(check_ws(workspace, workspace_bytes, need));
    const Rows space = vector_row(need ? workspace : nullptr, int64_t(need), 1);
    const Rows outs[] = {out, vector_row(dweight, C), vector_row(dbias, C), space};
    const Rows st = vector_row(stats, 2 * l->n * l->groups);
    const Rows w = vector_row(l->weight, C), b = vector_row(l->bias, C);
    const Rows fixed[] = {st}, tensors[] = {in, grad};
    IABN_TRY(check_distinct(outs));
    IABN_TRY(check_all_apart(outs, fixed));
    IABN_TRY(check_out(out, in));
    IABN_TRY(check_out(out, grad));
    for (int i = 1; i < 4; ++i)
        for (const Rows& t : tensors) IABN_TRY(check_apart(outs[i], t));
    // written by the last kernel, which reads neither
    IABN_TRY(check_out(outs[1], w));
    IABN_TRY(check_out(outs[2], b));
    IABN_TRY(check_apart(outs[1], b));
    IABN_TRY(check_apart(outs[2], w));
    const Rows rest[] = {out, space}, vectors[] = {w, b};
    IABN_TRY(check_all_apart(rest, vectors));
    GnArgs a = gn_args(l);
    a.x = x; a.ldx = ldx;
    a.dy = dy; a.lddy = lddy;
    a.out = dx; a.ldo = lddx;
    a.stats = const_cast<float*>(stats);
    a.dweight = dweight; a.dbias = dbias;
    launch_gn_backward(a, l->dtype, device_cus(), workspace, stream);
    return launched();
}

}  // extern "C"
