// C ABI of the residual-block operators: argument validation (before any HIP
// call) and launches on the caller's stream.  Declared in iabn.h.
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "block.hpp"
#include "checks.hpp"
#include "iabn.h"

using namespace iabn;

namespace {

bool glu_act_ok(int a)
{
    return a == IABN_GLU_SILU || a == IABN_GLU_GELU || a == IABN_GLU_GELU_TANH;
}

bool norm_ok(int k) { return k == IABN_NORM_NONE || k == IABN_NORM_RMS || k == IABN_NORM_LAYER; }

iabn_status check_layer(const iabn_resnorm* l)
{
    if (!l) return IABN_ERR_INVALID_ARG;
    IABN_TRY(check_extents(l->rows, l->cols, l->dtype));
    if (!norm_ok(l->post) || !norm_ok(l->pre)) return IABN_ERR_INVALID_ARG;
    if (!isfinite(l->alpha) || !(l->eps >= 0.f) || !isfinite(l->eps)) return IABN_ERR_INVALID_ARG;
    IABN_TRY(check_vec(l->post_weight));
    IABN_TRY(check_vec(l->post_bias));
    IABN_TRY(check_vec(l->pre_weight));
    IABN_TRY(check_vec(l->pre_bias));
    if (l->gate) {
        if (l->gate_dtype != IABN_F32 && l->gate_dtype != l->dtype) return IABN_ERR_INVALID_ARG;
        if (l->rows_per_gate < 1 || (l->rows > 0 && l->rows % l->rows_per_gate != 0))
            return IABN_ERR_INVALID_ARG;
        if (!aligned(l->gate, size_t(esize(l->gate_dtype)))) return IABN_ERR_MISALIGNED;
    }
    return l->cols <= kResnormMaxC ? IABN_OK : IABN_ERR_UNSUPPORTED;
}

Rows gate_tensor(const iabn_resnorm* l, const void* p)
{
    const int64_t groups = l->gate && l->rows > 0 ? l->rows / l->rows_per_gate : 0;
    return Rows{p, l->cols, groups, l->cols, esize(l->gate_dtype)};
}
Rows gate_tensor(const iabn_resnorm* l) { return gate_tensor(l, l->gate); }

int64_t gate_rows(const iabn_resnorm* l)
{
    return l->gate ? l->rows_per_gate : max64(1, l->rows);
}

}  // namespace

extern "C" {

iabn_status iabn_codes_pack(const void* x, int64_t ldx, int64_t rows, int64_t cols,
                            iabn_dtype dtype, int8_t* codes, uint8_t* exps, hipStream_t stream)
{
    IABN_TRY(check_extents(rows, cols, dtype));
    if (rows == 0 || cols == 0) return IABN_OK;
    const Rows in{x, ldx, rows, cols, esize(dtype)};
    IABN_TRY(check_rows(in));
    IABN_TRY(check_codes(codes, exps));
    IABN_TRY(check_codes_apart(codes, exps, rows, cols, in));
    IABN_TRY(check_apart(code_rows(codes, rows, cols), exp_rows(exps, rows, cols)));
    launch_codes_pack(x, ldx, rows, cols, dtype, codes, exps, stream);
    return launched();
}

iabn_status iabn_codes_unpack(const int8_t* codes, const uint8_t* exps, int64_t rows,
                              int64_t cols, const float* scale, const float* shift, void* y,
                              int64_t ldy, iabn_dtype dtype, hipStream_t stream)
{
    IABN_TRY(check_extents(rows, cols, dtype));
    if (rows == 0 || cols == 0) return IABN_OK;
    const Rows out{y, ldy, rows, cols, esize(dtype)};
    IABN_TRY(check_rows(out));
    IABN_TRY(check_codes(codes, exps));
    IABN_TRY(check_vec(scale));
    IABN_TRY(check_vec(shift));
    IABN_TRY(check_codes_apart(codes, exps, rows, cols, out));
    IABN_TRY(check_apart(out, vector_row(scale, cols)));
    IABN_TRY(check_apart(out, vector_row(shift, cols)));
    launch_codes_unpack(codes, exps, rows, cols, scale, shift, y, ldy, dtype, stream);
    return launched();
}

iabn_status iabn_glu_forward(const void* gate, int64_t ldgate, const void* up, int64_t ldup,
                             void* out, int64_t ldout, int64_t rows, int64_t cols,
                             iabn_dtype dtype, iabn_glu_act act, int8_t* codes_gate,
                             uint8_t* exps_gate, int8_t* codes_up, uint8_t* exps_up,
                             hipStream_t stream)
{
    IABN_TRY(check_extents(rows, cols, dtype));
    if (!glu_act_ok(act)) return IABN_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return IABN_OK;
    const int64_t es = esize(dtype);
    const Rows g{gate, ldgate, rows, cols, es}, u{up, ldup, rows, cols, es},
        o{out, ldout, rows, cols, es};
    IABN_TRY(check_rows(g));
    if (up) IABN_TRY(check_rows(u));
    IABN_TRY(check_rows(o));
    IABN_TRY(check_codes_opt(codes_gate, exps_gate));
    IABN_TRY(check_codes_opt(codes_up, exps_up));
    if ((codes_up != nullptr) != (codes_gate != nullptr && up != nullptr))
        return IABN_ERR_INVALID_ARG;
    IABN_TRY(check_out(o, g));
    IABN_TRY(check_out(o, u));
    for (const Rows& t : {g, u, o}) {
        IABN_TRY(check_codes_apart(codes_gate, exps_gate, rows, cols, t));
        IABN_TRY(check_codes_apart(codes_up, exps_up, rows, cols, t));
    }
    const Rows kept[] = {code_rows(codes_gate, rows, cols), exp_rows(exps_gate, rows, cols),
                         code_rows(codes_up, rows, cols), exp_rows(exps_up, rows, cols)};
    IABN_TRY(check_distinct(kept));
    const GluFwd a{gate, up, out, ldgate, ldup, ldout, codes_gate, codes_up, exps_gate, exps_up};
    launch_glu_forward(a, rows, cols, dtype, act, stream);
    return launched();
}

iabn_status iabn_glu_backward(const int8_t* codes_gate, const uint8_t* exps_gate,
                              const int8_t* codes_up, const uint8_t* exps_up, const void* dout,
                              int64_t lddout, void* dgate, int64_t lddgate, void* dup,
                              int64_t lddup, void* out, int64_t ldout, int64_t rows, int64_t cols,
                              iabn_dtype dtype, iabn_glu_act act, hipStream_t stream)
{
    IABN_TRY(check_extents(rows, cols, dtype));
    if (!glu_act_ok(act)) return IABN_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return IABN_OK;
    const int64_t es = esize(dtype);
    const Rows d{dout, lddout, rows, cols, es}, dg{dgate, lddgate, rows, cols, es},
        du{dup, lddup, rows, cols, es}, o{out, ldout, rows, cols, es};
    IABN_TRY(check_codes(codes_gate, exps_gate));
    IABN_TRY(check_codes_opt(codes_up, exps_up));
    if ((codes_up != nullptr) != (dup != nullptr)) return IABN_ERR_INVALID_ARG;
    IABN_TRY(check_rows(d));
    IABN_TRY(check_rows(dg));
    if (dup) IABN_TRY(check_rows(du));
    if (out) IABN_TRY(check_rows(o));
    IABN_TRY(check_out(dg, d));
    IABN_TRY(check_out(du, d));
    IABN_TRY(check_out(o, d));
    IABN_TRY(check_apart(dg, du));
    IABN_TRY(check_apart(dg, o));
    IABN_TRY(check_apart(du, o));
    for (const Rows& t : {dg, du, o}) {
        IABN_TRY(check_codes_apart(codes_gate, exps_gate, rows, cols, t));
        IABN_TRY(check_codes_apart(codes_up, exps_up, rows, cols, t));
    }
    const GluBwd a{codes_gate, codes_up, exps_gate, exps_up, dout,  dgate,
                   dup,        out,      lddout,    lddgate, lddup, ldout};
    launch_glu_backward(a, rows, cols, dtype, act, stream);
    return launched();
}

size_t iabn_linear_wgrad_workspace_size(int64_t rows, int64_t n, int64_t k, iabn_dtype dtype)
{
    if (check_extents(rows, n, dtype) != IABN_OK || check_extents(rows, k, dtype) != IABN_OK)
        return 0;
    if (n == 0) return 0;
    return wgrad_workspace_bytes(rows, n, k, dtype, device_cus());
}

iabn_status iabn_linear_wgrad(const void* dy, int64_t lddy, iabn_dtype dtype, const int8_t* codes,
                              const uint8_t* exps, const float* scale, const float* shift,
                              void* dw, int64_t lddw, iabn_dtype dw_dtype, float* dbias,
                              int accumulate, int64_t rows, int64_t n, int64_t k,
                              void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    IABN_TRY(check_extents(rows, n, dtype));
    IABN_TRY(check_extents(rows, k, dw_dtype));
    if (n == 0 || (k == 0 && !dbias)) return IABN_OK;
    // tiles of 128 x 128 in 31 bits of workgroups
    if (double(ceil_div(n, 128)) * double(ceil_div(k, 128)) > 2.0e9) return IABN_ERR_UNSUPPORTED;
    if (lddy >= kWgradMaxLd || k >= kWgradMaxLd) return IABN_ERR_UNSUPPORTED;
    const Rows out{dw, lddw, n, k, esize(dw_dtype)};
    const Rows in{dy, lddy, rows, n, esize(dtype)};
    if (k > 0) IABN_TRY(check_rows(out));
    IABN_TRY(check_vec(scale));
    IABN_TRY(check_vec(shift));
    IABN_TRY(check_vec(dbias));
    if (rows > 0) {
        IABN_TRY(check_rows(in));
        if (k > 0) IABN_TRY(check_codes(codes, exps));
    }
    const int64_t cus = device_cus();
    const size_t need = wgrad_workspace_bytes(rows, n, k, dtype, cus);
    IABN_TRY(check_ws(workspace, workspace_bytes, need));
    const Rows outs[] = {out, vector_row(dbias, n),
                         vector_row(need ? workspace : nullptr, int64_t(need), 1)};
    const Rows ins[] = {in, code_rows(codes, rows, k), exp_rows(exps, rows, k),
                        vector_row(scale, k), vector_row(shift, k)};
    IABN_TRY(check_distinct(outs));
    IABN_TRY(check_all_apart(outs, ins));
    const WgradArgs a{dy,    lddy,       codes, exps, scale, shift, dw, lddw, dw_dtype,
                      accumulate != 0, dbias, rows, n,     k};
    launch_linear_wgrad(a, dtype, cus, workspace, stream);
    return launched();
}

iabn_status iabn_resnorm_forward(const iabn_resnorm* l, const void* r, int64_t ldr, const void* b,
                                 int64_t ldb, void* r_out, int64_t ldr_out, void* n, int64_t ldn,
                                 float* post_stats, float* pre_stats, int8_t* codes_b,
                                 uint8_t* exps_b, int8_t* codes_n, uint8_t* exps_n,
                                 hipStream_t stream)
{
    IABN_TRY(check_layer(l));
    const int64_t T = l->rows, C = l->cols, es = esize(l->dtype);
    if (T == 0 || C == 0) return IABN_OK;
    const Rows tr{r, ldr, T, C, es}, tb{b, ldb, T, C, es}, to{r_out, ldr_out, T, C, es},
        tn{n, ldn, T, C, es};
    IABN_TRY(check_rows(tr));
    if (b) IABN_TRY(check_rows(tb));
    if (r_out) IABN_TRY(check_rows(to));
    if ((n != nullptr) != (l->pre != IABN_NORM_NONE)) return IABN_ERR_INVALID_ARG;
    if (!n && !r_out) return IABN_ERR_INVALID_ARG;
    if (n) IABN_TRY(check_rows(tn));
    IABN_TRY(check_vec(post_stats));
    IABN_TRY(check_vec(pre_stats));
    IABN_TRY(check_codes_opt(codes_b, exps_b));
    IABN_TRY(check_codes_opt(codes_n, exps_n));
    if ((codes_b && !b) || (codes_n && !n)) return IABN_ERR_INVALID_ARG;
    const Rows tensors[] = {to, tn};
    const Rows kept[] = {vector_row(post_stats, 2 * T), vector_row(pre_stats, 2 * T),
                         code_rows(codes_b, T, C), exp_rows(exps_b, T, C),
                         code_rows(codes_n, T, C), exp_rows(exps_n, T, C)};
    const Rows ins[] = {tr, tb, gate_tensor(l)};
    const Rows vectors[] = {vector_row(l->post_weight, C), vector_row(l->post_bias, C),
                            vector_row(l->pre_weight, C), vector_row(l->pre_bias, C)};
    IABN_TRY(check_apart(to, tn));
    IABN_TRY(check_distinct(kept));
    IABN_TRY(check_outs(tensors, ins));
    IABN_TRY(check_all_apart(tensors, vectors));
    IABN_TRY(check_all_apart(kept, tensors));
    IABN_TRY(check_all_apart(kept, ins));
    IABN_TRY(check_all_apart(kept, vectors));
    ResnormFwd a{};
    a.r = r; a.b = b; a.r_out = r_out; a.n = n;
    a.ldr = ldr; a.ldb = ldb; a.ldro = ldr_out; a.ldn = ldn;
    a.post_w = l->post_weight; a.post_b = l->post_bias;
    a.pre_w = l->pre_weight; a.pre_b = l->pre_bias;
    a.gate = b ? l->gate : nullptr;
    a.gate_f32 = l->gate_dtype == IABN_F32;
    a.R = gate_rows(l);
    a.alpha = l->alpha; a.eps = l->eps;
    a.post = l->post; a.pre = l->pre;
    a.post_stats = post_stats; a.pre_stats = pre_stats;
    a.codes_b = codes_b; a.codes_n = codes_n;
    a.exps_b = exps_b; a.exps_n = exps_n;
    a.T = T; a.C = C;
    launch_resnorm_forward(a, l->dtype, device_cus(), stream);
    return launched();
}

size_t iabn_resnorm_workspace_size(int64_t rows, int64_t cols, int64_t rows_per_gate)
{
    if (check_extents(rows, cols, IABN_F32) != IABN_OK || cols > kResnormMaxC ||
        rows_per_gate < 1)
        return 0;
    if (rows == 0 || cols == 0) return 0;
    // a call without a gate treats all rows as one group, whatever was passed here
    const int64_t cus = device_cus();
    const size_t with = resnorm_workspace_bytes(rows, cols, min64(rows, rows_per_gate), cus);
    const size_t without = resnorm_workspace_bytes(rows, cols, rows, cus);
    return with > without ? with : without;
}

iabn_status iabn_resnorm_backward(const iabn_resnorm* l, const void* dr_out, int64_t lddr_out,
                                  const void* dn, int64_t lddn, const void* r_out,
                                  int64_t ldr_out, const void* b, int64_t ldb,
                                  const int8_t* codes_n, const uint8_t* exps_n,
                                  const int8_t* codes_b, const uint8_t* exps_b,
                                  const float* post_stats, const float* pre_stats, void* dr,
                                  int64_t lddr, void* db, int64_t lddb, float* dpost_weight,
                                  float* dpost_bias, float* dpre_weight, float* dpre_bias,
                                  void* dgate, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream)
{
    IABN_TRY(check_layer(l));
    const int64_t T = l->rows, C = l->cols, es = esize(l->dtype);
    if (C == 0) return IABN_OK;
    const bool post = l->post != IABN_NORM_NONE, pre = l->pre != IABN_NORM_NONE;
    const float* vecs[] = {dpost_weight, dpost_bias, dpre_weight, dpre_bias, post_stats, pre_stats};
    for (const float* v : vecs) IABN_TRY(check_vec(v));
    if (!db && T > 0 && (dpost_weight || dpost_bias || dgate)) return IABN_ERR_INVALID_ARG;
    if ((dpost_weight || dpost_bias) && !post) return IABN_ERR_INVALID_ARG;
    if ((dpre_weight || dpre_bias) && !pre) return IABN_ERR_INVALID_ARG;
    if (dgate && !l->gate) return IABN_ERR_INVALID_ARG;
    if (dgate && !aligned(dgate, size_t(esize(l->gate_dtype)))) return IABN_ERR_MISALIGNED;
    if (dn && !pre) return IABN_ERR_INVALID_ARG;
    const bool need_n = dn != nullptr, need_b = db && (post || dgate);
    const bool codes = codes_n || codes_b;
    if (codes && (r_out || b)) return IABN_ERR_INVALID_ARG;
    const Rows tdo{dr_out, lddr_out, T, C, es}, tdn{dn, lddn, T, C, es},
        tro{r_out, ldr_out, T, C, es}, tb{b, ldb, T, C, es}, tdr{dr, lddr, T, C, es},
        tdb{db, lddb, T, C, es};
    if (T > 0) {
        if (dr_out) IABN_TRY(check_rows(tdo));
        if (dn) IABN_TRY(check_rows(tdn));
        if (dr) IABN_TRY(check_rows(tdr));
        if (db) IABN_TRY(check_rows(tdb));
        if (need_n && !pre_stats) return IABN_ERR_INVALID_ARG;
        if (db && post && !post_stats) return IABN_ERR_INVALID_ARG;
        IABN_TRY(check_codes_opt(codes_n, exps_n));
        IABN_TRY(check_codes_opt(codes_b, exps_b));
        if (need_n && !codes_n && !r_out) return IABN_ERR_INVALID_ARG;
        if (need_b && !codes_b && !b) return IABN_ERR_INVALID_ARG;
        if (r_out) IABN_TRY(check_rows(tro));
        if (b) IABN_TRY(check_rows(tb));
    }
    const int64_t cus = device_cus(), R = gate_rows(l);
    const size_t need = T > 0 ? resnorm_workspace_bytes(T, C, R, cus) : 0;
    IABN_TRY(check_ws(workspace, workspace_bytes, need));
    const Rows saved[] = {tro, tb, code_rows(codes_n, T, C), exp_rows(exps_n, T, C),
                          code_rows(codes_b, T, C), exp_rows(exps_b, T, C),
                          vector_row(post_stats, 2 * T), vector_row(pre_stats, 2 * T)};
    const Rows gate = gate_tensor(l), space = vector_row(need ? workspace : nullptr, int64_t(need), 1);
    const Rows vectors[] = {vector_row(l->post_weight, C), vector_row(l->post_bias, C),
                            vector_row(l->pre_weight, C)};
    const Rows grads[] = {tdr, tdb}, dgates[] = {gate_tensor(l, dgate)};
    const Rows dvectors[] = {vector_row(dpost_weight, C), vector_row(dpost_bias, C),
                             vector_row(dpre_weight, C), vector_row(dpre_bias, C)};
    const Rows outs[] = {tdr, tdb, dgates[0], dvectors[0], dvectors[1], dvectors[2], dvectors[3],
                         space};
    const Rows in[] = {tdo, tdn}, in_gate[] = {tdo, tdn, gate};
    const Rows gate_vectors[] = {gate, vectors[0], vectors[1], vectors[2]};
    IABN_TRY(check_distinct(outs));
    IABN_TRY(check_all_apart(outs, saved));
    IABN_TRY(check_outs(grads, in));
    IABN_TRY(check_all_apart(grads, gate_vectors));
    IABN_TRY(check_outs(dgates, in_gate));
    IABN_TRY(check_all_apart(dgates, vectors));
    IABN_TRY(check_outs(dvectors, vectors));       // finished by a later kernel
    IABN_TRY(check_all_apart(dvectors, in_gate));
    const Rows spaces[] = {space};
    IABN_TRY(check_all_apart(spaces, in_gate));
    IABN_TRY(check_all_apart(spaces, vectors));
    ResnormBwd a{};
    a.dr_out = dr_out; a.dn = dn; a.lddro = lddr_out; a.lddn = lddn;
    a.r_out = r_out; a.b = b; a.ldro = ldr_out; a.ldb = ldb;
    a.codes_n = codes_n; a.codes_b = codes_b; a.exps_n = exps_n; a.exps_b = exps_b;
    a.post_stats = post_stats; a.pre_stats = pre_stats;
    a.post_w = l->post_weight; a.post_b = l->post_bias; a.pre_w = l->pre_weight;
    a.gate = l->gate;
    a.gate_f32 = l->gate_dtype == IABN_F32;
    a.R = R;
    a.alpha = l->alpha;
    a.post = l->post; a.pre = l->pre;
    a.dr = dr; a.db = db; a.lddr = lddr; a.lddb = lddb;
    a.dpost_w = dpost_weight; a.dpost_b = dpost_bias;
    a.dpre_w = dpre_weight; a.dpre_b = dpre_bias;
    a.dgate = T > 0 ? dgate : nullptr;
    a.T = T; a.C = C;
    launch_resnorm_backward(a, l->dtype, cus, workspace, stream);
    return launched();
}

}  // extern "C"
