// C ABI of attention and rotary positions: argument validation (before any HIP call) and
// launches on the caller's stream.  Declared in iabn.h.
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "attn.hpp"
#include "checks.hpp"
#include "iabn.h"

using namespace iabn;

namespace {

// A tensor of heads: extents and strides in bytes, smallest stride first.
struct Strided {
    uintptr_t p;
    int64_t es, n[4], s[4];
    bool empty() const { return n[0] == 0 || n[1] == 0 || n[2] == 0 || n[3] == 0; }
    int64_t span(int64_t below) const          // bytes that dimensions of smaller strides cover
    {
        int64_t e = es;
        for (int i = 0; i < 4; ++i)
            if (n[i] > 1 && s[i] < below) e += (n[i] - 1) * s[i];
        return e;
    }
    int64_t span() const { return span(INT64_MAX); }
    bool divides(int64_t pitch) const          // whether the larger strides are its multiples
    {
        for (int i = 0; i < 4; ++i)
            if (n[i] > 1 && s[i] >= pitch && s[i] % pitch != 0) return false;
        return true;
    }
};

Strided strided(const iabn_heads* t, int64_t B, int64_t R, int64_t H, int64_t D, int64_t es)
{
    Strided x{t ? reinterpret_cast<uintptr_t>(t->data) : 0, es, {D, H, R, B}, {es, 0, 0, 0}};
    if (t) {
        x.s[1] = t->head * es;
        x.s[2] = t->row * es;
        x.s[3] = t->batch * es;
    }
    for (int i = 2; i < 4; ++i)                // by stride
        for (int j = i; j > 1 && x.s[j] < x.s[j - 1]; --j) {
            const int64_t a = x.s[j], b = x.n[j];
            x.s[j] = x.s[j - 1]; x.n[j] = x.n[j - 1];
            x.s[j - 1] = a; x.n[j - 1] = b;
        }
    return x;
}

Strided flat(const void* p, int64_t bytes)
{
    return Strided{reinterpret_cast<uintptr_t>(p), 1, {bytes, 1, 1, 1}, {1, 0, 0, 0}};
}

iabn_status check_heads(const iabn_heads* t, int64_t B, int64_t R, int64_t H, int64_t D, int64_t es)
{
    if (!t || t->batch < 0 || t->row < 0 || t->head < 0) return IABN_ERR_INVALID_ARG;
    const Strided x = strided(t, B, R, H, D, es);
    if (x.empty()) return IABN_OK;
    if (!t->data) return IABN_ERR_INVALID_ARG;
    if (double(B) * double(t->batch) + double(R) * double(t->row) + double(H) * double(t->head) >
        9.0e15)
        return IABN_ERR_UNSUPPORTED;
    return aligned(t->data, size_t(es)) ? IABN_OK : IABN_ERR_MISALIGNED;
}

// An output: no two of its elements in one place.
iabn_status check_heads_out(const iabn_heads* t, int64_t B, int64_t R, int64_t H, int64_t D,
                            int64_t es)
{
    IABN_TRY(check_heads(t, B, R, H, D, es));
    const Strided x = strided(t, B, R, H, D, es);
    int64_t inner = x.n[0] * es;
    for (int i = 1; i < 4; ++i) {
        if (x.n[i] <= 1) continue;
        if (!x.empty() && x.s[i] < inner) return IABN_ERR_INVALID_ARG;
        inner += (x.n[i] - 1) * x.s[i];
    }
    return IABN_OK;
}

// Whether two tensors may share memory.  They do not where their addresses do not meet, or
// where both repeat with one pitch in which they keep to different bytes (slices of a
// buffer).
bool meet(const Strided& a, const Strided& b)
{
    if (!a.p || !b.p || a.empty() || b.empty()) return false;
    if (a.p + uintptr_t(a.span()) <= b.p || b.p + uintptr_t(b.span()) <= a.p) return false;
    for (const Strided* t : {&a, &b})
        for (int i = 0; i < 4; ++i) {
            const int64_t pitch = t->s[i];
            if (t->n[i] <= 1 || pitch == 0 || !a.divides(pitch) || !b.divides(pitch)) continue;
            const int64_t ea = a.span(pitch), eb = b.span(pitch);
            const uintptr_t d = b.p >= a.p ? (b.p - a.p) % uintptr_t(pitch)
                                           : (uintptr_t(pitch) - (a.p - b.p) % uintptr_t(pitch)) %
                                                 uintptr_t(pitch);
            if (int64_t(d) >= ea && pitch - int64_t(d) >= eb) return false;
        }
    return true;
}

bool same(const iabn_heads* a, const iabn_heads* b, int64_t B, int64_t R, int64_t H)
{
    return a->data == b->data && (B <= 1 || a->batch == b->batch) &&
           (R <= 1 || a->row == b->row) && (H <= 1 || a->head == b->head);
}

Heads heads_of(const iabn_heads* t)
{
    return t ? Heads{static_cast<char*>(t->data), t->batch, t->row, t->head} : Heads{};
}

iabn_status check_problem(const iabn_attention* p)
{
    if (!p || !dtype_ok(p->dtype)) return IABN_ERR_INVALID_ARG;
    if (p->batch < 0 || p->heads < 0 || p->kv_heads < 0 || p->q_len < 0 || p->k_len < 0 ||
        p->head_dim < 1)
        return IABN_ERR_INVALID_ARG;
    if (p->heads > 0 && (p->kv_heads == 0 || p->heads % p->kv_heads != 0)) return IABN_ERR_INVALID_ARG;
    if (p->heads == 0 && p->kv_heads != 0) return IABN_ERR_INVALID_ARG;
    if (!(p->scale > 0.f) || !isfinite(p->scale * 1.442695f)) return IABN_ERR_INVALID_ARG;
    if ((p->q_starts && p->q_lens) || (p->k_starts && p->k_lens)) return IABN_ERR_INVALID_ARG;
    if ((p->q_starts && p->q_rows < 0) || (p->k_starts && p->k_rows < 0)) return IABN_ERR_INVALID_ARG;
    for (const int32_t* v : {p->q_starts, p->k_starts, p->q_lens, p->k_lens})
        if (!aligned(v, 4)) return IABN_ERR_MISALIGNED;
    if (p->head_dim % 8 != 0 || p->head_dim > kAttnMaxD) return IABN_ERR_UNSUPPORTED;
    if (p->q_len > kAttnMaxLen || p->k_len > kAttnMaxLen) return IABN_ERR_UNSUPPORTED;
    if (p->heads > 0) {
        const double group = double(p->heads / p->kv_heads), most = double(kAttnMaxLen);
        const double rows = double(p->q_len) * group, keys = double(p->k_len) * group;
        if (rows > most || keys > most) return IABN_ERR_UNSUPPORTED;
        // threads of a launch, two for a row or a key and a workgroup's for a head, in 32 bits
        const double heads = double(p->batch) * double(p->kv_heads);
        if (heads * (2. * (rows > p->k_len ? rows : double(p->k_len)) + 256.) > 4294967295.)
            return IABN_ERR_UNSUPPORTED;
    }
    if ((p->q_starts && p->q_rows > kMaxExtent) || (p->k_starts && p->k_rows > kMaxExtent))
        return IABN_ERR_UNSUPPORTED;
    return IABN_OK;
}

AttnArgs attn_args(const iabn_attention* p)
{
    AttnArgs a{};
    a.B = int(p->batch);
    a.KV = int(p->kv_heads);
    a.G = int(p->kv_heads > 0 ? p->heads / p->kv_heads : 1);
    a.D = int(p->head_dim);
    a.Sq = int(p->q_len);
    a.Sk = int(p->k_len);
    a.q_rows = p->q_rows;
    a.k_rows = p->k_rows;
    a.q_starts = p->q_starts;
    a.k_starts = p->k_starts;
    a.q_lens = p->q_lens;
    a.k_lens = p->k_lens;
    a.left = int(p->left < 0 ? kAttnMaxLen : min64(p->left, kAttnMaxLen));
    a.right = int(p->right < 0 ? kAttnMaxLen : min64(p->right, kAttnMaxLen));
    a.scale = p->scale;
    a.c = p->scale * 1.44269504088896341f;
    a.group = make_fast_div(uint32_t(a.G));
    return a;
}

// The tensors of a problem: (batch, rows) of the queries' side and of the keys'.
struct Sides {
    int64_t qb, qr, kb, kr;
};

Sides sides(const iabn_attention* p)
{
    Sides s{p->batch, p->q_len, p->batch, p->k_len};
    if (p->q_starts) {
        s.qb = 1;
        s.qr = p->q_rows;
    }
    if (p->k_starts) {
        s.kb = 1;
        s.kr = p->k_rows;
    }
    return s;
}

Strided lse_tensor(const iabn_attention* p, const Sides& s, const float* lse)
{
    return flat(lse, s.qb * s.qr * p->heads * 4);
}

// Outputs against what the call reads, and against one another.
template <size_t N, size_t M>
iabn_status check_apart(const Strided (&outs)[N], const Strided (&ins)[M])
{
    for (size_t i = 0; i < N; ++i) {
        for (const Strided& t : ins)
            if (meet(outs[i], t)) return IABN_ERR_INVALID_ARG;
        for (size_t j = 0; j < i; ++j)
            if (meet(outs[i], outs[j])) return IABN_ERR_INVALID_ARG;
    }
    return IABN_OK;
}

Strided vector_of(const iabn_attention* p, const int32_t* v, int64_t more)
{
    return flat(v, (p->batch + more) * 4);
}

}  // namespace

extern "C" {

size_t iabn_attention_workspace_size(const iabn_attention* p, int backward)
{
    if (check_problem(p) != IABN_OK || p->batch == 0 || p->heads == 0 || p->q_len == 0) return 0;
    const AttnArgs a = attn_args(p);
    return backward ? attn_bwd_workspace_bytes(a, device_cus())
                    : attn_fwd_workspace_bytes(a, p->dtype, device_cus());
}

iabn_status iabn_attention_forward(const iabn_attention* p, const iabn_heads* q,
                                   const iabn_heads* k, const iabn_heads* v,
                                   const iabn_heads* out, float* lse, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream)
{
    IABN_TRY(check_problem(p));
    if (p->batch == 0 || p->heads == 0 || p->q_len == 0) return IABN_OK;
    const int64_t es = esize(p->dtype), D = p->head_dim, H = p->heads, KV = p->kv_heads;
    const Sides s = sides(p);
    IABN_TRY(check_heads(q, s.qb, s.qr, H, D, es));
    IABN_TRY(check_heads(k, s.kb, s.kr, KV, D, es));
    IABN_TRY(check_heads(v, s.kb, s.kr, KV, D, es));
    IABN_TRY(check_heads_out(out, s.qb, s.qr, H, D, es));
    if (!aligned(lse, 4)) return IABN_ERR_MISALIGNED;
    AttnArgs a = attn_args(p);
    const int64_t cus = device_cus();
    const size_t need = attn_fwd_workspace_bytes(a, p->dtype, cus);
    IABN_TRY(check_ws(workspace, workspace_bytes, need));
    const Strided outs[] = {strided(out, s.qb, s.qr, H, D, es), lse_tensor(p, s, lse),
                            flat(need ? workspace : nullptr, int64_t(need))};
    const Strided ins[] = {strided(q, s.qb, s.qr, H, D, es), strided(k, s.kb, s.kr, KV, D, es),
                           strided(v, s.kb, s.kr, KV, D, es), vector_of(p, p->q_starts, 1),
                           vector_of(p, p->k_starts, 1), vector_of(p, p->q_lens, 0),
                           vector_of(p, p->k_lens, 0)};
    IABN_TRY(check_apart(outs, ins));
    a.q = heads_of(q);
    a.k = heads_of(k);
    a.v = heads_of(v);
    a.out = heads_of(out);
    a.lse = lse;
    launch_attn_forward(a, p->dtype, cus, workspace, stream);
    return launched();
}

iabn_status iabn_attention_backward(const iabn_attention* p, const iabn_heads* q,
                                    const iabn_heads* k, const iabn_heads* v,
                                    const iabn_heads* out, const float* lse,
                                    const iabn_heads* dout, const iabn_heads* dq,
                                    const iabn_heads* dk, const iabn_heads* dv, void* workspace,
                                    size_t workspace_bytes, hipStream_t stream)
{
    IABN_TRY(check_problem(p));
    if (p->batch == 0 || p->heads == 0) return IABN_OK;
    const int64_t es = esize(p->dtype), D = p->head_dim, H = p->heads, KV = p->kv_heads;
    const Sides s = sides(p);
    IABN_TRY(check_heads(q, s.qb, s.qr, H, D, es));
    IABN_TRY(check_heads(k, s.kb, s.kr, KV, D, es));
    IABN_TRY(check_heads(v, s.kb, s.kr, KV, D, es));
    IABN_TRY(check_heads(out, s.qb, s.qr, H, D, es));
    IABN_TRY(check_heads(dout, s.qb, s.qr, H, D, es));
    IABN_TRY(check_heads_out(dq, s.qb, s.qr, H, D, es));
    IABN_TRY(check_heads_out(dk, s.kb, s.kr, KV, D, es));
    IABN_TRY(check_heads_out(dv, s.kb, s.kr, KV, D, es));
    if (!lse && p->q_len > 0 && s.qr > 0) return IABN_ERR_INVALID_ARG;
    if (!aligned(lse, 4)) return IABN_ERR_MISALIGNED;
    AttnArgs a = attn_args(p);
    const int64_t cus = device_cus();
    const size_t need = p->q_len > 0 ? attn_bwd_workspace_bytes(a, cus) : 0;
    IABN_TRY(check_ws(workspace, workspace_bytes, need));
    const Strided outs[] = {strided(dq, s.qb, s.qr, H, D, es), strided(dk, s.kb, s.kr, KV, D, es),
                            strided(dv, s.kb, s.kr, KV, D, es),
                            flat(need ? workspace : nullptr, int64_t(need))};
    const Strided ins[] = {strided(q, s.qb, s.qr, H, D, es),
                           strided(k, s.kb, s.kr, KV, D, es),
                           strided(v, s.kb, s.kr, KV, D, es),
                           strided(out, s.qb, s.qr, H, D, es),
                           strided(dout, s.qb, s.qr, H, D, es),
                           lse_tensor(p, s, lse),
                           vector_of(p, p->q_starts, 1), vector_of(p, p->k_starts, 1),
                           vector_of(p, p->q_lens, 0), vector_of(p, p->k_lens, 0)};
    IABN_TRY(check_apart(outs, ins));
    a.q = heads_of(q);
    a.k = heads_of(k);
    a.v = heads_of(v);
    a.out = heads_of(out);
    a.lse = const_cast<float*>(lse);
    const AttnGrads g{heads_of(dout), heads_of(dq), heads_of(dk), heads_of(dv)};
    launch_attn_backward(a, g, p->dtype, cus, workspace, stream);
    return launched();
}

iabn_status iabn_rotary(const iabn_rotary_spec* r, const iabn_heads* q, int64_t q_heads,
                        const iabn_heads* q_out, const iabn_heads* k, int64_t k_heads,
                        const iabn_heads* k_out, int inverse, hipStream_t stream)
{
    if (!r || !dtype_ok(r->dtype)) return IABN_ERR_INVALID_ARG;
    if (r->batch < 0 || r->rows < 0 || q_heads < 0 || k_heads < 0 || r->pairs < 1 || r->axes < 1)
        return IABN_ERR_INVALID_ARG;
    if (r->head_dim < 2 * r->pairs || r->pos_batch < 0 || r->pos_row < 0) return IABN_ERR_INVALID_ARG;
    if (r->pos_type != IABN_POS_I32 && r->pos_type != IABN_POS_I64 && r->pos_type != IABN_POS_F32)
        return IABN_ERR_INVALID_ARG;
    if (r->head_dim > 65536 || r->axes > 65536 || q_heads + k_heads > 65536)
        return IABN_ERR_UNSUPPORTED;
    if (r->rows >= (int64_t(1) << 30) || double(r->batch) * double(r->rows) > 2147483647. * 4.)
        return IABN_ERR_UNSUPPORTED;
    if (r->batch == 0 || r->rows == 0 || q_heads + k_heads == 0) return IABN_OK;
    const int64_t es = esize(r->dtype), D = r->head_dim, B = r->batch, S = r->rows;
    if (q_heads > 0) {
        IABN_TRY(check_heads(q, B, S, q_heads, D, es));
        IABN_TRY(check_heads_out(q_out, B, S, q_heads, D, es));
    }
    if (k_heads > 0) {
        IABN_TRY(check_heads(k, B, S, k_heads, D, es));
        IABN_TRY(check_heads_out(k_out, B, S, k_heads, D, es));
    }
    if (!r->inv_freq || !r->positions) return IABN_ERR_INVALID_ARG;
    const size_t pos_size = r->pos_type == IABN_POS_I64 ? 8 : 4;
    if (!aligned(r->inv_freq, 8) || !aligned(r->axis, 4) || !aligned(r->positions, pos_size))
        return IABN_ERR_MISALIGNED;
    if (double(B) * double(r->pos_batch) + double(S) * double(r->pos_row) > 9.0e15)
        return IABN_ERR_UNSUPPORTED;
    const Strided qi = strided(q_heads ? q : nullptr, B, S, q_heads, D, es),
                  qo = strided(q_heads ? q_out : nullptr, B, S, q_heads, D, es),
                  ki = strided(k_heads ? k : nullptr, B, S, k_heads, D, es),
                  ko = strided(k_heads ? k_out : nullptr, B, S, k_heads, D, es);
    const Strided pos = flat(r->positions, ((B - 1) * r->pos_batch + (S - 1) * r->pos_row + r->axes) *
                                               int64_t(pos_size));
    const Strided tables[] = {flat(r->inv_freq, r->pairs * 8), flat(r->axis, r->pairs * 4), pos};
    for (const Strided& o : {qo, ko})
        for (const Strided& t : tables)
            if (meet(o, t)) return IABN_ERR_INVALID_ARG;
    if (meet(qo, ko) || meet(qo, ki) || meet(ko, qi)) return IABN_ERR_INVALID_ARG;
    if (meet(qo, qi) && !same(q, q_out, B, S, q_heads)) return IABN_ERR_INVALID_ARG;
    if (meet(ko, ki) && !same(k, k_out, B, S, k_heads)) return IABN_ERR_INVALID_ARG;
    RotaryArgs a{};
    a.heads[0] = int(q_heads);
    a.heads[1] = int(k_heads);
    if (q_heads > 0) {
        a.x[0] = heads_of(q);
        a.y[0] = heads_of(q_out);
    }
    if (k_heads > 0) {
        a.x[1] = heads_of(k);
        a.y[1] = heads_of(k_out);
    }
    a.B = B;
    a.S = S;
    a.D = int(D);
    a.pairs = int(r->pairs);
    a.axes = int(r->axes);
    a.interleaved = r->interleaved != 0;
    a.pos_type = r->pos_type;
    a.inv_freq = r->inv_freq;
    a.axis = r->axis;
    a.positions = r->positions;
    a.pos_batch = r->pos_batch;
    a.pos_row = r->pos_row;
    a.sign = inverse ? -1.f : 1.f;
    launch_rotary(a, r->dtype, device_cus(), stream);
    return launched();
}

}  // extern "C"
