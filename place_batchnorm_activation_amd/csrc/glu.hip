// Gated activations whose inputs are kept in 8 bits.
//
//   forward    out = act(g) * u (without u: act(g)), from the tensors themselves,
//              and the codes of g and u for the backward
//   backward   with g', u' the decoded codes:
//              dg = dout * u' * act'(g'), du = dout * act(g'),
//              and, where asked for, out' = act(g') * u', the next layer's input
//              for its own gradient (so that out need not be kept)
//
// act: SiLU x*s(x), s(x) = 1/(1 + e^-x), with slope s*(1 + x*(1 - s));
//      GELU x*P(x), P the normal distribution, with slope P + x*p(x), p its density;
//      GELU by tanh: x*(1 + t)/2 = x*s(2w) with w = k*(x + 0.044715*x^3),
//      k = sqrt(2/pi), because (1 + tanh w)/2 = s(2w); slope s + x*s*(1 - s)*2w'.
//
// The forward uses the tensors and not their codes, so that keeping codes changes
// no output of the network; only gradients see the 8 bits.  One pass over the
// data, eight columns a thread, no reduction beyond the quad's largest magnitude.
#include <hip/hip_runtime.h>

#include "acts.hpp"
#include "block.hpp"
#include "rows.hpp"

namespace iabn {

namespace {

template <int DT, int ACT, bool WHOLE>
__global__ __launch_bounds__(kThreads) void k_glu_fwd(GluFwd a, int64_t row0, uint32_t nvec,
                                                      uint32_t vpr, FastDiv dv, int F)
{
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= nvec) return;
    const uint32_t r = fast_div(i, dv);
    const int64_t row = row0 + r;
    const uint32_t c = (i - r * vpr) * kRowV, Fp = vpr * kRowV;
    float g[8], u[8];
    const Raw8<DT> rg = load8<DT, WHOLE, uint64_t>(row_ptr<DT>(a.gate, row, a.ldg), c, F);
    if (a.up) {
        const Raw8<DT> ru = load8<DT, WHOLE, uint64_t>(row_ptr<DT>(a.up, row, a.ldu), c, F);
        widen8<DT>(ru, u);
    }
    widen8<DT>(rg, g);
    uint32_t E;
    if (a.codes_g) {
        const uint2 q = encode8(g, E);
        store_codes(a.codes_g + row * Fp, a.exps_g + row * (Fp / kGroup), Fp, c, q, E);
        if (a.up) {
            const uint2 p = encode8(u, E);
            store_codes(a.codes_u + row * Fp, a.exps_u + row * (Fp / kGroup), Fp, c, p, E);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float f, d;
        glu_act<ACT>(g[e], f, d);
        g[e] = a.up ? f * u[e] : f;
    }
    store8<DT, WHOLE, uint64_t>(row_ptr<DT>(a.out, row, a.ldo), c, F, g);
}

template <int DT, int ACT, bool WHOLE>
__global__ __launch_bounds__(kThreads) void k_glu_bwd(GluBwd a, int64_t row0, uint32_t nvec,
                                                      uint32_t vpr, FastDiv dv, int F)
{
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= nvec) return;
    const uint32_t r = fast_div(i, dv);
    const int64_t row = row0 + r;
    const uint32_t c = (i - r * vpr) * kRowV, Fp = vpr * kRowV;
    if (c >= uint32_t(F)) return;
    const Raw8<DT> ro = load8<DT, WHOLE, uint64_t>(row_ptr<DT>(a.dout, row, a.lddo), c, F);
    float g[8], u[8], o[8];
    decode8(*reinterpret_cast<const uint2*>(a.codes_g + row * Fp + c),
            a.exps_g[row * (Fp / kGroup) + c / kGroup], g);
    if (a.codes_u)
        decode8(*reinterpret_cast<const uint2*>(a.codes_u + row * Fp + c),
                a.exps_u[row * (Fp / kGroup) + c / kGroup], u);
    widen8<DT>(ro, o);
    float dg[8], du[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float f, d;
        glu_act<ACT>(g[e], f, d);
        du[e] = o[e] * f;
        dg[e] = a.codes_u ? o[e] * u[e] * d : o[e] * d;
        o[e] = a.codes_u ? f * u[e] : f;
    }
    store8<DT, WHOLE, uint64_t>(row_ptr<DT>(a.dgate, row, a.lddg), c, F, dg);
    if (a.codes_u) store8<DT, WHOLE, uint64_t>(row_ptr<DT>(a.dup, row, a.lddu), c, F, du);
    if (a.out) store8<DT, WHOLE, uint64_t>(row_ptr<DT>(a.out, row, a.ldo), c, F, o);
}

template <class F>
void with_glu_act(int act, F&& f)
{
    switch (act) {
    case kSilu: f(std::integral_constant<int, kSilu>{}); break;
    case kGelu: f(std::integral_constant<int, kGelu>{}); break;
    default: f(std::integral_constant<int, kGeluTanh>{}); break;
    }
}

}  // namespace

void launch_glu_forward(const GluFwd& a, int64_t T, int64_t F, int dtype, int act, hipStream_t s)
{
    const int64_t vpr = code_pitch(F) / kRowV;
    const FastDiv dv = make_fast_div(uint32_t(vpr));
    with_dtype(dtype, [&](auto d) {
        with_glu_act(act, [&](auto ac) { with_whole(F, [&](auto whole) {
            each_row_block(T, vpr, kThreads, [&](int64_t row0, uint32_t nvec, dim3 grid) {
                hipLaunchKernelGGL((k_glu_fwd<decltype(d)::value, decltype(ac)::value, decltype(whole)::value>), grid,
                                   dim3(kThreads), 0, s, a, row0, nvec, uint32_t(vpr), dv, int(F));
            });
        }); });
    });
}

void launch_glu_backward(const GluBwd& a, int64_t T, int64_t F, int dtype, int act, hipStream_t s)
{
    const int64_t vpr = code_pitch(F) / kRowV;
    const FastDiv dv = make_fast_div(uint32_t(vpr));
    with_dtype(dtype, [&](auto d) {
        with_glu_act(act, [&](auto ac) { with_whole(F, [&](auto whole) {
            each_row_block(T, vpr, kThreads, [&](int64_t row0, uint32_t nvec, dim3 grid) {
                hipLaunchKernelGGL((k_glu_bwd<decltype(d)::value, decltype(ac)::value, decltype(whole)::value>), grid,
                                   dim3(kThreads), 0, s, a, row0, nvec, uint32_t(vpr), dv, int(F));
            });
        }); });
    });
}

}  // namespace iabn
