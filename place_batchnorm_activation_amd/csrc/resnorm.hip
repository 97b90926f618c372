// The boundary between two residual blocks: post-norm of the block's output, its
// gate and residual scale, the residual sum, and the next block's pre-norm.
//
//   forward, a row of C columns:
//     p = post(b),  r' = r + alpha * g * p,  n = pre(r')
//     norm(x) = xhat * w + beta,  xhat = (x - mean) * rstd; RMS norms take mean 0,
//     rstd = 1/sqrt(mean((x - mean)^2) + eps)
//   backward, from dr' and dn, with <.> the mean over the row:
//     q  = dn * w_pre
//     D  = dr' + rstd_pre * (q - [<q>] - xn * <q xn>)           = dr
//     dz = alpha * D,  dg = sum dz * p,  h = g * dz * w_post
//     db = rstd_post * (h - [<h>] - xb * <h xb>)                [layer norms only]
//     dw_pre = sum dn * xn, dbeta_pre = sum dn, dw_post = sum g dz xb, dbeta_post = sum g dz
//   xn, xb come from the stored tensors and their statistics, or from 8-bit codes of
//   xn and xb themselves (rows.hpp), which stand in for both tensors.
//
// The work is a few operations an element on 8 to 12 bytes of traffic: HBM bounds
// it, so each kernel reads every tensor once and holds the row in registers across
// its reductions.  n is formed from the unrounded r'.  Statistics, sums and
// gradients of the vectors are fp32 (two passes over the registers for a layer
// norm's variance, so that no digits cancel); the sums over row blocks are finished
// in fp64, in a fixed order.
#include <hip/hip_runtime.h>

#include "block.hpp"
#include "rows.hpp"

namespace iabn {

namespace {

// Sum over the wave, in every lane: shifts within rows of 16 lanes, then broadcasts of
// a row's last lane into the next ones; lane 63 ends with the total.
__device__ __forceinline__ float wave_total(float v)
{
    auto step = [&](auto ctrl, auto rows) {
        v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v),
                                                         decltype(ctrl)::value,
                                                         decltype(rows)::value, 0xF, false));
    };
    using std::integral_constant;
    step(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});   // row_shr:1
    step(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});   // row_shr:2
    step(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});   // row_shr:4
    step(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});   // row_shr:8
    step(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});   // row_bcast:15
    step(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});   // row_bcast:31
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}

// Sums over the TPR threads that hold a row.  Wider rows exchange wave totals
// through `slots` (kSlots x 2 x waves floats): consecutive calls take consecutive
// slots, so that one barrier a call suffices.
constexpr int kSlots = 4;

template <int TPR>
struct RowSum {
    static constexpr int kWaves = TPR / kWave;
    float (*slots)[2][kWaves];
    int at = 0;

    template <int N>
    __device__ __forceinline__ void add(float (&v)[N])
    {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = wave_total(v[k]);
        if constexpr (kWaves > 1) {
            float (*s)[kWaves] = slots[at];
            at = (at + 1) % kSlots;
            const int w = threadIdx.x / kWave;
            if (threadIdx.x % kWave == 0) {
#pragma unroll
                for (int k = 0; k < N; ++k) s[k][w] = v[k];
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < N; ++k) {
                v[k] = 0.f;
#pragma unroll
                for (int i = 0; i < kWaves; ++i) v[k] += s[k][i];
            }
        }
    }
    __device__ __forceinline__ void operator()(float& a, float& b)
    {
        float v[2] = {a, b};
        add(v);
        a = v[0];
        b = v[1];
    }
    __device__ __forceinline__ void operator()(float& a)
    {
        float v[1] = {a};
        add(v);
        a = v[0];
    }
};

// xhat of a row held as NV vectors a thread, in place, and its statistics.
template <int NV, class SUM>
__device__ __forceinline__ void normalise(float (&x)[NV][8], const int (&col)[NV], int C, bool layer,
                                          float inv_c, float eps, SUM& sum, float& mean,
                                          float& rstd)
{
    mean = 0.f;
    if (layer) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) mean += x[k][e];
        sum(mean);
        mean *= inv_c;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] = col[k] + e < C ? x[k][e] - mean : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(x[k][e], x[k][e], s);
    sum(s);
    rstd = 1.f / sqrtf(fmaf(s, inv_c, eps));
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] *= rstd;
}

// A thread's eight columns of a row of C >= 8 columns: those at `at`, which for the last
// vector of a ragged row begin `skip` columns early, so that every access of the row is
// one wide one inside it.  The skipped columns belong to the thread before: they are kept
// out of sums (mask) and are not written.  Threads past the row (in == false) read its
// last columns and own none.
struct Span {
    uint32_t c, at, skip;
    bool in;
    __device__ __forceinline__ Span(uint32_t thread, int C)
        : c(thread * kRowV), in(c < uint32_t(C))
    {
        const uint32_t last = uint32_t(C) - kRowV;
        at = c < last ? c : last;
        skip = in ? c - at : 0u;
    }
    __device__ __forceinline__ bool own(int e) const { return in && uint32_t(e) >= skip; }
    // zero where not owned, by selection: the columns read twice may hold an infinity
    __device__ __forceinline__ void mask(bool ragged, float (&v)[8]) const
    {
        if (ragged || !in) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = own(e) ? v[e] : 0.f;
        }
    }
    template <int DT>
    __device__ __forceinline__ Raw8<DT> load(const char* row) const
    {
        Raw8<DT> r;
#pragma unroll
        for (int h = 0; h < (DT == kF32 ? 2 : 1); ++h)
            r.q[h] = load16_any(row + at * (DT == kF32 ? 4 : 2) + 16 * h);
        return r;
    }
    template <int DT>
    __device__ __forceinline__ void store(const char* row, const float (&v)[8]) const
    {
        if (!in) return;
        if (skip == 0) {
            store8<DT, true>(row, at, int(at) + kRowV, v);
        } else {
#pragma unroll
            for (int e = 1; e < 8; ++e)
                if (uint32_t(e) >= skip) {
                    char* p = const_cast<char*>(row) + (at + e) * (DT == kF32 ? 4 : 2);
                    if constexpr (DT == kF32) *reinterpret_cast<float*>(p) = v[e];
                    else *reinterpret_cast<uint16_t*>(p) = pack1<DT>(v[e]);
                }
        }
    }
    // of a per-column vector (null: `none`), zero where not owned
    __device__ __forceinline__ void cols(const float* p, float none, float (&v)[8]) const
    {
        if (p) {
            widen8<kF32>(load<kF32>(reinterpret_cast<const char*>(p)), v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = none;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = own(e) ? v[e] : 0.f;
    }
    // of a gate row (1 without a gate)
    template <int DT>
    __device__ __forceinline__ void gate(const void* g, bool f32, int64_t grow, int64_t C,
                                         float (&v)[8]) const
    {
        if (!g) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 1.f;
        } else if (f32) widen8<kF32>(load<kF32>(row_ptr<kF32>(g, grow, C)), v);
        else widen8<DT>(load<DT>(row_ptr<DT>(g, grow, C)), v);
    }
    // codes lie by whole vectors, at c
    __device__ __forceinline__ uint2 load_codes(const int8_t* row) const
    {
        const uint64_t q = *reinterpret_cast<const uint64_t*>(row + (in ? c : 0u)) << (8 * skip);
        return make_uint2(uint32_t(q), uint32_t(q >> 32));
    }
};

// Eight gate values of gate row `grow` (1 without a gate).
template <int DT, bool WHOLE>
__device__ __forceinline__ void load_gate(const void* gate, bool f32, int64_t grow, int64_t C,
                                          uint32_t c, float (&g)[8])
{
    if (!gate) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 1.f;
    } else if (f32) widen8<kF32>(load8<kF32, WHOLE>(row_ptr<kF32>(gate, grow, C), c, int(C)), g);
    else widen8<DT>(load8<DT, WHOLE>(row_ptr<DT>(gate, grow, C), c, int(C)), g);
}

// TPR threads a row, NV vectors a thread.
template <int DT, int TPR, int NV, bool WHOLE>
__global__ __launch_bounds__((TPR > kThreads ? TPR : kThreads)) void k_resnorm_fwd(ResnormFwd a,
                                                                                   FastDiv dr)
{
    constexpr int NT = TPR > kThreads ? TPR : kThreads;
    constexpr int RPW = NT / TPR;                     // rows a workgroup holds
    __shared__ float slots[kSlots][2][TPR / kWave];
    RowSum<TPR> sum{slots};
    const int t = threadIdx.x % TPR;
    const int C = int(a.C);
    const float inv_c = 1.f / float(a.C);
    const int64_t Cp = code_pitch(a.C);
    int col[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        col[k] = (t + k * TPR) * kRowV;
    }
    const int64_t step = int64_t(gridDim.x) * RPW;
    // uniform over a wave (and a barrier's workgroup)
    const int sub = RPW > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / TPR) : 0;
    for (int64_t row = int64_t(blockIdx.x) * RPW + sub; row < a.T; row += step) {
#pragma unroll
        for (int k = 0; k < NV; ++k) asm volatile("" : "+v"(col[k]));    // as in the backward
        Raw8<DT> rr[NV];
        float x[NV][8];
#pragma unroll
        for (int k = 0; k < NV; ++k) rr[k] = load8<DT, WHOLE>(row_ptr<DT>(a.r, row, a.ldr), col[k], C);
        float mean, rstd;
        if (a.b) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                widen8<DT>(load8<DT, WHOLE>(row_ptr<DT>(a.b, row, a.ldb), col[k], C), x[k]);
            if (a.post != kNormNone) {
                normalise<NV>(x, col, C, a.post == kNormLayer, inv_c, a.eps, sum, mean, rstd);
                if (a.post_stats && t == 0) {
                    a.post_stats[2 * row] = mean;
                    a.post_stats[2 * row + 1] = rstd;
                }
            }
            const int64_t grow = a.gate ? fast_div(uint32_t(row), dr) : 0;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (a.codes_b) {
                    uint32_t E;
                    const uint2 q = encode8(x[k], E);
                    store_codes(a.codes_b + row * Cp, a.exps_b + row * (Cp / kGroup), Cp,
                                col[k], q, E);
                }
                float v[8];
                if (a.post != kNormNone) {
                    float w[8], o[8];
                    load_cols<WHOLE>(a.post_w, col[k], C, 1.f, w);
                    load_cols<WHOLE>(a.post_b, col[k], C, 0.f, o);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[k][e] = fmaf(x[k][e], w[e], o[e]);
                }
                if (a.gate) {
                    float g[8];
                    load_gate<DT, WHOLE>(a.gate, a.gate_f32, grow, a.C, col[k], g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[k][e] *= g[e];
                }
                widen8<DT>(rr[k], v);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[k][e] = fmaf(a.alpha, x[k][e], v[e]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < NV; ++k) widen8<DT>(rr[k], x[k]);
        }
        if (a.r_out) {
#pragma unroll
            for (int k = 0; k < NV; ++k) store8<DT, WHOLE>(row_ptr<DT>(a.r_out, row, a.ldro), col[k], C, x[k]);
        }
        if (a.pre == kNormNone) continue;
        normalise<NV>(x, col, C, a.pre == kNormLayer, inv_c, a.eps, sum, mean, rstd);
        if (a.pre_stats && t == 0) {
            a.pre_stats[2 * row] = mean;
            a.pre_stats[2 * row + 1] = rstd;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (a.codes_n) {
                uint32_t E;
                const uint2 q = encode8(x[k], E);
                store_codes(a.codes_n + row * Cp, a.exps_n + row * (Cp / kGroup), Cp,
                                col[k], q, E);
            }
            float w[8], o[8];
            load_cols<WHOLE>(a.pre_w, col[k], C, 1.f, w);
            load_cols<WHOLE>(a.pre_b, col[k], C, 0.f, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] = fmaf(x[k][e], w[e], o[e]);
            store8<DT, WHOLE>(row_ptr<DT>(a.n, row, a.ldn), col[k], C, x[k]);
        }
    }
}

// The same for rows of 8 to 4096 columns, one vector a thread: the vectors that all rows
// use stay in registers (a gate for some of the rows is read with them), and r and b of the
// next row are in flight over this one's reductions.  Rows go to workgroups in turn, 16 waves a
// CU (32 measure the same).  16384 x 4096 bf16: 104 us, 5.2 TB/s; with both codes 146 us; one
// row of 4096: 3.8 us.
template <int DT, int TPR>
__global__ __launch_bounds__(TPR == kWave ? kThreads : TPR) void k_resnorm_fwd_row(ResnormFwd a,
                                                                                  FastDiv dr)
{
    constexpr int NT = TPR == kWave ? kThreads : TPR, RPW = NT / TPR;
    __shared__ float slots[kSlots][2][TPR / kWave];
    RowSum<TPR> sum{slots};
    const int C = int(a.C);
    const float inv_c = 1.f / float(C);
    const int64_t Cp = code_pitch(a.C);
    const bool ragged = C % kRowV != 0, post = a.post != kNormNone, pre = a.pre != kNormNone;
    Span span(threadIdx.x % TPR, C);
    // uniform over a wave (and a barrier's workgroup)
    const int sub = RPW > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / TPR) : 0;
    const int64_t step = int64_t(gridDim.x) * RPW;
    int64_t row = int64_t(blockIdx.x) * RPW + sub;
    if (row >= a.T) return;                 // RPW == 1: whole workgroups; else single waves

    float w_b[8], o_b[8], w_n[8], o_n[8];
    if (post) {
        span.cols(a.post_w, 1.f, w_b);
        span.cols(a.post_b, 0.f, o_b);
    }
    if (pre) {
        span.cols(a.pre_w, 1.f, w_n);
        span.cols(a.pre_b, 0.f, o_n);
    }
    Raw8<DT> rr, rb{};
    auto load = [&](int64_t i) {
        rr = span.load<DT>(row_ptr<DT>(a.r, i, a.ldr));
        if (a.b) rb = span.load<DT>(row_ptr<DT>(a.b, i, a.ldb));
    };
    auto normed = [&](float (&x)[8], bool layer, float* stats) {
        float mean = 0.f;
        span.mask(ragged, x);
        if (layer) {
#pragma unroll
            for (int e = 0; e < 8; ++e) mean += x[e];
            sum(mean);
            mean *= inv_c;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] -= mean;
            span.mask(ragged, x);
        }
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
        sum(s);
        const float rstd = 1.f / sqrtf(fmaf(s, inv_c, a.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= rstd;
        if (stats && threadIdx.x % TPR == 0) {
            stats[2 * row] = mean;
            stats[2 * row + 1] = rstd;
        }
    };
    // codes of eight values that are zero where not owned; they lie by whole vectors
    auto put_codes = [&](int8_t* codes, uint8_t* exps, const float (&x)[8]) {
        uint32_t E;
        const uint2 q = encode8(x, E);
        const uint64_t v = ((uint64_t(q.y) << 32) | q.x) >> (8 * span.skip);
        store_codes(codes + row * Cp, exps + row * (Cp / kGroup), uint32_t(Cp), span.c,
                    make_uint2(uint32_t(v), uint32_t(v >> 32)), E);
    };
    load(row);
    for (; row < a.T; row += step) {
        float x[8], v[8];
        widen8<DT>(rr, v);
        if (a.b) widen8<DT>(rb, x);
        load(row + step < a.T ? row + step : row);
        if (a.b) {
            if (post) normed(x, a.post == kNormLayer, a.post_stats);
            if (a.codes_b) {
                if (!post) span.mask(ragged, x);
                put_codes(a.codes_b, a.exps_b, x);
            }
            if (post) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], w_b[e], o_b[e]);
            }
            if (a.gate) {
                float g[8];
                span.gate<DT>(a.gate, a.gate_f32, fast_div(uint32_t(row), dr), a.C, g);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= g[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = fmaf(a.alpha, x[e], v[e]);
        }
        if (a.r_out) span.store<DT>(row_ptr<DT>(a.r_out, row, a.ldro), v);
        if (!pre) continue;
        normed(v, a.pre == kNormLayer, a.pre_stats);
        if (a.codes_n) put_codes(a.codes_n, a.exps_n, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e], w_n[e], o_n[e]);
        span.store<DT>(row_ptr<DT>(a.n, row, a.ldn), v);
    }
}

// ---------------------------------------------------------------------------
// backward

// A saved vector: the stored tensor's elements, or codes and exponent.
template <int DT, bool CODES, bool WHOLE>
struct Saved {
    Raw8<DT> raw;
    __device__ __forceinline__ void load(const void* x, int64_t ld, const int8_t*, const uint8_t*,
                                         int64_t row, int64_t, uint32_t c, int C)
    {
        raw = load8<DT, WHOLE>(row_ptr<DT>(x, row, ld), c, C);
    }
    __device__ __forceinline__ void xhat(float mean, float rstd, float (&v)[8]) const
    {
        widen8<DT>(raw, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (v[e] - mean) * rstd;
    }
};

template <int DT, bool WHOLE>
struct Saved<DT, true, WHOLE> {
    uint2 q;
    uint32_t E;
    __device__ __forceinline__ void load(const void*, int64_t, const int8_t* codes,
                                         const uint8_t* exps, int64_t row, int64_t Cp,
                                         uint32_t c, int)
    {
        q = make_uint2(0u, 0u);
        E = 0;
        if (c < Cp) {
            q = *reinterpret_cast<const uint2*>(codes + row * Cp + c);
            E = (exps + row * (Cp / kGroup))[c / kGroup];
        }
    }
    __device__ __forceinline__ void xhat(float, float, float (&v)[8]) const { decode8(q, E, v); }
};

// How the rows are dealt: every workgroup walks rows of whole gate groups
// (cpg == 1: gpw groups each), or a part of one group's rows (cpg > 1 workgroups
// a group, rc rows each), so that no workgroup holds a share of two gate sums.
// Without a gate all rows are one group.
struct RowDeal {
    int64_t R, cpg, rc, gpw, grid;
};

RowDeal deal_rows(int64_t T, int64_t R, int64_t target)
{
    RowDeal d;
    d.R = R;
    const int64_t per = max64(1, ceil_div(T, target));
    if (R >= 2 * per) {
        d.cpg = ceil_div(R, per);
        d.rc = ceil_div(R, d.cpg);
        d.cpg = ceil_div(R, d.rc);
        d.gpw = 1;
        d.grid = T / R * d.cpg;
    } else {
        d.cpg = 1;
        d.rc = R;
        d.gpw = max64(1, per / R);
        d.grid = ceil_div(T / R, d.gpw);
    }
    return d;
}

// The sums over rows that a call needs, in the order of their workspace sections.
enum { kSumPreW = 0, kSumPreB, kSumPostW, kSumPostB, kSumGate, kSums };

struct SumSlots {
    int at[kSums];       // section of each sum, or -1
    int count;
};

SumSlots sum_slots(const ResnormBwd& a, int64_t cpg)
{
    SumSlots s;
    s.count = 0;
    const bool want[kSums] = {a.dpre_w != nullptr, a.dpre_b != nullptr, a.dpost_w != nullptr,
                              a.dpost_b != nullptr, a.dgate != nullptr && cpg > 1};
    for (int i = 0; i < kSums; ++i) s.at[i] = want[i] ? s.count++ : -1;
    return s;
}

// NT threads hold a row, NV vectors each.
//
// NV = 2: a row's raw vectors stay in registers over its phases.  NV = 4 (WIDE): they
// would not fit next to five sums of 32 columns; every phase reads them again, from
// cache, and the sums of the weights lie in LDS, each in its thread's own slots.
template <int DT, int NT, int NV, bool CODES, bool BIAS, bool GATE, bool WHOLE>
__global__ __launch_bounds__(NT) void k_resnorm_bwd(ResnormBwd a, RowDeal d, SumSlots ss,
                                                    float* part)
{
    constexpr bool WIDE = NV == 4;
    __shared__ float slots[kSlots][2][NT / kWave];
    RowSum<NT> sum{slots};
    const int C = int(a.C);
    const float inv_c = 1.f / float(a.C);
    const int64_t Cp = code_pitch(a.C);
    const bool has_b = a.db != nullptr;
    const bool pre = a.pre != kNormNone && a.dn;
    const bool read_b = has_b && (a.post != kNormNone || (GATE && a.dgate));
    int col[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        col[k] = (int(threadIdx.x) + k * NT) * kRowV;
    }
    // sums: 0 pre weight, 1 post weight, 2 pre bias, 3 post bias, 4 gate
    constexpr int kInLds = WIDE ? 2 : 0, kInRegs = 5 - kInLds;
    float s_v[kInRegs][NV][8];
    __shared__ float4 s_lds[WIDE ? 4 * NV : 1][WIDE ? NT : 1];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int s = 0; s < kInRegs; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) s_v[s][k][e] = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * kInLds; ++i)
            s_lds[i * NV + k][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // adds to sum s of vector k
    auto add = [&](auto s_, int k, const float (&v)[8]) {
        constexpr int s = decltype(s_)::value;
        if constexpr (s >= kInLds) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s_v[s - kInLds][k][e] += v[e];
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float4& q = s_lds[(2 * s + h) * NV + k][threadIdx.x];
                q = make_float4(q.x + v[4 * h], q.y + v[4 * h + 1], q.z + v[4 * h + 2],
                                q.w + v[4 * h + 3]);
            }
        }
    };
    // sum s of vector k
    auto get = [&](auto s_, int k, float (&v)[8]) {
        constexpr int s = decltype(s_)::value;
        if constexpr (s >= kInLds) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = s_v[s - kInLds][k][e];
        } else {
            const float4 q0 = s_lds[2 * s * NV + k][threadIdx.x];
            const float4 q1 = s_lds[(2 * s + 1) * NV + k][threadIdx.x];
            v[0] = q0.x; v[1] = q0.y; v[2] = q0.z; v[3] = q0.w;
            v[4] = q1.x; v[5] = q1.y; v[6] = q1.z; v[7] = q1.w;
        }
    };
    using std::integral_constant;
    constexpr integral_constant<int, 0> kPreW{};
    constexpr integral_constant<int, 1> kPostW{};
    constexpr integral_constant<int, 2> kPreB{};
    constexpr integral_constant<int, 3> kPostB{};
    constexpr integral_constant<int, 4> kGateS{};
    // keeps the loads of one vector from moving over another's work, which would
    // hold all of them in registers at once
    auto fence = [&](int k) {
        if constexpr (WIDE) asm volatile("" : "+v"(col[k]) : : "memory");
    };

    const int64_t group0 = int64_t(blockIdx.x) / d.cpg * d.gpw;
    const int64_t row0 = group0 * d.R + int64_t(blockIdx.x) % d.cpg * d.rc;
    const int64_t row1 = d.cpg > 1 ? dmin(row0 + d.rc, (group0 + 1) * d.R)
                                   : dmin(row0 + d.gpw * d.R, a.T);
    int64_t grow = group0, in_group = 0;       // gate row, rows of it seen (cpg == 1)

    // what a row reads
    struct RowIn {
        Raw8<DT> dn[NV], dro[NV];
        Saved<DT, CODES, WHOLE> sn[NV], sb[NV];
        float mn, rn, mb, rb;
    };
    auto load_pre = [&](int64_t row, int k, RowIn& q) {
        q.dro[k] = Raw8<DT>{};
        if (a.dr_out) q.dro[k] = load8<DT, WHOLE>(row_ptr<DT>(a.dr_out, row, a.lddro), col[k], C);
        if (pre) {
            q.dn[k] = load8<DT, WHOLE>(row_ptr<DT>(a.dn, row, a.lddn), col[k], C);
            q.sn[k].load(a.r_out, a.ldro, a.codes_n, a.exps_n, row, Cp, col[k], C);
        }
    };
    auto load_post = [&](int64_t row, int k, RowIn& q) {
        if (read_b) q.sb[k].load(a.b, a.ldb, a.codes_b, a.exps_b, row, Cp, col[k], C);
    };
    auto load_row = [&](int64_t row, RowIn& q) {
        q.mn = q.rn = q.mb = 0.f;
        q.rb = 1.f;
        if (pre) {
            q.mn = a.pre_stats[2 * row];
            q.rn = a.pre_stats[2 * row + 1];
        }
        if (has_b && a.post != kNormNone) {
            q.mb = a.post_stats[2 * row];
            q.rb = a.post_stats[2 * row + 1];
        }
        if constexpr (!WIDE) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                load_pre(row, k, q);
                load_post(row, k, q);
            }
        }
    };
    RowIn now;
    for (int64_t row = row0; row < row1; ++row) {
        // everything that follows from the columns (addresses, masks of a ragged
        // end) is formed anew in each row: held over the loop it takes the registers
        // that the row needs
#pragma unroll
        for (int k = 0; k < NV; ++k) asm volatile("" : "+v"(col[k]));
        load_row(row, now);
        const float mn = now.mn, rn = now.rn, mb = now.mb, rb = now.rb;
        auto& dn = now.dn;
        auto& dro = now.dro;
        auto& sn = now.sn;
        auto& sb = now.sb;

        // <q xn>, <q>, and the sums of the pre-norm's vectors
        float c1 = 0.f, c0 = 0.f;
        if (pre) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                fence(k);
                if constexpr (WIDE) load_pre(row, k, now);
                float g[8], x[8], w[8];
                widen8<DT>(dn[k], g);
                sn[k].xhat(mn, rn, x);
                load_cols<WHOLE>(a.pre_w, col[k], C, 1.f, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    c0 = fmaf(g[e], w[e], c0);
                    x[e] *= g[e];
                    c1 = fmaf(x[e], w[e], c1);
                }
                add(kPreW, k, x);
                if constexpr (BIAS) add(kPreB, k, g);
            }
            sum(c1, c0);
            c1 *= inv_c;
            c0 = a.pre == kNormLayer ? c0 * inv_c : 0.f;
        }

        // D, and dz = alpha*g*D with its sums
        float D[NV][8];
        float e1 = 0.f, e0 = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            fence(k);
            if constexpr (WIDE) load_pre(row, k, now);
            widen8<DT>(dro[k], D[k]);
            if (pre) {
                float g[8], x[8], w[8];
                widen8<DT>(dn[k], g);
                sn[k].xhat(mn, rn, x);
                load_cols<WHOLE>(a.pre_w, col[k], C, 1.f, w);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    D[k][e] = fmaf(rn, fmaf(g[e], w[e], -c0) - x[e] * c1, D[k][e]);
            }
            if (a.dr) store8<DT, WHOLE>(row_ptr<DT>(a.dr, row, a.lddr), col[k], C, D[k]);
            if (!has_b) continue;
            if constexpr (WIDE) load_post(row, k, now);
            float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, w[8];
            if (read_b) sb[k].xhat(mb, rb, x);
            if (a.post != kNormNone) load_cols<WHOLE>(a.post_w, col[k], C, 1.f, w);
            if constexpr (GATE) {
                float g[8];
                load_gate<DT, WHOLE>(a.gate, a.gate_f32, grow, a.C, col[k], g);
#pragma unroll
                for (int e = 0; e < 8; ++e) D[k][e] *= a.alpha;
                float p[8];
                load_cols<WHOLE>(a.post != kNormNone ? a.post_b : nullptr, col[k], C, 0.f, p);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    p[e] = D[k][e] * (a.post != kNormNone ? fmaf(x[e], w[e], p[e]) : x[e]);
                add(kGateS, k, p);
                if (a.dgate && d.R == 1) {
                    if (a.gate_f32) store8<kF32, WHOLE>(row_ptr<kF32>(a.dgate, row, a.C), col[k], C, p);
                    else store8<DT, WHOLE>(row_ptr<DT>(a.dgate, row, a.C), col[k], C, p);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) D[k][e] *= g[e];
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) D[k][e] *= a.alpha;
            }
            if (a.post != kNormNone) {
                if constexpr (BIAS) add(kPostB, k, D[k]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] *= D[k][e];
                    e1 = fmaf(x[e], w[e], e1);
                    D[k][e] *= w[e];
                    e0 += D[k][e];
                }
                add(kPostW, k, x);
            }
        }
        if constexpr (GATE) {
            // a whole group's gate sum is done: write it and start the next
            if (d.cpg == 1 && ++in_group == d.R) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    float v[8];
                    get(kGateS, k, v);
                    if (a.dgate && d.R > 1) {
                        if (a.gate_f32) store8<kF32, WHOLE>(row_ptr<kF32>(a.dgate, grow, a.C), col[k], C, v);
                        else store8<DT, WHOLE>(row_ptr<DT>(a.dgate, grow, a.C), col[k], C, v);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) s_v[kInRegs - 1][k][e] = 0.f;
                }
                in_group = 0;
                ++grow;
            }
        }
        if (!has_b) continue;
        if (a.post != kNormNone) {
            sum(e1, e0);
            e1 *= inv_c;
            e0 = a.post == kNormLayer ? e0 * inv_c : 0.f;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            fence(k);
            if (a.post != kNormNone) {
                float x[8];
                if constexpr (WIDE) load_post(row, k, now);
                sb[k].xhat(mb, rb, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) D[k][e] = rb * (D[k][e] - e0 - x[e] * e1);
            }
            store8<DT, WHOLE>(row_ptr<DT>(a.db, row, a.lddb), col[k], C, D[k]);
        }
    }

    // this workgroup's share of the sums: section s, workgroup, column
    auto put = [&](int section, auto s_, int k) {
        if (section < 0) return;
        float v[8];
        get(s_, k, v);
        store8<kF32, true>(row_ptr<kF32>(part, int64_t(section) * d.grid + blockIdx.x, Cp), col[k], int(Cp), v);
    };
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        put(ss.at[kSumPreW], kPreW, k);
        put(ss.at[kSumPostW], kPostW, k);
        if constexpr (BIAS) {
            put(ss.at[kSumPreB], kPreB, k);
            put(ss.at[kSumPostB], kPostB, k);
        }
        if constexpr (GATE) put(ss.at[kSumGate], kGateS, k);
    }
}

// The same for rows of up to 4096 columns, one vector a thread: what all rows use stays
// in registers, and each raw vector is replaced by the next row's as soon as it has been
// used, so that a row's loads are in flight over the reductions of the one before.
// FULL: layer norms, or biases; without it (RMS norms) the means of q and h and the
// biases' sums are left out.  ALL: both norms, both gradients in and both out (what a
// training step asks for), so that nothing in a row depends on a pointer being there.
// At 16384 x 4096 bf16 from codes with a gate vector: 142 us, 4.8 TB/s of the 675 MB it
// cannot do without (a large copy runs at 4.9).  Vector instructions bounded earlier forms
// of it as much as HBM (205 us at twice their number); 128 registers or fewer, two
// workgroups of 512 a CU, are worth 40 us.
template <int DT, int NT, bool CODES, bool FULL, bool GATE, bool ALL>
__global__ __launch_bounds__(NT) void k_resnorm_bwd_row(ResnormBwd a, RowDeal d, SumSlots ss,
                                                        float* part)
{
    constexpr int M = FULL ? 2 : 1;
    __shared__ float slots[kSlots][2][NT / kWave];
    RowSum<NT> sum{slots};
    const int C = int(a.C);
    const float inv_c = 1.f / float(C);
    const int64_t Cp = code_pitch(a.C);
    const bool has_b = ALL || a.db != nullptr, post = ALL || a.post != kNormNone;
    const bool pre = ALL || (a.pre != kNormNone && a.dn);
    const bool read_b = ALL || (has_b && (post || (GATE && a.dgate)));
    const bool ragged = C % kRowV != 0;
    Span span(threadIdx.x, C);
    auto load_saved = [&](Saved<DT, CODES, true>& s, const char* x, const int8_t* codes,
                          const uint8_t* exps) {
        if constexpr (CODES) {
            s.q = span.load_codes(codes);
            s.E = exps[(span.in ? span.c : 0u) / kGroup];
        } else {
            s.raw = span.load<DT>(x);
        }
    };

    const int64_t group0 = int64_t(blockIdx.x) / d.cpg * d.gpw;
    const int64_t row0 = group0 * d.R + int64_t(blockIdx.x) % d.cpg * d.rc;
    const int64_t row1 = d.cpg > 1 ? dmin(row0 + d.rc, (group0 + 1) * d.R)
                                   : dmin(row0 + d.gpw * d.R, a.T);
    int64_t grow = group0, in_group = 0;       // gate row, rows of it seen (cpg == 1)

    // What all rows use: in LDS, each thread its own (registers would not leave 4 waves a
    // SIMD): pre and post weight, alpha * gate, post bias.
    float s_nw[8] = {}, s_bw[8] = {}, s_nb[8] = {}, s_bb[8] = {}, s_g[8] = {};
    constexpr int NW = 2 + (GATE ? (FULL ? 2 : 1) : 0);
    __shared__ float4 w_lds[NW][2][NT];
    auto keep = [&](int i, const float (&v)[8]) {
        w_lds[i][0][threadIdx.x] = make_float4(v[0], v[1], v[2], v[3]);
        w_lds[i][1][threadIdx.x] = make_float4(v[4], v[5], v[6], v[7]);
    };
    auto kept = [&](int i, float (&v)[8]) {
        const float4 f = w_lds[i][0][threadIdx.x], g = w_lds[i][1][threadIdx.x];
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
        v[4] = g.x; v[5] = g.y; v[6] = g.z; v[7] = g.w;
    };
    {
        float w[8];
        span.cols(a.pre_w, 1.f, w);
        keep(0, w);
        span.cols(post ? a.post_w : nullptr, 1.f, w);
        keep(1, w);
        if constexpr (GATE && FULL) {
            span.cols(post ? a.post_b : nullptr, 0.f, w);
            keep(NW - 1, w);
        }
    }
    auto load_gates = [&] {
        float w[8];
        span.gate<DT>(a.gate, a.gate_f32, grow, a.C, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= a.alpha;
        keep(2, w);
    };
    if constexpr (GATE) {
        if (row0 < row1) load_gates();
    }

    Raw8<DT> dn{}, dro{};
    Saved<DT, CODES, true> sn{}, sb{};
    float mn = 0.f, rn = 0.f, mb = 0.f, rb = 1.f;
    auto load_pre = [&](int64_t row) {
        if (ALL || a.dr_out) dro = span.load<DT>(row_ptr<DT>(a.dr_out, row, a.lddro));
        if (pre) {
            dn = span.load<DT>(row_ptr<DT>(a.dn, row, a.lddn));
            load_saved(sn, row_ptr<DT>(a.r_out, row, a.ldro), a.codes_n + row * Cp,
                       a.exps_n + row * (Cp / kGroup));
        }
    };
    auto load_post = [&](int64_t row) {
        if (read_b)
            load_saved(sb, row_ptr<DT>(a.b, row, a.ldb), a.codes_b + row * Cp,
                       a.exps_b + row * (Cp / kGroup));
    };
    auto load_stats = [&](int64_t row) {
        if (pre) {
            if constexpr (!CODES) mn = a.pre_stats[2 * row];
            rn = a.pre_stats[2 * row + 1];
        }
        if (has_b && post) {
            if constexpr (!CODES) mb = a.post_stats[2 * row];
            rb = a.post_stats[2 * row + 1];
        }
    };
    if (row0 < row1) {
        load_stats(row0);
        load_pre(row0);
        load_post(row0);
    }
    for (int64_t row = row0; row < row1; ++row) {
        const int64_t next = row + 1 < row1 ? row + 1 : row;
        // what follows from the column is formed anew in each row: held over the loop it
        // takes registers that the row needs
        asm volatile("" : "+v"(span.at), "+v"(span.c));
        // <q xn>, <q>, and the sums of the pre-norm's vectors
        float x[8], q[8], D[8], m[M] = {};
        widen8<DT>(dro, D);
        const float rn_row = rn, mb_row = mb, rb_row = rb;
        if (pre) {
            float g[8], w_n[8];
            kept(0, w_n);
            widen8<DT>(dn, g);
            sn.xhat(mn, rn, x);
            span.mask(ragged, g);
            span.mask(ragged, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s_nw[e] = fmaf(g[e], x[e], s_nw[e]);
                q[e] = g[e] * w_n[e];
                m[0] = fmaf(q[e], x[e], m[0]);
                if constexpr (FULL) {
                    s_nb[e] += g[e];
                    m[1] += q[e];
                }
            }
        }
        load_pre(next);
        load_stats(next);
        if (pre) {
            sum.add(m);
            const float c1 = m[0] * inv_c;
            const float c0 = FULL && a.pre == kNormLayer ? m[FULL ? 1 : 0] * inv_c : 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (FULL) q[e] -= c0;
                D[e] = fmaf(rn_row, fmaf(-x[e], c1, q[e]), D[e]);
            }
        }
        if (ALL || a.dr) span.store<DT>(row_ptr<DT>(a.dr, row, a.lddr), D);
        if (!has_b) continue;

        // h = alpha*g*D*w_post with its sums
        if (read_b) {
            sb.xhat(mb_row, post ? rb_row : 1.f, x);
            span.mask(ragged, x);
            span.mask(ragged, D);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0.f;
        }
        float w_b[8];
        kept(1, w_b);
        if constexpr (GATE) {
            float o[8];
            if constexpr (FULL) kept(NW - 1, o);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s_g[e] = fmaf(D[e], FULL ? fmaf(x[e], w_b[e], o[e]) : x[e] * w_b[e], s_g[e]);
            kept(2, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) D[e] *= o[e];
        }
#pragma unroll
        for (int k = 0; k < M; ++k) m[k] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (!GATE) D[e] *= a.alpha;
            s_bw[e] = fmaf(D[e], x[e], s_bw[e]);
            if constexpr (FULL) s_bb[e] += D[e];
            D[e] *= w_b[e];
            m[0] = fmaf(D[e], x[e], m[0]);
            if constexpr (FULL) m[1] += D[e];
        }
        if constexpr (GATE) {
            // a whole group's gate sum is done: write it and start the next
            if (d.cpg == 1 && ++in_group == d.R) {
#pragma unroll
                for (int e = 0; e < 8; ++e) s_g[e] *= a.alpha;
                if (a.dgate) {
                    if (a.gate_f32) span.store<kF32>(row_ptr<kF32>(a.dgate, grow, a.C), s_g);
                    else span.store<DT>(row_ptr<DT>(a.dgate, grow, a.C), s_g);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) s_g[e] = 0.f;
                in_group = 0;
                ++grow;
                if (row + 1 < row1) load_gates();
            }
        }
        load_post(next);
        if (post) {
            sum.add(m);
            const float e1 = m[0] * inv_c * rb_row;
            const float e0 = FULL && a.post == kNormLayer ? m[FULL ? 1 : 0] * inv_c * rb_row : 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                D[e] = fmaf(D[e], rb_row, -x[e] * e1);
                if constexpr (FULL) D[e] -= e0;
            }
        }
        span.store<DT>(row_ptr<DT>(a.db, row, a.lddb), D);
    }

    // this workgroup's share of the sums: section, workgroup, column
    auto put = [&](int section, const float (&v)[8]) {
        if (section >= 0)
            span.store<kF32>(row_ptr<kF32>(part, int64_t(section) * d.grid + blockIdx.x, Cp), v);
    };
    put(ss.at[kSumPreW], s_nw);
    put(ss.at[kSumPostW], s_bw);
    if constexpr (FULL) {
        put(ss.at[kSumPreB], s_nb);
        put(ss.at[kSumPostB], s_bb);
    }
    if constexpr (GATE) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s_g[e] *= a.alpha;
        put(ss.at[kSumGate], s_g);
    }
}

// Adds the workgroups' shares in fp64, in their order: blockIdx.y below ss.count
// (without the gate) one vector's sum over all of them, above it one gate row's over
// its cpg.
constexpr int kFinCols = 64, kFinRows = 16;

template <int DT>
__global__ __launch_bounds__(kFinCols* kFinRows) void k_resnorm_fin(ResnormBwd a, RowDeal d,
                                                                    SumSlots ss,
                                                                    const float* part)
{
    const int64_t Cp = code_pitch(a.C);
    const int64_t c = int64_t(blockIdx.x) * kFinCols + threadIdx.x % kFinCols;
    const int ph = threadIdx.x / kFinCols;
    const bool gate = ss.at[kSumGate] >= 0;
    const int vectors = ss.count - (gate ? 1 : 0);
    const int y = blockIdx.y;
    int64_t w0 = 0, w1 = d.grid;
    int s = y;
    if (y >= vectors) {
        s = ss.at[kSumGate];
        w0 = (y - vectors) * d.cpg;
        w1 = w0 + d.cpg;
    }
    double v = 0.0;
    if (c < a.C)
#pragma unroll 8
        for (int64_t w = w0 + ph; w < w1; w += kFinRows)
            v += double(part[(int64_t(s) * d.grid + w) * Cp + c]);
    __shared__ double sh[kFinRows][kFinCols];
    sh[ph][threadIdx.x % kFinCols] = v;
    __syncthreads();
    if (ph != 0 || c >= a.C) return;
    for (int i = 1; i < kFinRows; ++i) v += sh[i][threadIdx.x % kFinCols];
    const float f = float(v);
    if (y >= vectors) {
        const int64_t i = int64_t(y - vectors) * a.C + c;
        if (a.gate_f32) static_cast<float*>(a.dgate)[i] = f;
        else if constexpr (DT == kF32) static_cast<float*>(a.dgate)[i] = f;
        else static_cast<uint16_t*>(a.dgate)[i] = pack1<DT>(f);
    } else if (s == ss.at[kSumPreW]) a.dpre_w[c] = f;
    else if (s == ss.at[kSumPreB]) a.dpre_b[c] = f;
    else if (s == ss.at[kSumPostW]) a.dpost_w[c] = f;
    else a.dpost_b[c] = f;
}

// Threads and vectors that hold a row of the backward.
struct BwdShape {
    int nt, nv;
};

BwdShape bwd_shape(int64_t C)
{
    const int64_t v = code_pitch(C) / kRowV;
    if (C < kRowV) return {512, 2};            // no vector fits: element by element
    if (v <= 64) return {64, 1};
    if (v <= 128) return {128, 1};
    if (v <= 256) return {256, 1};
    if (v <= 512) return {512, 1};
    if (v <= 1024) return {512, 2};
    return {512, 4};
}

// Workgroups the row blocks are dealt to: 16 waves a CU.
int64_t bwd_target(int64_t C, int64_t cus)
{
    return cus * max64(1, 1024 / bwd_shape(C).nt);
}

}  // namespace

size_t resnorm_workspace_bytes(int64_t T, int64_t C, int64_t R, int64_t cus)
{
    if (T <= 0 || C <= 0) return 0;
    const RowDeal d = deal_rows(T, R, bwd_target(C, cus));
    return size_t(kSums) * size_t(d.grid) * size_t(code_pitch(C)) * 4;
}

void launch_resnorm_forward(const ResnormFwd& a, int dtype, int64_t cus, hipStream_t s)
{
    const int64_t v = code_pitch(a.C) / kRowV;
    const FastDiv dr = make_fast_div(uint32_t(a.R));
    with_dtype(dtype, [&](auto dt) {
        auto row = [&](auto tpr) {
            constexpr int TPR = decltype(tpr)::value;
            constexpr int NT = TPR == kWave ? kThreads : TPR;
            const dim3 grid(unsigned(min64(ceil_div(a.T, NT / TPR), cus * (1024 / NT))));
            hipLaunchKernelGGL((k_resnorm_fwd_row<decltype(dt)::value, TPR>), grid, dim3(NT), 0, s,
                               a, dr);
        };
        auto wide = [&](auto tpr) {
            constexpr int TPR = decltype(tpr)::value;
            const dim3 grid(unsigned(min64(a.T, cus * (2048 / TPR))));
            with_whole(a.C, [&](auto whole) {
                hipLaunchKernelGGL((k_resnorm_fwd<decltype(dt)::value, TPR, 2,
                                                  decltype(whole)::value>),
                                   grid, dim3(TPR), 0, s, a, dr);
            });
        };
        using std::integral_constant;
        if (a.C < kRowV) wide(integral_constant<int, 512>{});      // element by element
        else if (v <= 64) row(integral_constant<int, 64>{});
        else if (v <= 128) row(integral_constant<int, 128>{});
        else if (v <= 256) row(integral_constant<int, 256>{});
        else if (v <= 512) row(integral_constant<int, 512>{});
        else if (v <= 1024) wide(integral_constant<int, 512>{});
        else wide(integral_constant<int, 1024>{});
    });
}

void launch_resnorm_backward(const ResnormBwd& a, int dtype, int64_t cus, void* ws,
                             hipStream_t s)
{
    RowDeal d{a.R, 1, a.R, 1, 0};
    if (a.T > 0) d = deal_rows(a.T, a.R, bwd_target(a.C, cus));
    const SumSlots ss = sum_slots(a, d.cpg);
    float* part = static_cast<float*>(ws);
    const bool codes = a.codes_n != nullptr || a.codes_b != nullptr;
    const bool full = a.pre == kNormLayer || a.post == kNormLayer || a.dpre_b || a.dpost_b ||
                      a.post_b;
    const bool gate = a.gate != nullptr && a.db != nullptr;
    const bool all = a.pre != kNormNone && a.post != kNormNone && a.dn && a.dr_out && a.dr && a.db;
    const BwdShape sh = bwd_shape(a.C);
    with_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        using std::integral_constant;
        using Y = std::true_type;
        using N = std::false_type;
        auto on = [](bool v, auto&& f) {
            if (v) f(Y{});
            else f(N{});
        };
        const dim3 grid(unsigned(d.grid));
        auto row_kernel = [&](auto nt) {
            constexpr int NT = decltype(nt)::value;
            on(codes, [&](auto cd) { on(full, [&](auto fu) { on(gate, [&](auto ga) {
                on(all, [&](auto all_) {
                    hipLaunchKernelGGL(
                        (k_resnorm_bwd_row<DT, NT, decltype(cd)::value, decltype(fu)::value,
                                           decltype(ga)::value, decltype(all_)::value>),
                        grid, dim3(NT), 0, s, a, d, ss, part);
                });
            }); }); });
        };
        // f(codes, full, gate, whole); ragged rows take the kernel with every sum, whether
        // wanted or not
        auto wide_kernel = [&](auto nv) {
            auto go = [&](auto cd, auto fu, auto ga, auto whole) {
                hipLaunchKernelGGL(
                    (k_resnorm_bwd<DT, 512, decltype(nv)::value, decltype(cd)::value,
                                   decltype(fu)::value, decltype(ga)::value,
                                   decltype(whole)::value>),
                    grid, dim3(512), 0, s, a, d, ss, part);
            };
            on(codes, [&](auto cd) {
                if (a.C % kRowV != 0) {
                    go(cd, Y{}, Y{}, N{});
                    return;
                }
                on(full, [&](auto fu) { on(gate, [&](auto ga) { go(cd, fu, ga, Y{}); }); });
            });
        };
        if (d.grid > 0) {
            if (sh.nv == 4) wide_kernel(integral_constant<int, 4>{});
            else if (sh.nv == 2) wide_kernel(integral_constant<int, 2>{});
            else if (sh.nt == 64) row_kernel(integral_constant<int, 64>{});
            else if (sh.nt == 128) row_kernel(integral_constant<int, 128>{});
            else if (sh.nt == 256) row_kernel(integral_constant<int, 256>{});
            else row_kernel(integral_constant<int, 512>{});
        }
        const int vectors = ss.count - (ss.at[kSumGate] >= 0 ? 1 : 0);
        const int64_t gates = ss.at[kSumGate] >= 0 ? a.T / a.R : 0;
        if (vectors + gates > 0)
            hipLaunchKernelGGL((k_resnorm_fin<DT>),
                               dim3(unsigned(ceil_div(a.C, kFinCols)), unsigned(vectors + gates)),
                               dim3(kFinCols * kFinRows), 0, s, a, d, ss, part);
    });
}

}  // namespace iabn
