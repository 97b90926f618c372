// Activations kept in 8 bits: pack (tensor -> codes and scale exponents) and unpack
// (codes -> tensor, with an optional column scale and shift).  The format and why it
// was taken: rows.hpp.
//
// Both are one pass over the data: thread i of the launch owns vector i (eight
// columns) of the flat list of rows x vectors; a quad of lanes finds its group's
// largest magnitude with two lane exchanges, and nothing else is shared.  The list
// covers a row's padded width (a whole number of groups), so quads never
// straddle rows.
#include <hip/hip_runtime.h>

#include "block.hpp"
#include "rows.hpp"

namespace iabn {

namespace {

template <int DT, bool WHOLE>
__global__ __launch_bounds__(kThreads) void k_codes_pack(const void* __restrict__ x, int64_t ldx,
                                                         int64_t row0, uint32_t nvec, uint32_t vpr,
                                                         FastDiv dv, int C,
                                                         int8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ exps)
{
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= nvec) return;                 // whole quads: nvec is a multiple of 4
    const uint32_t r = fast_div(i, dv);
    const int64_t row = row0 + r;
    const uint32_t c = (i - r * vpr) * kRowV, Cp = vpr * kRowV;
    float v[8];
    widen8<DT>(load8<DT, WHOLE, uint64_t>(row_ptr<DT>(x, row, ldx), c, C), v);
    uint32_t E;
    const uint2 q = encode8(v, E);
    store_codes(codes + row * Cp, exps + row * (Cp / kGroup), Cp, c, q, E);
}

template <int DT, bool WHOLE>
__global__ __launch_bounds__(kThreads) void k_codes_unpack(
    const int8_t* __restrict__ codes, const uint8_t* __restrict__ exps, int64_t row0,
    uint32_t nvec, uint32_t vpr, FastDiv dv, int C, const float* __restrict__ scale,
    const float* __restrict__ shift, void* __restrict__ y, int64_t ldy)
{
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= nvec) return;
    const uint32_t r = fast_div(i, dv);
    const int64_t row = row0 + r;
    const uint32_t c = (i - r * vpr) * kRowV, Cp = vpr * kRowV;
    if (c >= uint32_t(C)) return;
    float v[8];
    decode8(*reinterpret_cast<const uint2*>(codes + row * Cp + c),
            exps[row * (Cp / kGroup) + c / kGroup], v);
    if (scale || shift) {                   // uniform over the launch
        float a[8], b[8];
        load_cols<WHOLE, uint64_t>(scale, c, C, 1.f, a);
        load_cols<WHOLE, uint64_t>(shift, c, C, 0.f, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e], a[e], b[e]);
    }
    store8<DT, WHOLE, uint64_t>(row_ptr<DT>(y, row, ldy), c, C, v);
}

}  // namespace

void launch_codes_pack(const void* x, int64_t ldx, int64_t T, int64_t C, int dtype, int8_t* codes,
                       uint8_t* exps, hipStream_t s)
{
    const int64_t vpr = code_pitch(C) / kRowV;
    const FastDiv dv = make_fast_div(uint32_t(vpr));
    with_dtype(dtype, [&](auto d) { with_whole(C, [&](auto whole) {
        each_row_block(T, vpr, kThreads, [&](int64_t row0, uint32_t nvec, dim3 grid) {
            hipLaunchKernelGGL((k_codes_pack<decltype(d)::value, decltype(whole)::value>), grid, dim3(kThreads), 0, s, x,
                               ldx, row0, nvec, uint32_t(vpr), dv, int(C), codes, exps);
        });
    }); });
}

void launch_codes_unpack(const int8_t* codes, const uint8_t* exps, int64_t T, int64_t C,
                         const float* scale, const float* shift, void* y, int64_t ldy, int dtype,
                         hipStream_t s)
{
    const int64_t vpr = code_pitch(C) / kRowV;
    const FastDiv dv = make_fast_div(uint32_t(vpr));
    with_dtype(dtype, [&](auto d) { with_whole(C, [&](auto whole) {
        each_row_block(T, vpr, kThreads, [&](int64_t row0, uint32_t nvec, dim3 grid) {
            hipLaunchKernelGGL((k_codes_unpack<decltype(d)::value, decltype(whole)::value>), grid, dim3(kThreads), 0, s,
                               codes, exps, row0, nvec, uint32_t(vpr), dv, int(C), scale, shift, y,
                               ldy);
        });
    }); });
}

}  // namespace iabn
