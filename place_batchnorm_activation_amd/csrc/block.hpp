// Host launchers of the residual-block operators.  They enqueue on `s` and return;
// arguments are validated by the C ABI layer (api_block.cpp) before any of these is
// called.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "plan.hpp"

namespace iabn {

constexpr int kGroup = 32;     // values that share a scale

constexpr int64_t code_pitch(int64_t C) { return (C + kGroup - 1) / kGroup * kGroup; }

// Division of n < 2^31 by d through one product: (n * m) >> s.
struct FastDiv {
    uint32_t m, s;
};

inline FastDiv make_fast_div(uint32_t d)
{
    uint32_t s = 0;
    while ((uint64_t(1) << s) < d) ++s;
    const uint64_t m = ((uint64_t(1) << (31 + s)) + d - 1) / d;
    return FastDiv{uint32_t(m), 31 + s};
}

// Calls f(row0, vectors, grid) over blocks of rows whose vectors index in 31 bits
// (larger problems take several launches).
template <class F>
inline void each_row_block(int64_t T, int64_t vectors_per_row, int64_t vectors_per_wg, F&& f)
{
    const int64_t most = ((int64_t(1) << 31) - 1) / max64(1, vectors_per_row);
    const int64_t step = min64(T, max64(1, most));
    for (int64_t row0 = 0; row0 < T; row0 += step) {
        const int64_t nvec = min64(step, T - row0) * vectors_per_row;
        f(row0, uint32_t(nvec), dim3(unsigned(ceil_div(nvec, vectors_per_wg))));
    }
}

// Calls f(std::true_type) when rows of C columns are whole vectors of 8, else
// f(std::false_type).
template <class F>
inline void with_whole(int64_t C, F&& f)
{
    if (C % 8 == 0) f(std::true_type{});
    else f(std::false_type{});
}

// codes.hip
void launch_codes_pack(const void* x, int64_t ldx, int64_t T, int64_t C, int dtype, int8_t* codes,
                       uint8_t* exps, hipStream_t s);
void launch_codes_unpack(const int8_t* codes, const uint8_t* exps, int64_t T, int64_t C,
                         const float* scale, const float* shift, void* y, int64_t ldy, int dtype,
                         hipStream_t s);

// glu.hip
enum GluAct { kSilu = 0, kGelu = 1, kGeluTanh = 2 };

struct GluFwd {
    const void *gate, *up;
    void* out;
    int64_t ldg, ldu, ldo;
    int8_t *codes_g, *codes_u;
    uint8_t *exps_g, *exps_u;
};
struct GluBwd {
    const int8_t *codes_g, *codes_u;
    const uint8_t *exps_g, *exps_u;
    const void* dout;
    void *dgate, *dup, *out;
    int64_t lddo, lddg, lddu, ldo;
};
void launch_glu_forward(const GluFwd& a, int64_t T, int64_t F, int dtype, int act, hipStream_t s);
void launch_glu_backward(const GluBwd& a, int64_t T, int64_t F, int dtype, int act, hipStream_t s);

// wgrad.hip: lanes reach up to 16 rows of dy and of the codes in 32 bits of bytes
constexpr int64_t kWgradMaxLd = int64_t(1) << 26;
struct WgradArgs {
    const void* dy;
    int64_t lddy;
    const int8_t* codes;
    const uint8_t* exps;
    const float *scale, *shift;
    void* dw;
    int64_t lddw;
    int dw_dtype;
    int accumulate;
    float* dbias;
    int64_t T, N, K;
};
size_t wgrad_workspace_bytes(int64_t T, int64_t N, int64_t K, int dtype, int64_t cus);
void launch_linear_wgrad(const WgradArgs& a, int dtype, int64_t cus, void* ws, hipStream_t s);

// resnorm.hip
enum NormKind { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };
constexpr int64_t kResnormMaxC = 16384;

struct ResnormFwd {
    const void *r, *b;
    void *r_out, *n;
    int64_t ldr, ldb, ldro, ldn;
    const float *post_w, *post_b, *pre_w, *pre_b;
    const void* gate;
    int gate_f32;
    int64_t R;
    float alpha, eps;
    int post, pre;
    float *post_stats, *pre_stats;
    int8_t *codes_b, *codes_n;
    uint8_t *exps_b, *exps_n;
    int64_t T, C;
};
struct ResnormBwd {
    const void *dr_out, *dn;
    int64_t lddro, lddn;
    const void *r_out, *b;           // the stored tensors, or
    int64_t ldro, ldb;
    const int8_t *codes_n, *codes_b; // their codes
    const uint8_t *exps_n, *exps_b;
    const float *post_stats, *pre_stats;
    const float *post_w, *post_b, *pre_w;
    const void* gate;
    int gate_f32;
    int64_t R;
    float alpha;
    int post, pre;
    void *dr, *db;
    int64_t lddr, lddb;
    float *dpost_w, *dpost_b, *dpre_w, *dpre_b;
    void* dgate;
    int64_t T, C;
};
size_t resnorm_workspace_bytes(int64_t T, int64_t C, int64_t R, int64_t cus);
void launch_resnorm_forward(const ResnormFwd& a, int dtype, int64_t cus, hipStream_t s);
void launch_resnorm_backward(const ResnormBwd& a, int dtype, int64_t cus, void* ws,
                             hipStream_t s);

}  // namespace iabn
