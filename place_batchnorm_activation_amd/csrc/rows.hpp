// Device helpers of the residual-block operators (codes.hip, glu.hip, wgrad.hip,
// resnorm.hip): rows of any stride in eight-element vectors, and the 8-bit codes.
//
// A row of C elements is walked in vectors of kRowV = 8.  Vector j covers columns
// 8j .. 8j + 7; four neighbouring vectors (four neighbouring lanes) are one group of
// kGroup = 32 values that share a scale.  Rows may start at any element: the 16-byte
// accesses below promise the alignment of one element only, which the hardware's
// unaligned access mode serves, so odd widths and slices keep wide loads.
//
// OFF is the type of a byte offset within a row: uint64_t where a row may have 2^30 columns
// and more (codes, gated unit: its address is a lane's own there, and 64 bits cost nothing),
// uint32_t in the norms, whose rows are narrow and whose row addresses are scalar.
//
// Codes: value = q * 2^(E - 127), q in [-127, 127], E one byte for each group.
// E is the smallest exponent under which the group's largest magnitude rounds to
// at most 127: with that magnitude m * 2^k, 1 <= m < 2, m * 64 rounds to at most
// 127 exactly when m < 127.5/64, so the step is 2^(k-6), else 2^(k-5).  A power of
// two was taken over max/127 (at most one bit finer): q times a power of two has 8
// significant bits and is therefore exact in bfloat16, so that products with
// decoded codes run on the matrix units without another rounding, and one byte
// holds the scale.  E = 0 marks a group of zeros, E = 255 one that held an infinity
// or a NaN; it decodes to NaN throughout (q = 0 times infinity).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.hpp"
#include "block.hpp"

namespace iabn {

constexpr int kRowV = 8;

// Valid elements of the vector at column c of a row of C columns.
__device__ __forceinline__ int valid8(int c, int C)
{
    const int n = C - c;
    return n >= kRowV ? kRowV : (n > 0 ? n : 0);
}

// 16 bytes at an address aligned to one element only.
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any_t __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_any_t __attribute__((aligned(2)));

__device__ __forceinline__ uint4 load16_any(const void* p)
{
    const u32x4_any_t q = *static_cast<const u32x4_any_t*>(p);
    return make_uint4(q.x, q.y, q.z, q.w);
}

// Eight raw elements: one 16-byte access for 16-bit storage, two for fp32.
template <int DT>
struct Raw8 {
    uint4 q[DT == kF32 ? 2 : 1];
};

// Row `row` of a tensor whose rows are ld elements apart.  With a wave-uniform row
// the address stays scalar, and vectors of it are reached by 32-bit offsets.
template <int DT>
__device__ __forceinline__ const char* row_ptr(const void* base, int64_t row, int64_t ld)
{
    return static_cast<const char*>(base) + row * ld * (DT == kF32 ? 4 : 2);
}

// v moved down by s elements (0 < s < 8), zeros from above.
template <int DT>
__device__ __forceinline__ void shift_down(uint32_t (&w)[DT == kF32 ? 8 : 4], uint32_t s)
{
    constexpr int N = DT == kF32 ? 8 : 4;
    uint32_t words = DT == kF32 ? s : s >> 1;      // whole words first, then half a word
#pragma unroll
    for (int b = 1; b < N; b *= 2)
#pragma unroll
        for (int i = 0; i < N; ++i)
            w[i] = (words & b) ? (i + b < N ? w[i + b] : 0u) : w[i];
    if constexpr (DT != kF32) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t up = i + 1 < N ? w[i + 1] : 0u;
            w[i] = (s & 1) ? __builtin_amdgcn_alignbyte(up, w[i], 2) : w[i];
        }
    }
}

// Eight elements from column c of a row of C columns on; those past its end read as
// zero.  WHOLE: C is a multiple of 8, and a vector is in the row or past it.  Otherwise
// the vector that holds the end is the row's last eight elements moved down, so
// every load is one wide access; rows of fewer than eight columns are read one by one.
// (The ragged form takes dozens of vector instructions a load, which bounds kernels of
// several loads a row: 16640 x 1151 in resnorm's backward took 158 us with it, and takes 78
// where the last vector begins early instead, which is what rows of up to 4096 columns do.)
template <int DT, bool WHOLE, class OFF = uint32_t>
__device__ __forceinline__ Raw8<DT> load8(const char* row, uint32_t c, int C)
{
    constexpr int N = DT == kF32 ? 8 : 4, es = DT == kF32 ? 4 : 2;
    Raw8<DT> r;
#pragma unroll
    for (int h = 0; h < N / 4; ++h) r.q[h] = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (WHOLE) {
        if (c < uint32_t(C)) {
#pragma unroll
            for (int h = 0; h < N / 4; ++h) r.q[h] = load16_any(row + OFF(c) * es + 16 * h);
        }
        return r;
    }
    uint32_t w[N];
    if (C >= kRowV) {
        const uint32_t last = uint32_t(C) - kRowV, at = c < last ? c : last;
        if (c < uint32_t(C)) {
#pragma unroll
            for (int h = 0; h < N / 4; ++h) r.q[h] = load16_any(row + OFF(at) * es + 16 * h);
        }
        if (c > last && c < uint32_t(C)) {
#pragma unroll
            for (int h = 0; h < N / 4; ++h) {
                w[4 * h] = r.q[h].x; w[4 * h + 1] = r.q[h].y;
                w[4 * h + 2] = r.q[h].z; w[4 * h + 3] = r.q[h].w;
            }
            shift_down<DT>(w, c - last);
#pragma unroll
            for (int h = 0; h < N / 4; ++h)
                r.q[h] = make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
        }
    } else if (c == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = 0u;
#pragma unroll 1
        for (int e = C - 1; e >= 0; --e) {
#pragma unroll
            for (int i = N - 1; i >= 0; --i) {
                const uint32_t dn = i > 0 ? w[i - 1] : 0u;
                w[i] = DT == kF32 ? dn : __builtin_amdgcn_alignbyte(w[i], dn, 2);
            }
            if constexpr (DT == kF32) w[0] = reinterpret_cast<const uint32_t*>(row)[e];
            else w[0] |= reinterpret_cast<const uint16_t*>(row)[e];
        }
#pragma unroll
        for (int h = 0; h < N / 4; ++h)
            r.q[h] = make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
    }
    return r;
}

template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT>& r, float (&v)[8])
{
    if constexpr (DT == kF32) {
        v[0] = __uint_as_float(r.q[0].x); v[1] = __uint_as_float(r.q[0].y);
        v[2] = __uint_as_float(r.q[0].z); v[3] = __uint_as_float(r.q[0].w);
        v[4] = __uint_as_float(r.q[1].x); v[5] = __uint_as_float(r.q[1].y);
        v[6] = __uint_as_float(r.q[1].z); v[7] = __uint_as_float(r.q[1].w);
    } else {
        unpack16<DT>(r.q[0], v);
    }
}

// Eight values at column c of a row of C columns, rounded once to the storage dtype;
// those past its end are not written (WHOLE as above; else four, two and one of the rest).
template <int DT, bool WHOLE, class OFF = uint32_t>
__device__ __forceinline__ void store8(const char* row, uint32_t c, int C, const float (&v)[8])
{
    constexpr int es = DT == kF32 ? 4 : 2;
    char* p = const_cast<char*>(row) + OFF(c) * es;
    const int nv = valid8(int(c), C);
    if (nv >= kRowV) {
        if constexpr (DT == kF32) {
            const u32x4_any_t a = {__float_as_uint(v[0]), __float_as_uint(v[1]),
                                   __float_as_uint(v[2]), __float_as_uint(v[3])};
            const u32x4_any_t b = {__float_as_uint(v[4]), __float_as_uint(v[5]),
                                   __float_as_uint(v[6]), __float_as_uint(v[7])};
            reinterpret_cast<u32x4_any_t*>(p)[0] = a;
            reinterpret_cast<u32x4_any_t*>(p)[1] = b;
        } else {
            const uint4 q = pack16<DT>(v);
            const u32x4_any_t a = {q.x, q.y, q.z, q.w};
            *reinterpret_cast<u32x4_any_t*>(p) = a;
        }
    } else if constexpr (WHOLE) {
    } else if constexpr (DT == kF32) {
        if (nv & 4) {
            const u32x4_any_t a = {__float_as_uint(v[0]), __float_as_uint(v[1]),
                                   __float_as_uint(v[2]), __float_as_uint(v[3])};
            *reinterpret_cast<u32x4_any_t*>(p) = a;
        }
        float* f = reinterpret_cast<float*>(p) + (nv & 4);
        const bool up = nv & 4;
        // values first: a select of array elements would put the array in memory
        const float v0 = v[0], v1 = v[1], v2 = v[2], v4 = v[4], v5 = v[5], v6 = v[6];
        const float a = up ? v4 : v0, b = up ? v5 : v1, d = up ? v6 : v2;
        if (nv & 2) {
            f[0] = a;
            f[1] = b;
        }
        if (nv & 1) f[nv & 2] = (nv & 2) ? d : a;
    } else {
        const uint4 q = pack16<DT>(v);
        if (nv & 4) {
            const u32x2_any_t a = {q.x, q.y};
            *reinterpret_cast<u32x2_any_t*>(p) = a;
        }
        uint16_t* h = reinterpret_cast<uint16_t*>(p) + (nv & 4);
        const bool up = nv & 4;
        const uint32_t q0 = q.x, q1 = q.y, q2 = q.z, q3 = q.w;
        const uint32_t a = up ? q2 : q0, b = up ? q3 : q1;
        if (nv & 2) *reinterpret_cast<u32_any_t*>(h) = a;
        if (nv & 1) h[nv & 2] = uint16_t((nv & 2) ? b : a);
    }
}

// Eight of a per-column vector of C fp32 values (null: `none`); zero past its end.
template <bool WHOLE, class OFF = uint32_t>
__device__ __forceinline__ void load_cols(const float* p, uint32_t c, int C, float none,
                                          float (&v)[8])
{
    if (p) {
        widen8<kF32>(load8<kF32, WHOLE, OFF>(reinterpret_cast<const char*>(p), c, C), v);
    } else {
        const int nv = valid8(int(c), C);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < nv ? none : 0.f;
    }
}

// ---------------------------------------------------------------------------
// codes

// The largest of a quad of neighbouring lanes (lanes 4i .. 4i + 3).
__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    const uint32_t a = __builtin_amdgcn_mov_dpp(int(v), 0xB1, 0xF, 0xF, true);   // 1,0,3,2
    v = v > a ? v : a;
    const uint32_t b = __builtin_amdgcn_mov_dpp(int(v), 0x4E, 0xF, 0xF, true);   // 2,3,0,1
    return v > b ? v : b;
}

// The largest scale exponent: 127 * 2^(248 - 127) is finite, and 64 * 2^(249 - 127)
// would not be.  Magnitudes of 127.5 * 2^121 and above, which it cuts off from their
// own exponent, become 127 * 2^121.
constexpr int kMaxExp = 248;

// Scale exponent of a group from the bits of its largest magnitude.
__host__ __device__ __forceinline__ uint32_t group_exp(uint32_t amax)
{
    const uint32_t k = amax >> 23;
    if (k == 255u) return 255u;
    if (amax == 0u) return 0u;
    const int e = int(k) - 6 + ((amax & 0x7FFFFFu) >= 0x7F0000u ? 1 : 0);
    return e < 1 ? 1u : e > kMaxExp ? uint32_t(kMaxExp) : uint32_t(e);
}

// Codes of eight values, and their group's exponent.  Every lane of the quad
// takes part.  x * 2^(127-E) + 1.5 * 2^23 rounds the product to the nearest
// integer, ties to even (the product alone is exact), and leaves it in two's
// complement in the low byte.
__device__ __forceinline__ uint2 encode8(const float (&v)[8], uint32_t& E)
{
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = __float_as_uint(v[e]) & 0x7FFFFFFFu;
        m = m > b ? m : b;
    }
    E = group_exp(quad_max(m));
    const float inv = __uint_as_float((254u - E) << 23);
    uint32_t b[8];
    if (E == uint32_t(kMaxExp)) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            b[e] = __float_as_uint(fminf(fmaxf(v[e] * inv, -127.f), 127.f) + 12582912.f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = __float_as_uint(fmaf(v[e], inv, 12582912.f));
    }
    // low bytes of four words into one
    const uint32_t lo01 = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
    const uint32_t hi23 = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
    const uint32_t lo45 = __builtin_amdgcn_perm(b[5], b[4], 0x0c0c0400u);
    const uint32_t hi67 = __builtin_amdgcn_perm(b[7], b[6], 0x04000c0cu);
    uint2 q = make_uint2(lo01 | hi23, lo45 | hi67);
    if (E == 255u) q = make_uint2(0u, 0u);
    return q;
}

__device__ __forceinline__ float group_scale(uint32_t E) { return __uint_as_float(E << 23); }

// Four codes of a word, with scale s (exact; NaN for s = infinity, whose codes are 0).
__device__ __forceinline__ void decode4(uint32_t w, float s, float* v)
{
    v[0] = float(int8_t(w)) * s;
    v[1] = float(int8_t(w >> 8)) * s;
    v[2] = float(int8_t(w >> 16)) * s;
    v[3] = float(int8_t(w >> 24)) * s;
}

__device__ __forceinline__ void decode8(uint2 q, uint32_t E, float (&v)[8])
{
    const float s = group_scale(E);
    decode4(q.x, s, v);
    decode4(q.y, s, v + 4);
}

// The codes at column c of a row (`codes` and `exps` the row's own), and from one
// lane of the quad the group's exponent.  Vectors past the padded width Cp are not
// written.
__device__ __forceinline__ void store_codes(int8_t* codes, uint8_t* exps, uint32_t Cp, uint32_t c,
                                            uint2 q, uint32_t E)
{
    if (c < Cp) {
        *reinterpret_cast<uint2*>(codes + c) = q;
        if (c % kGroup == 0) exps[c / kGroup] = uint8_t(E);
    }
}

// ---------------------------------------------------------------------------
// flat walk over the vectors of a block of rows: n / d for n < 2^31 by one product
// (m = ceil(2^(31+s)/d), 2^s >= d: the quotient's error stays below 1/d)
__device__ __forceinline__ uint32_t fast_div(uint32_t n, FastDiv f)
{
    return uint32_t((uint64_t(n) * f.m) >> f.s);
}

}  // namespace iabn
