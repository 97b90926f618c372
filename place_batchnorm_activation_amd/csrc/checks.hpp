// Argument checks that the C ABI files of the block operators share (api_block.cpp,
// api_attn.cpp, api_gnorm.cpp); host only, before any HIP call but the device query.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include <hip/hip_runtime_api.h>

#include "block.hpp"
#include "iabn.h"

namespace iabn {

#define IABN_TRY(expr)                          \
    do {                                        \
        const iabn_status st_ = (expr);         \
        if (st_ != IABN_OK) return st_;         \
    } while (0)

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool dtype_ok(int d) { return d == IABN_F32 || d == IABN_BF16 || d == IABN_F16; }

inline int64_t esize(int d) { return d == IABN_F32 ? 4 : 2; }

// CUs of the current device (cached per device); without one the MI355X's 256.
inline int64_t device_cus()
{
    static std::atomic<int> cache[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) {
        (void)hipGetLastError();
        return 256;
    }
    int cus = cache[dev].load(std::memory_order_relaxed);
    if (cus == 0) {
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
            cus <= 0) {
            (void)hipGetLastError();
            return 256;
        }
        cache[dev].store(cus, std::memory_order_relaxed);
    }
    return cus;
}

inline iabn_status launched()
{
    return hipGetLastError() == hipSuccess ? IABN_OK : IABN_ERR_HIP;
}

constexpr int64_t kMaxExtent = (int64_t(1) << 31) - 1;

inline iabn_status check_extents(int64_t rows, int64_t cols, int dtype)
{
    if (!dtype_ok(dtype) || rows < 0 || cols < 0) return IABN_ERR_INVALID_ARG;
    return rows <= kMaxExtent && cols <= kMaxExtent - kGroup ? IABN_OK : IABN_ERR_UNSUPPORTED;
}

// A tensor of rows: where it lies.
struct Rows {
    const void* p;
    int64_t ld, rows, cols, es;
};

inline iabn_status check_rows(const Rows& t)
{
    if (!t.p || t.ld < t.cols) return IABN_ERR_INVALID_ARG;
    if (double(t.rows) * double(t.ld) > 9.0e15) return IABN_ERR_UNSUPPORTED;
    return aligned(t.p, size_t(t.es)) ? IABN_OK : IABN_ERR_MISALIGNED;
}

// Whether two tensors share memory.  Rows at one distance whose columns keep out of
// each other's way (slices of one buffer) do not.
inline bool overlap(const Rows& a, const Rows& b)
{
    if (!a.p || !b.p || a.rows == 0 || b.rows == 0 || a.cols == 0 || b.cols == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    const uintptr_t xe = x + uintptr_t(((a.rows - 1) * a.ld + a.cols) * a.es);
    const uintptr_t ye = y + uintptr_t(((b.rows - 1) * b.ld + b.cols) * b.es);
    if (xe <= y || ye <= x) return false;
    if (a.ld * a.es == b.ld * b.es) {
        const uintptr_t pitch = uintptr_t(a.ld * a.es);
        const bool ylater = y >= x;
        const uintptr_t off = (ylater ? y - x : x - y) % pitch;
        const uintptr_t first = uintptr_t((ylater ? a : b).cols * (ylater ? a : b).es);
        const uintptr_t second = uintptr_t((ylater ? b : a).cols * (ylater ? b : a).es);
        if (off >= first && pitch - off >= second) return false;
    }
    return true;
}

inline bool same(const Rows& a, const Rows& b)
{
    return a.p == b.p && (a.ld == b.ld || a.rows <= 1) && a.es == b.es && a.cols == b.cols &&
           a.rows == b.rows;
}

// An output against an input that it may replace exactly.
inline iabn_status check_out(const Rows& out, const Rows& in)
{
    return !overlap(out, in) || same(out, in) ? IABN_OK : IABN_ERR_INVALID_ARG;
}

inline iabn_status check_apart(const Rows& a, const Rows& b)
{
    return overlap(a, b) ? IABN_ERR_INVALID_ARG : IABN_OK;
}

inline Rows code_rows(const void* codes, int64_t rows, int64_t cols)
{
    return Rows{codes, code_pitch(cols), rows, code_pitch(cols), 1};
}

inline Rows exp_rows(const void* exps, int64_t rows, int64_t cols)
{
    return Rows{exps, code_pitch(cols) / kGroup, rows, code_pitch(cols) / kGroup, 1};
}

inline Rows vector_row(const void* p, int64_t n, int64_t es = 4) { return Rows{p, n, 1, n, es}; }

// Outputs of one call against each other.
template <size_t N>
inline iabn_status check_distinct(const Rows (&outs)[N])
{
    for (size_t i = 1; i < N; ++i)
        for (size_t j = 0; j < i; ++j) IABN_TRY(check_apart(outs[i], outs[j]));
    return IABN_OK;
}

// Outputs against inputs that they may (check_outs) or may not replace exactly.
template <size_t N, size_t M>
inline iabn_status check_outs(const Rows (&outs)[N], const Rows (&ins)[M])
{
    for (const Rows& o : outs)
        if (o.p)
            for (const Rows& i : ins) IABN_TRY(check_out(o, i));
    return IABN_OK;
}
template <size_t N, size_t M>
inline iabn_status check_all_apart(const Rows (&outs)[N], const Rows (&ins)[M])
{
    for (const Rows& o : outs)
        if (o.p)
            for (const Rows& i : ins) IABN_TRY(check_apart(o, i));
    return IABN_OK;
}

inline iabn_status check_codes(const int8_t* codes, const uint8_t* exps)
{
    if (!codes || !exps) return IABN_ERR_INVALID_ARG;
    return aligned(codes, 16) ? IABN_OK : IABN_ERR_MISALIGNED;
}

// Both, or neither.
inline iabn_status check_codes_opt(const int8_t* codes, const uint8_t* exps)
{
    return codes || exps ? check_codes(codes, exps) : IABN_OK;
}

inline iabn_status check_vec(const float* p)
{
    return !p || aligned(p, 4) ? IABN_OK : IABN_ERR_MISALIGNED;
}

// Codes an operator writes, against a tensor it reads or writes.
inline iabn_status check_codes_apart(const int8_t* codes, const uint8_t* exps, int64_t rows,
                              int64_t cols, const Rows& t)
{
    IABN_TRY(check_apart(code_rows(codes, rows, cols), t));
    return check_apart(exp_rows(exps, rows, cols), t);
}

inline iabn_status check_ws(const void* ws, size_t bytes, size_t need)
{
    if (need == 0) return IABN_OK;
    if (!ws || bytes < need) return IABN_ERR_WORKSPACE;
    return aligned(ws, 16) ? IABN_OK : IABN_ERR_MISALIGNED;
}

}  // namespace iabn
