// Weight gradient of a linear layer whose input is kept as 8-bit codes (rows.hpp):
//
//   dW[n,k] = s_k * sum_t dY[t,n] * X[t,k] + t_k * sum_t dY[t,n],   db[n] = sum_t dY[t,n]
//
// X the decoded codes, s and t the optional column scale and shift between them and
// the layer's input (a norm keeps xhat, its weight and bias are s and t), so that
// one buffer of codes serves the norm's backward and this product.
//
// 2*T*N*K operations on the matrix units, which bound it but for small T, N, K.  A
// decoded code is exact in bfloat16 (rows.hpp), and dY is cut into bfloat16 pieces
// whose sum it is exactly: one for bf16, two for f16 (8 + 3 bits), three for f32
// (8 + 8 + 8), each a product of its own; every product of two bfloat16 is exact in
// fp32, so the only roundings are those of the fp32 accumulators.
//
// Both operands have the summed index t as their slow one, while the matrix
// instruction wants 8 consecutive t of one column in a lane.  A thread therefore
// takes blocks of 8 rows x 4 columns through its registers: the transposition costs
// one byte permutation for two elements of dY, and nothing for X, whose decoded
// values are packed in pairs anyway.  Tiles of 64 t lie in LDS as [column][t], 128
// bytes a column, in 16-byte chunks (8 t) whose place is their index XOR a mix of
// the column, so that the 16 lanes of an access phase meet 16 different bank quads.
// Two LDS stages: while one is multiplied, the next tile's loads are in flight.
//
// Few output tiles: the t axis is cut among workgroups, whose fp32 shares go
// through the workspace and are added in their order by a second kernel.
#include <hip/hip_runtime.h>

#include "block.hpp"
#include "rows.hpp"

namespace iabn {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int kBT = 64;                    // t of a tile

constexpr int pieces(int dtype) { return dtype == kBF16 ? 1 : dtype == kF16 ? 2 : 3; }

// 16-byte slot of chunk c (0..7) of column n of a tile.  A read moves 16 lanes at a
// time over 64 banks and meets none twice if their slots differ modulo 16: lanes that
// read one chunk of 16 neighbouring columns differ in n's bits 0-3, of which the row's
// lowest bit holds bit 2 and the mix bits 0, 1 and 3.  (Writes move 8 lanes over 32 banks
// and meet a bank twice: 512 of 1790 LDS cycles a 256 x 256 tile, by the counters.  A mix
// of bits 2, 3 and 1^4 on plain rows frees both, and was slower: 303 against 282 us at
// 8192 x 4096 x 4096 bf16.)
__device__ __forceinline__ int lds_slot(int n, int c)
{
    const int row = (n & ~5) | ((n & 1) << 2) | ((n >> 2) & 1);
    const int mix = ((n ^ (n >> 4)) & 3) | ((n >> 1) & 4);
    return row * 8 + (c ^ mix);
}

// The value of lane j of each quad, in all four.
template <int J>
__device__ __forceinline__ uint32_t quad_lane(uint32_t v)
{
    return uint32_t(__builtin_amdgcn_mov_dpp(int(v), J * 0x55, 0xF, 0xF, true));
}

// High halves of two words: (hi16(b) << 16) | hi16(a).
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b)
{
    return __builtin_amdgcn_perm(b, a, 0x07060302u);
}
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b)
{
    return __builtin_amdgcn_perm(b, a, 0x05040100u);
}

// C (4 or 2) consecutive elements of dY, nv of them valid.
template <int DT, int C>
struct RawC {
    uint32_t w[DT == kF32 ? C : C / 2];
};

template <int DT, int C>
__device__ __forceinline__ RawC<DT, C> load_c(const char* p, int nv)
{
    constexpr int N = DT == kF32 ? C : C / 2;
    RawC<DT, C> r;
    if (nv >= C) {
        if constexpr (N == 4) {
            const u32x4_any_t q = *reinterpret_cast<const u32x4_any_t*>(p);
            r.w[0] = q.x; r.w[1] = q.y; r.w[2] = q.z; r.w[3] = q.w;
        } else if constexpr (N == 2) {
            const u32x2_any_t q = *reinterpret_cast<const u32x2_any_t*>(p);
            r.w[0] = q.x; r.w[1] = q.y;
        } else {
            r.w[0] = *reinterpret_cast<const u32_any_t*>(p);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) r.w[i] = 0u;
#pragma unroll
        for (int e = 0; e < C - 1; ++e)
            if (e < nv) {
                if constexpr (DT == kF32) r.w[e] = reinterpret_cast<const uint32_t*>(p)[e];
                else r.w[e / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(p)[e]) << (16 * (e & 1));
            }
    }
    return r;
}

template <int DT, int C>
__device__ __forceinline__ float elem_c(const RawC<DT, C>& r, int e)
{
    if constexpr (DT == kF32) return __uint_as_float(r.w[e]);
    else return unpack1<DT>(uint16_t(r.w[e / 2] >> (16 * (e & 1))));
}

// C codes of a row.
template <int C>
__device__ __forceinline__ uint32_t codes_c(const int8_t* p)
{
    if constexpr (C == 4) return *reinterpret_cast<const uint32_t*>(p);
    else return *reinterpret_cast<const uint16_t*>(p);
}

// What is left of v after its leading 8 bits are taken.  After an infinity or a NaN,
// whose product with the first piece decides the sum, any finite value serves.
template <int DT>
__device__ __forceinline__ float rest(float v)
{
    const float r = v - __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
    if constexpr (DT == kF16) return fmaxf(r, -1024.f);             // |r| < 2^9; NaN: -1024
    else return __builtin_amdgcn_classf(v, 0x204) ? 0.f : r;        // -inf, +inf
}

struct WgradTiles {
    int64_t splits, chunk;      // workgroups of the t axis, and t of each (multiple of kBT)
    int bm, bn;                 // an output tile
    uint32_t nt, kt;            // their numbers along N and K
    float* part;                // fp32 shares [split][N][K], then [split][N] of dY's sums
    float* part_sum;
    int want_sum;               // dY's sums: 0 none, 1 the first column of tiles, 2 every tile
};

// Which tile and range of t workgroup b takes.  Workgroups go to the 8 XCDs in turn, so
// each XCD is given a run of consecutive tiles, and these walk bands of 4 tiles of N: an
// XCD's L2 then holds what its tiles share (32 tiles: 4 column blocks of dY and 8 of X).
__device__ __forceinline__ void tile_of(uint32_t b, uint32_t grid, const WgradTiles& tl,
                                        uint32_t& tn, uint32_t& tk, uint32_t& split)
{
    const uint32_t per = grid / 8, rest = grid % 8, x = b % 8;
    const uint32_t r = x * per + (x < rest ? x : rest) + b / 8;
    const uint32_t tiles = tl.nt * tl.kt;
    split = r / tiles;
    const uint32_t i = r % tiles, band = i / (4 * tl.kt), in = i % (4 * tl.kt);
    const uint32_t rows = tl.nt - 4 * band < 4 ? tl.nt - 4 * band : 4;
    tn = 4 * band + in % rows;
    tk = in / rows;
}

// Calls f(put), put(o, v) writing v to element o of dW, or adding it.
template <class F>
__device__ __forceinline__ void with_out(const WgradArgs& a, F&& f)
{
    if (a.dw_dtype == kF32) {
        float* d = static_cast<float*>(a.dw);
        if (a.accumulate) f([&](int64_t o, float v) { d[o] += v; });
        else f([&](int64_t o, float v) { d[o] = v; });
    } else {
        uint16_t* d = static_cast<uint16_t*>(a.dw);
        const bool bf = a.dw_dtype == kBF16, add = a.accumulate;
        f([&](int64_t o, float v) {
            if (add) v += bf ? unpack1<kBF16>(d[o]) : unpack1<kF16>(d[o]);
            d[o] = bf ? pack1<kBF16>(v) : pack1<kF16>(v);
        });
    }
}

// One output tile (BM columns of dY x BN columns of X) over one range of t.  WM x WN
// is a wave's share.
//
// FAST: both extents reach a tile's.  The last tile of a ragged extent then begins
// earlier, inside the tensor, and writes only what the tile before it does not, so
// that no load needs a mask but those of the last t.
template <int DT, int BM, int BN, int WM, int WN, int D, bool FAST, bool SUMS>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * kWave) void k_wgrad(WgradArgs a,
                                                                         WgradTiles tl)
{
    constexpr int P = pieces(DT), ES = DT == kF32 ? 4 : 2;
    constexpr int NT = (BM / WM) * (BN / WN) * kWave;
    constexpr int MI = WM / 32, NI = WN / 32, KS = kBT / 16;
    // a thread takes a block of 8 t x CA columns of dY and one of 8 t x CB columns of X
    constexpr int CA = BM * 8 / NT, CB = BN * 8 / NT, QA = BM / CA, QB = BN / CB;
    constexpr int kStage = (P * BM + BN) * 8;        // 16-byte slots
    static_assert((CA == 2 || CA == 4) && (CB == 2 || CB == 4), "blocks of 2 or 4 columns");
    __shared__ uint4 lds[2 * kStage];

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    uint32_t tn, tk, split;
    tile_of(blockIdx.x, gridDim.x, tl, tn, tk, split);
    const int64_t n_own = int64_t(tn) * BM, k_own = int64_t(tk) * BN;
    const int64_t t0 = int64_t(split) * tl.chunk, t1 = dmin(t0 + tl.chunk, a.T);
    const int64_t Kp = code_pitch(a.K), G = Kp / kGroup;
    const int64_t n0 = FAST ? dmin(n_own, a.N - BM) : n_own;
    const int64_t k0 = FAST ? dmin(k_own, Kp - BN) : k_own;
    const bool sums = SUMS && (tl.want_sum == 2 || k_own == 0);

    const int qa = tid % QA, ca = tid / QA, qb = tid % QB, cb = tid / QB;

    // Addresses: a wave-uniform row plus a lane's 32-bit offset.  A wave holds chunk
    // ca0 (and where a tile is narrower than a wave's 64 blocks, the next ones).  For
    // the scales, lane i of a quad reads those of rows i and i + 4 of its group.
    const int ca0 = __builtin_amdgcn_readfirstlane(ca), cb0 = __builtin_amdgcn_readfirstlane(cb);
    const uint32_t oa = uint32_t(8 * (ca - ca0)) * uint32_t(a.lddy * ES) + CA * qa * ES;
    const uint32_t ob = uint32_t(8 * (cb - cb0)) * uint32_t(Kp) + CB * qb;
    const uint32_t oe = uint32_t(8 * (cb - cb0) + lane % 4) * uint32_t(G) + CB * qb / kGroup;

    struct Block {
        RawC<DT, CA> a[8];
        uint32_t b[8], e[2];
    } raw[D];                                       // tiles on their way
    auto fetch = [&](int64_t t, Block& r) {         // a whole tile, of FAST
        const char* ua = static_cast<const char*>(a.dy) + ((t + 8 * ca0) * a.lddy + n0) * ES;
        const int8_t* ub = a.codes + (t + 8 * cb0) * Kp + k0;
        const uint8_t* ue = a.exps + (t + 8 * cb0) * G + k0 / kGroup;
#pragma unroll
        for (int j = 0; j < 8; ++j) r.a[j] = load_c<DT, CA>(ua + j * a.lddy * ES + oa, CA);
#pragma unroll
        for (int j = 0; j < 8; ++j) r.b[j] = codes_c<CB>(ub + j * Kp + ob);
        r.e[0] = ue[oe];
        r.e[1] = (ue + 4 * G)[oe];
    };
    auto fetch_part = [&](int64_t t, Block& r) {              // rows past t1 (and columns) read as zero
        const char* ua = static_cast<const char*>(a.dy) + ((t + 8 * ca0) * a.lddy + n0) * ES;
        const int8_t* ub = a.codes + (t + 8 * cb0) * Kp + k0;
        const uint8_t* ue = a.exps + (t + 8 * cb0) * G + k0 / kGroup;
        const int64_t left = a.N - (n0 + CA * qa);
        const int nv = FAST || left >= CA ? CA : (left > 0 ? int(left) : 0);
        const int rows_a = int(dmin(t1 - t - 8 * ca, 8));
        const int rows_b = FAST || k0 + CB * qb < Kp ? int(dmin(t1 - t - 8 * cb, 8)) : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            r.a[j] = load_c<DT, CA>(ua + j * a.lddy * ES + oa, j < rows_a ? nv : 0);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            r.b[j] = j < rows_b ? codes_c<CB>(ub + j * Kp + ob) : 0u;
        r.e[0] = lane % 4 < rows_b ? ue[oe] : 0u;
        r.e[1] = lane % 4 + 4 < rows_b ? (ue + 4 * G)[oe] : 0u;
    };

    float sum[CA] = {};

    // column e of this thread's blocks, from registers into a stage
    auto stage_a = [&](int st, int e, const Block& r) {
        const auto& ra = r.a;
        uint4* A = lds + st * kStage;
        if constexpr (P == 1) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = (e & 1) ? high_halves(ra[2 * j].w[e / 2], ra[2 * j + 1].w[e / 2])
                               : low_halves(ra[2 * j].w[e / 2], ra[2 * j + 1].w[e / 2]);
            A[lds_slot(CA * qa + e, ca)] = make_uint4(w[0], w[1], w[2], w[3]);
            if constexpr (SUMS) {
                // two elements at a time: their dot product with ones
                const bf16x2_t one = {(__bf16)1.f, (__bf16)1.f};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sum[e] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w[j]), one,
                                                             sum[e], false);
            }
        } else {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = elem_c<DT, CA>(ra[j], e);
            if constexpr (SUMS) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) s += v[j];
                sum[e] += s;
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = high_halves(__float_as_uint(v[2 * j]), __float_as_uint(v[2 * j + 1]));
                A[p * BM * 8 + lds_slot(CA * qa + e, ca)] = make_uint4(w[0], w[1], w[2], w[3]);
                if (p + 1 < P) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = rest<DT>(v[j]);
                }
            }
        }
    };
    float scale[8];
    auto scales = [&](const Block& r) {
        const uint32_t lo = r.e[0] << 23, hi = r.e[1] << 23;
        scale[0] = __uint_as_float(quad_lane<0>(lo));
        scale[1] = __uint_as_float(quad_lane<1>(lo));
        scale[2] = __uint_as_float(quad_lane<2>(lo));
        scale[3] = __uint_as_float(quad_lane<3>(lo));
        scale[4] = __uint_as_float(quad_lane<0>(hi));
        scale[5] = __uint_as_float(quad_lane<1>(hi));
        scale[6] = __uint_as_float(quad_lane<2>(hi));
        scale[7] = __uint_as_float(quad_lane<3>(hi));
    };
    auto stage_b = [&](int st, int e, const Block& r) {
        const auto& rb = r.b;
        uint4* B = lds + st * kStage + P * BM * 8;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = float(int8_t(rb[2 * j] >> (8 * e))) * scale[2 * j];
            const float y = float(int8_t(rb[2 * j + 1] >> (8 * e))) * scale[2 * j + 1];
            w[j] = high_halves(__float_as_uint(x), __float_as_uint(y));
        }
        B[lds_slot(CB * qb + e, cb)] = make_uint4(w[0], w[1], w[2], w[3]);
    };

    f32x16_t acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    const int wm = (wave / (BN / WN)) * WM, wn = (wave % (BN / WN)) * WN;
    // fragments of 16 t of the stage, and their products
    struct Frags {
        bf16x8_t a[P][MI], b[NI];
    };
    auto load_frags = [&](int st, int ks, Frags& f) {
        const uint4* A = lds + st * kStage;
        const uint4* B = A + P * BM * 8;
        const int c = ks * 2 + lane / 32;
#pragma unroll
        for (int j = 0; j < NI; ++j)
            f.b[j] = __builtin_bit_cast(bf16x8_t, B[lds_slot(wn + j * 32 + lane % 32, c)]);
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < MI; ++i)
                f.a[p][i] = __builtin_bit_cast(
                    bf16x8_t, A[p * BM * 8 + lds_slot(wm + i * 32 + lane % 32, c)]);
    };
    auto multiply = [&](const Frags& f) {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[p][i], f.b[j],
                                                                       acc[i][j], 0, 0, 0);
    };
    auto multiply_all = [&](int st) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            Frags f;
            load_frags(st, ks, f);
            multiply(f);
        }
    };
    auto stage_all = [&](int st, const Block& r) {
        scales(r);
#pragma unroll
        for (int e = 0; e < CA; ++e) stage_a(st, e, r);
#pragma unroll
        for (int e = 0; e < CB; ++e) stage_b(st, e, r);
    };

    // Whole tiles: while stage st is multiplied, a slice of t at a time, the next one is
    // made from the registers, a column at a time, and the loads of the one after it go
    // out.  All of it is one run of instructions without a branch, over which the compiler
    // deals matrix and vector ones.
    int64_t t = t0;
    int st = 0;
    const int whole = FAST && t0 < t1 ? int((t1 - t0) / kBT) : 0;
    // past the last whole tile: that one again (read, not used)
    auto tile_t = [&](int i) { return t0 + int64_t(i < whole ? i : whole - 1) * kBT; };
    if (whole > 0) {
        auto step = [&](int i, Block& r) {
            __syncthreads();       // stage st is written, the other read by nobody
            // keeps the conversions, which wait for their loads, behind the barrier
            if constexpr (D > 1) __builtin_amdgcn_sched_barrier(0);
            scales(r);
            // the next slice's fragments are read ahead where registers allow it
            constexpr int FB = SUMS && BM * BN >= 128 * 256 ? 1 : 2;
            Frags f[FB];
            load_frags(st, 0, f[0]);
#pragma unroll
            for (int e = 0; e < KS; ++e) {
                if (FB == 2 && e + 1 < KS) load_frags(st, e + 1, f[(e + 1) % FB]);
                multiply(f[e % FB]);
                if (e % (KS / CA) == 0) stage_a(st ^ 1, e * CA / KS, r);
                if (e % (KS / CB) == 0) stage_b(st ^ 1, e * CB / KS, r);
                if (FB == 1 && e + 1 < KS) load_frags(st, e + 1, f[0]);
            }
            fetch(tile_t(i + D), r);
            st ^= 1;
        };
#pragma unroll
        for (int d = 0; d < D; ++d) fetch(tile_t(d), raw[d]);
        stage_all(0, raw[0]);
        fetch(tile_t(D), raw[0]);
        int i = 1;
        for (; i + D <= whole; i += D)
#pragma unroll
            for (int d = 0; d < D; ++d) step(i + d, raw[(1 + d) % D]);
#pragma unroll
        for (int d = 0; d < D - 1; ++d)
            if (i + d < whole) step(i + d, raw[(1 + d) % D]);
        t += int64_t(whole) * kBT;
        __syncthreads();
        multiply_all(st);
        st ^= 1;
    }
    // the last, partial tile (without FAST: all of them)
    for (; t < t1; t += kBT) {
        fetch_part(t, raw[0]);
        stage_all(st, raw[0]);
        __syncthreads();
        multiply_all(st);
        st ^= 1;
    }

    // dY's sums of this tile's columns, added over the 8 chunks in their order
    float* ls = reinterpret_cast<float*>(lds);
    if constexpr (SUMS) {
        __syncthreads();
        if (sums) {
#pragma unroll
            for (int e = 0; e < CA; ++e) ls[ca * BM + CA * qa + e] = sum[e];
        }
        __syncthreads();
        if (sums) {
            for (int n = tid; n < BM; n += NT) {
                float s = 0.f;
#pragma unroll
                for (int c = 0; c < 8; ++c) s += ls[c * BM + n];
                ls[8 * BM + n] = s;
                if (k_own == 0 && n0 + n >= n_own && n0 + n < a.N) {
                    if (tl.splits > 1) tl.part_sum[int64_t(split) * a.N + n0 + n] = s;
                    else if (a.dbias) a.dbias[n0 + n] = a.accumulate ? a.dbias[n0 + n] + s : s;
                }
            }
        }
        __syncthreads();
    }

    // accumulator element r of a lane: row 8*(r/4) + 4*(lane/32) + r%4, column lane%32;
    // out(row of the tile, n, k, value) for each that this tile owns
    auto each = [&](auto&& out) {
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int64_t k = k0 + wn + j * 32 + lane % 32;
            if (k < k_own || k >= a.K) continue;
            const float sc = a.scale ? a.scale[k] : 1.f, sh = a.shift ? a.shift[k] : 0.f;
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int m = wm + i * 32 + 8 * (r / 4) + 4 * (lane / 32) + r % 4;
                    const int64_t n = n0 + m;
                    if (n >= n_own && n < a.N) out(m, n, k, acc[i][j][r], sc, sh);
                }
        }
    };
    if (tl.splits > 1) {
        float* part = tl.part + int64_t(split) * a.N * a.K;
        each([&](int, int64_t n, int64_t k, float v, float, float) { part[n * a.K + k] = v; });
    } else {
        with_out(a, [&](auto put) {
            each([&](int m, int64_t n, int64_t k, float v, float sc, float sh) {
                v *= sc;
                if (a.shift) v = fmaf(sh, ls[8 * BM + m], v);
                put(n * a.lddw + k, v);
            });
        });
    }
}

// The sum of `count` shares, `stride` apart, in their order; eight loads at a time in
// flight (past the last share, the last one again).
__device__ __forceinline__ float sum_shares(const float* p, int64_t stride, int64_t count)
{
    float s = 0.f;
    for (int64_t i = 0; i < count; i += 8) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = p[(i + u < count ? i + u : count - 1) * stride];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (i + u < count) s += v[u];
    }
    return s;
}

// Adds the shares of the t axis: one output row a blockIdx.y.
__global__ __launch_bounds__(kThreads) void k_wgrad_join(WgradArgs a, WgradTiles tl)
{
    const int64_t n = blockIdx.y, k = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    float s = 0.f;
    if (a.shift || (a.dbias && k == 0)) s = sum_shares(tl.part_sum + n, a.N, tl.splits);
    if (a.dbias && k == 0) a.dbias[n] = a.accumulate ? a.dbias[n] + s : s;
    if (k >= a.K) return;
    float v = sum_shares(tl.part + n * a.K + k, a.N * a.K, tl.splits);
    if (a.scale) v *= a.scale[k];
    if (a.shift) v = fmaf(a.shift[k], s, v);
    with_out(a, [&](auto put) { put(n * a.lddw + k, v); });
}

// The tile, and the splits of the t axis: a workgroup for every place (one a CU; two of
// the bf16 128 x 128 tile, whose LDS is 64 KB), each with at least 4 tiles of t.
//
// bf16: 256 x 256 where these make a quarter of the CUs' number of tiles, else
// 128 x 128, whose shares of t are larger and fewer (us, 256 against 128 tiles, bf16:
// 8192 x 2048 x 4096 166 against 191, 8192 x 2048^2 95 against 108; 8192 x 1024^2 44 against
// 40, 1024^3 29 against 21).  f16 and f32: 128 x 256, which shares the conversion of dY
// among twice the products, where its tiles and their splits make a workgroup for every CU
// (8192 x 4096^2 503 against 675 us f16, 740 against 953 f32; 2048^2 x 1024 f32 43 against
// 47; but 1024 x 512^2 20 against 16 f32 and 300 x 1000 x 777 22 against 15 f16), else, and
// where K is under 256, 128 x 128.
WgradTiles make_tiles(int64_t T, int64_t N, int64_t K, int dtype, int64_t cus)
{
    WgradTiles tl{};
    const int64_t Kp = code_pitch(K);
    if (dtype == kBF16) {
        const bool big = N >= 256 && Kp >= 256 && ceil_div(N, 256) * ceil_div(K, 256) * 4 >= cus;
        tl.bm = tl.bn = big ? 256 : 128;
    } else {
        tl.bm = 128;
        const int64_t wide = ceil_div(N, 128) * ceil_div(K, 256) * max64(1, ceil_div(T, kBT) / 4);
        tl.bn = Kp >= 256 && N >= 128 && wide >= cus ? 256 : 128;
    }
    tl.nt = uint32_t(ceil_div(N, tl.bm));
    tl.kt = uint32_t(max64(1, ceil_div(K, tl.bn)));      // K == 0: dY's sums alone
    const int64_t tiles = int64_t(tl.nt) * tl.kt, steps = ceil_div(T, kBT);
    const int64_t places = dtype == kBF16 && tl.bm == 128 ? 2 * cus : cus;
    int64_t splits = max64(1, min64(places / tiles, steps / 4));
    const int64_t per = max64(1, ceil_div(steps, splits));
    tl.splits = max64(1, ceil_div(steps, per));
    tl.chunk = per * kBT;
    return tl;
}

}  // namespace

size_t wgrad_workspace_bytes(int64_t T, int64_t N, int64_t K, int dtype, int64_t cus)
{
    const WgradTiles tl = make_tiles(T, N, K, dtype, cus);
    return tl.splits > 1 ? size_t(tl.splits) * size_t(N) * size_t(K + 1) * 4 : 0;
}

void launch_linear_wgrad(const WgradArgs& a, int dtype, int64_t cus, void* ws, hipStream_t s)
{
    WgradTiles tl = make_tiles(a.T, a.N, a.K, dtype, cus);
    tl.part = static_cast<float*>(ws);
    tl.part_sum = tl.part + tl.splits * a.N * a.K;
    tl.want_sum = (a.shift && tl.splits == 1) ? 2 : (a.dbias || a.shift) ? 1 : 0;
    with_dtype(dtype, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        const dim3 grid(unsigned(int64_t(tl.nt) * tl.kt * tl.splits));
        const bool fast = a.N >= tl.bm && code_pitch(a.K) >= tl.bn;
        auto go = [&](auto sums) {
            constexpr bool S = decltype(sums)::value;
            if constexpr (DT == kBF16) {
                if (tl.bm == 256)
                    hipLaunchKernelGGL((k_wgrad<DT, 256, 256, 128, 64, 1, true, S>), grid,
                                       dim3(512), 0, s, a, tl);
                else if (fast)
                    hipLaunchKernelGGL((k_wgrad<DT, 128, 128, 64, 64, 2, true, S>), grid,
                                       dim3(256), 0, s, a, tl);
                else
                    hipLaunchKernelGGL((k_wgrad<DT, 128, 128, 64, 64, 1, false, S>), grid,
                                       dim3(256), 0, s, a, tl);
            } else {
                if (tl.bn == 256)
                    hipLaunchKernelGGL((k_wgrad<DT, 128, 256, 64, 64, DT == kF16 ? 2 : 1, true, S>), grid,
                                       dim3(512), 0, s, a, tl);
                else if (fast)
                    hipLaunchKernelGGL((k_wgrad<DT, 128, 128, 32, 64, 2, true, S>), grid,
                                       dim3(512), 0, s, a, tl);
                else
                    hipLaunchKernelGGL((k_wgrad<DT, 128, 128, 32, 64, 1, false, S>), grid,
                                       dim3(512), 0, s, a, tl);
            }
        };
        if (tl.want_sum) go(std::true_type{});
        else go(std::false_type{});
    });
    if (tl.splits > 1)
        hipLaunchKernelGGL(k_wgrad_join,
                           dim3(unsigned(max64(1, ceil_div(a.K, kThreads))), unsigned(a.N)),
                           dim3(kThreads), 0, s, a, tl);
}

}  // namespace iabn
