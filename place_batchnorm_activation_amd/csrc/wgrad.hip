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
constexpr int kChunk = 8;                  // t of a 16-byte chunk

constexpr int pieces(int dtype) { return dtype == kBF16 ? 1 : dtype == kF16 ? 2 : 3; }

// 16-byte slot of chunk c (0..7) of column n of a tile.
__device__ __forceinline__ int lds_slot(int n, int c)
{
    return n * 8 + (c ^ (((n >> 1) ^ (n >> 4)) & 7));
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

// Four consecutive elements of dY, nv of them valid.
template <int DT>
struct Raw4 {
    uint32_t w[DT == kF32 ? 4 : 2];
};

template <int DT>
__device__ __forceinline__ Raw4<DT> load4(const void* base, int64_t i, int nv)
{
    Raw4<DT> r;
    const char* p = static_cast<const char*>(base) + i * (DT == kF32 ? 4 : 2);
    if constexpr (DT == kF32) {
        r.w[0] = r.w[1] = r.w[2] = r.w[3] = 0u;
        if (nv >= 4) {
            const u32x4_any_t q = *reinterpret_cast<const u32x4_any_t*>(p);
            r.w[0] = q.x; r.w[1] = q.y; r.w[2] = q.z; r.w[3] = q.w;
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < nv) r.w[e] = reinterpret_cast<const uint32_t*>(p)[e];
        }
    } else {
        r.w[0] = r.w[1] = 0u;
        if (nv >= 4) {
            const u32x2_any_t q = *reinterpret_cast<const u32x2_any_t*>(p);
            r.w[0] = q.x; r.w[1] = q.y;
        } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
            if (nv > 0) r.w[0] = h[0];
            if (nv > 1) r.w[0] |= uint32_t(h[1]) << 16;
            if (nv > 2) r.w[1] = h[2];
        }
    }
    return r;
}

template <int DT>
__device__ __forceinline__ float elem4(const Raw4<DT>& r, int e)
{
    if constexpr (DT == kF32) return __uint_as_float(r.w[e]);
    else return unpack1<DT>(uint16_t(r.w[e / 2] >> (16 * (e & 1))));
}

// What is left of v after its leading 8 bits are taken (0 after an infinity).
__device__ __forceinline__ float rest(float v)
{
    const uint32_t b = __float_as_uint(v);
    const float r = v - __uint_as_float(b & 0xFFFF0000u);
    return (b & 0x7FFFFFFFu) == 0x7F800000u ? 0.f : r;
}

struct WgradTiles {
    int64_t splits, chunk;      // workgroups of the t axis, and t of each (multiple of kBT)
    uint32_t nt, kt;            // output tiles along N and K
    float* part;                // fp32 shares [split][N][K], then [split][N] of dY's sums
    float* part_sum;
    int want_sum;               // dY's sums: 0 none, 1 the first column of tiles, 2 every tile
};

// One output tile (BM columns of dY x BN columns of X) over one range of t.  WM x WN
// is a wave's share.
template <int DT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * kWave) void k_wgrad(WgradArgs a,
                                                                         WgradTiles tl)
{
    constexpr int P = pieces(DT);
    constexpr int NT = (BM / WM) * (BN / WN) * kWave;
    constexpr int MI = WM / 32, NI = WN / 32;
    constexpr int QA = BM / 4, QB = BN / 4;          // four-column blocks along a tile
    constexpr int IA = QA * 8 / NT, IB = QB * 8 / NT;
    static_assert(IA * NT == QA * 8 && IB * NT == QB * 8, "whole blocks a thread");
    constexpr int kStage = (P * BM + BN) * 8;        // 16-byte slots
    __shared__ uint4 lds[2 * kStage];

    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    const uint32_t tile = blockIdx.x % (tl.nt * tl.kt);
    const int64_t split = blockIdx.x / (tl.nt * tl.kt);
    const int64_t n0 = int64_t(tile / tl.kt) * BM, k0 = int64_t(tile % tl.kt) * BN;
    const int64_t t0 = split * tl.chunk, t1 = dmin(t0 + tl.chunk, a.T);
    const int64_t Kp = code_pitch(a.K), G = Kp / kGroup;
    const bool sums = tl.want_sum == 2 || (tl.want_sum == 1 && k0 == 0);

    Raw4<DT> ra[IA][8];
    uint32_t rb[IB][8];
    uint8_t re[IB][8];
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < IA; ++i) {
            const int id = tid + i * NT, q = id % QA, c = id / QA;
            const int64_t n = n0 + 4 * q, left = a.N - n;
            const int nv = left >= 4 ? 4 : (left > 0 ? int(left) : 0);
            const int64_t row = t + c * kChunk;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                ra[i][j] = load4<DT>(a.dy, (row + j) * a.lddy + n, row + j < t1 ? nv : 0);
        }
#pragma unroll
        for (int i = 0; i < IB; ++i) {
            const int id = tid + i * NT, q = id % QB, c = id / QB;
            const int64_t k = k0 + 4 * q;
            const int64_t row = t + c * kChunk;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = k < Kp && row + j < t1;
                rb[i][j] = in ? *reinterpret_cast<const uint32_t*>(a.codes + (row + j) * Kp + k)
                              : 0u;
                re[i][j] = in ? a.exps[(row + j) * G + k / kGroup] : uint8_t(0);
            }
        }
    };

    float sum[IA][4];
#pragma unroll
    for (int i = 0; i < IA; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[i][e] = 0.f;

    auto stage = [&](int st) {
        uint4* A = lds + st * kStage;
        uint4* B = A + P * BM * 8;
#pragma unroll
        for (int i = 0; i < IA; ++i) {
            const int id = tid + i * NT, q = id % QA, c = id / QA;
            if (sums) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float s = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) s += elem4<DT>(ra[i][j], e);
                    sum[i][e] += s;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = 4 * q + e;
                if constexpr (P == 1) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = (e & 1) ? high_halves(ra[i][2 * j].w[e / 2], ra[i][2 * j + 1].w[e / 2])
                                       : low_halves(ra[i][2 * j].w[e / 2], ra[i][2 * j + 1].w[e / 2]);
                    A[lds_slot(n, c)] = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = elem4<DT>(ra[i][j], e);
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = high_halves(__float_as_uint(v[2 * j]),
                                               __float_as_uint(v[2 * j + 1]));
                        A[p * BM * 8 + lds_slot(n, c)] = make_uint4(w[0], w[1], w[2], w[3]);
                        if (p + 1 < P) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[j] = rest(v[j]);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < IB; ++i) {
            const int id = tid + i * NT, q = id % QB, c = id / QB;
            float v[8][4];
#pragma unroll
            for (int j = 0; j < 8; ++j) decode4(rb[i][j], group_scale(re[i][j]), v[j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = high_halves(__float_as_uint(v[2 * j][e]), __float_as_uint(v[2 * j + 1][e]));
                B[lds_slot(4 * q + e, c)] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    };

    f32x16_t acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    const int wm = (wave / (BN / WN)) * WM, wn = (wave % (BN / WN)) * WN;
    auto multiply = [&](int st) {
        const uint4* A = lds + st * kStage;
        const uint4* B = A + P * BM * 8;
#pragma unroll
        for (int ks = 0; ks < kBT / 16; ++ks) {
            const int c = ks * 2 + lane / 32;
            bf16x8_t fb[NI];
#pragma unroll
            for (int j = 0; j < NI; ++j)
                fb[j] = __builtin_bit_cast(bf16x8_t, B[lds_slot(wn + j * 32 + lane % 32, c)]);
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const bf16x8_t fa = __builtin_bit_cast(
                        bf16x8_t, A[p * BM * 8 + lds_slot(wm + i * 32 + lane % 32, c)]);
#pragma unroll
                    for (int j = 0; j < NI; ++j)
                        acc[i][j] =
                            __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa, fb[j], acc[i][j], 0, 0, 0);
                }
        }
    };

    int st = 0;
    if (t0 < t1) {
        fetch(t0);
        stage(0);
        for (int64_t t = t0 + kBT; t < t1; t += kBT) {
            fetch(t);
            __syncthreads();           // stage st is written; the other is read by nobody
            multiply(st);
            stage(st ^ 1);
            st ^= 1;
        }
        __syncthreads();
        multiply(st);
    }

    // dY's sums of this tile's columns, added over the 8 chunks in their order
    float* ls = reinterpret_cast<float*>(lds);
    if (tl.want_sum) {
        __syncthreads();
        if (sums) {
#pragma unroll
            for (int i = 0; i < IA; ++i) {
                const int id = tid + i * NT, q = id % QA, c = id / QA;
#pragma unroll
                for (int e = 0; e < 4; ++e) ls[c * BM + 4 * q + e] = sum[i][e];
            }
        }
        __syncthreads();
        if (sums) {
            for (int n = tid; n < BM; n += NT) {
                float s = 0.f;
#pragma unroll
                for (int c = 0; c < 8; ++c) s += ls[c * BM + n];
                ls[8 * BM + n] = s;
                if (k0 == 0 && n0 + n < a.N) {
                    if (tl.splits > 1) tl.part_sum[split * a.N + n0 + n] = s;
                    else if (a.dbias) a.dbias[n0 + n] = a.accumulate ? a.dbias[n0 + n] + s : s;
                }
            }
        }
        __syncthreads();
    }

    // accumulator element r of a lane: row 8*(r/4) + 4*(lane/32) + r%4, column lane%32
#pragma unroll
    for (int j = 0; j < NI; ++j) {
        const int64_t k = k0 + wn + j * 32 + lane % 32;
        if (k >= a.K) continue;
        const float sc = a.scale ? a.scale[k] : 1.f, sh = a.shift ? a.shift[k] : 0.f;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int m = wm + i * 32 + 8 * (r / 4) + 4 * (lane / 32) + r % 4;
                const int64_t n = n0 + m;
                if (n >= a.N) continue;
                float v = acc[i][j][r];
                if (tl.splits > 1) {
                    tl.part[(split * a.N + n) * a.K + k] = v;
                    continue;
                }
                v *= sc;
                if (a.shift) v = fmaf(sh, ls[8 * BM + m], v);
                const int64_t o = n * a.lddw + k;
                if (a.dw_dtype == kF32) {
                    float* d = static_cast<float*>(a.dw);
                    d[o] = a.accumulate ? d[o] + v : v;
                } else if (a.dw_dtype == kBF16) {
                    uint16_t* d = static_cast<uint16_t*>(a.dw);
                    d[o] = pack1<kBF16>(a.accumulate ? unpack1<kBF16>(d[o]) + v : v);
                } else {
                    uint16_t* d = static_cast<uint16_t*>(a.dw);
                    d[o] = pack1<kF16>(a.accumulate ? unpack1<kF16>(d[o]) + v : v);
                }
            }
    }
}

// Adds the shares of the t axis in their order: one output row a blockIdx.y.
__global__ __launch_bounds__(kThreads) void k_wgrad_join(WgradArgs a, WgradTiles tl)
{
    const int64_t n = blockIdx.y, k = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    float s = 0.f;
    if (tl.want_sum) {
        for (int64_t i = 0; i < tl.splits; ++i) s += tl.part_sum[i * a.N + n];
        if (a.dbias && k == 0) a.dbias[n] = a.accumulate ? a.dbias[n] + s : s;
    }
    if (k >= a.K) return;
    float v = 0.f;
    for (int64_t i = 0; i < tl.splits; ++i) v += tl.part[(i * a.N + n) * a.K + k];
    if (a.scale) v *= a.scale[k];
    if (a.shift) v = fmaf(a.shift[k], s, v);
    const int64_t o = n * a.lddw + k;
    if (a.dw_dtype == kF32) {
        float* d = static_cast<float*>(a.dw);
        d[o] = a.accumulate ? d[o] + v : v;
    } else if (a.dw_dtype == kBF16) {
        uint16_t* d = static_cast<uint16_t*>(a.dw);
        d[o] = pack1<kBF16>(a.accumulate ? unpack1<kBF16>(d[o]) + v : v);
    } else {
        uint16_t* d = static_cast<uint16_t*>(a.dw);
        d[o] = pack1<kF16>(a.accumulate ? unpack1<kF16>(d[o]) + v : v);
    }
}

constexpr int kTile = 128;

// Splits of the t axis: enough workgroups for two a CU, each with at least 4 tiles
// of t.
WgradTiles make_tiles(int64_t T, int64_t N, int64_t K, int64_t cus)
{
    WgradTiles tl{};
    tl.nt = uint32_t(ceil_div(N, kTile));
    tl.kt = uint32_t(ceil_div(K, kTile));
    const int64_t tiles = int64_t(tl.nt) * tl.kt, steps = ceil_div(T, kBT);
    int64_t splits = max64(1, min64(2 * cus / tiles, steps / 4));
    const int64_t per = max64(1, ceil_div(steps, splits));
    tl.splits = max64(1, ceil_div(steps, per));
    tl.chunk = per * kBT;
    return tl;
}

}  // namespace

size_t wgrad_workspace_bytes(int64_t T, int64_t N, int64_t K, int, int64_t cus)
{
    const WgradTiles tl = make_tiles(T, N, K, cus);
    return tl.splits > 1 ? size_t(tl.splits) * size_t(N) * size_t(K + 1) * 4 : 0;
}

void launch_linear_wgrad(const WgradArgs& a, int dtype, int64_t cus, void* ws, hipStream_t s)
{
    WgradTiles tl = make_tiles(a.T, a.N, a.K, cus);
    tl.part = static_cast<float*>(ws);
    tl.part_sum = tl.part + tl.splits * a.N * a.K;
    tl.want_sum = (a.shift && tl.splits == 1) ? 2 : (a.dbias || a.shift) ? 1 : 0;
    with_dtype(dtype, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        const dim3 grid(unsigned(int64_t(tl.nt) * tl.kt * tl.splits));
        hipLaunchKernelGGL((k_wgrad<DT, kTile, kTile, 64, 64>), grid, dim3(256), 0, s, a, tl);
    });
    if (tl.splits > 1)
        hipLaunchKernelGGL(k_wgrad_join, dim3(unsigned(ceil_div(a.K, kThreads)), unsigned(a.N)),
                           dim3(kThreads), 0, s, a, tl);
}

}  // namespace iabn
