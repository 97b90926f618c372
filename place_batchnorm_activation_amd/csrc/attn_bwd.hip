// Attention backward, the probabilities recomputed from the rows' log-sum-exp:
//
//   P = exp(scale * q k^T - lse),  delta = sum_d dO * O,  dP = dO V^T,
//   dS = P * (dP - delta),  dV = P^T dO,  dQ = scale * dS K,  dK = scale * dS^T Q.
//
// Two kernels, each with its sums in registers, so that no gradient needs atomics and
// results are the same bits on every run (at the price of S and dP twice: seven products
// where one pass with atomics on dQ has five):
//   k_attn_dq    as the forward: a wave holds 32 rows (Q, dO and dQ^T in registers),
//                  S^T = K Q^T,  dP^T = V dO^T,  dQ^T += K^T dS^T
//                over tiles of keys and values in LDS; it also leaves delta for
//   k_attn_dkv   a wave holds 32 keys (K, V, dK^T and dV^T in registers),
//                  S = Q K^T,  dP = dO V^T,  dV^T += dO^T P,  dK^T += Q^T dS
//                over tiles of rows of Q and dO in LDS.  Rows of all query heads of the
//                key head's group follow one another, which sums a shared head's gradients.
//
// P and dS enter their second products in the storage type.  float16 has a range that P and
// dS leave downwards (P is 2^-15 over 32768 keys; dS has dO's scale besides): there P is
// carried times 2^10, and dS times a power of two of each lane's own, found from the
// largest magnitude so far and changed, with the sums, when a larger one would come near
// the type's end.
#include "attn_tile.hpp"

namespace iabn {

namespace {

constexpr float kUpP = 10.f;                       // f16: binary orders that P is raised by

// The factor of dS of a lane's column.
template <int DT>
struct Scaled {
    float up = DT == kF16 ? 0x1p100f : 1.f;

    // Values of 32 rows of the column (16 in each half), scaled; sums: what was made of the
    // column's values so far.
    template <int N>
    __device__ __forceinline__ void apply(f32x16_t& v, f32x16_t (&sums)[N])
    {
        if constexpr (DT == kF16) {
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(v[i]));
            most = both_max(most);
            const bool change = most * up > 16384.f;
            if (__any(change)) {
                // most * up in [2^6, 2^7): headroom of 2^7 before the next change
                const int e = max(6, int(__float_as_uint(most) >> 23));
                const float next = change ? __uint_as_float(uint32_t(127 + 127 + 6 - e) << 23) : up;
                const float f = next / up;
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int i = 0; i < 16; ++i) sums[n][i] *= f;
                up = next;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= up;
        }
    }
};

// Results 4i .. 4i + 3 times f at element d of a row; zeros for one that takes no part (its
// column may hold 0 * infinity of other columns' rows).
template <int DT>
__device__ __forceinline__ void store_scaled(char* row, int d, const f32x16_t& v, int i, float f,
                                             bool live)
{
    if (live) store4<DT>(row, d, v[4 * i] * f, v[4 * i + 1] * f, v[4 * i + 2] * f, v[4 * i + 3] * f);
    else store4<DT>(row, d, 0.f, 0.f, 0.f, 0.f);
}

// ---------------------------------------------------------------------------
// dQ and delta

template <int DT, int DP>
struct DqShape {
    static constexpr int NT = 256, KT = DT == kF32 ? 32 : 64;
    static constexpr int SLOTS = KT * TileShape<DT, DP>::NC;
    static constexpr int WAVES = DT == kF32 ? 1 : 2;
};

template <int DT, int DP>
__global__ __launch_bounds__(256, (DqShape<DT, DP>::WAVES)) void k_attn_dq(AttnArgs a, AttnGrads g,
                                                                          float* delta, int tiles)
{
    using F = DqShape<DT, DP>;
    using S = TileShape<DT, DP>;
    constexpr int ES = S::ES, KS = DP / 16, DB = DP / 32, KB = F::KT / 32;
    __shared__ uint4 lds[4 * F::SLOTS];

    const int lane = threadIdx.x % 64, h = lane / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    uint32_t head, tile;
    head_and_tile(uint32_t(a.B) * a.KV, uint32_t(tiles), head, tile);
    const int b = int(head / uint32_t(a.KV)), hk = int(head % uint32_t(a.KV));
    tile = uint32_t(tiles) - 1 - tile;             // causal rows with many keys first
    const Sequence sq = sequence_of(a, b);
    const int rows = sq.lq * a.G, all_rows = a.Sq * a.G;
    const int row0 = int(tile) * 128, r0 = row0 + wave * 32, r = r0 + lane % 32;
    const int tok = int(fast_div(uint32_t(r), a.group)), hq = hk * a.G + r - tok * a.G;
    const bool packed_q = a.q_starts != nullptr, packed_k = a.k_starts != nullptr;

    int lo = 0, hi = 0;                            // keys that the workgroup's rows see
    if (row0 < rows) {
        int x;
        visible(a, sq, int(fast_div(uint32_t(row0), a.group)), lo, x);
        visible(a, sq, int(fast_div(uint32_t(min(row0 + 128, rows) - 1), a.group)), x, hi);
    }
    int lo_min = 0, lo_max = 0, hi_min = 0, hi_max = 0;          // the wave's rows
    if (r0 < rows) {
        visible(a, sq, int(fast_div(uint32_t(r0), a.group)), lo_min, hi_min);
        visible(a, sq, int(fast_div(uint32_t(min(r0 + 32, rows) - 1), a.group)), lo_max, hi_max);
    }
    int row_lo = 0, row_hi = 0;
    float lse2 = INFINITY, dl = 0.f;               // a row that sees nothing: P = 0

    Frag<DT> q[KS], go[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        zero(q[ks]);
        zero(go[ks]);
    }
    if (r < rows) {
        visible(a, sq, tok, row_lo, row_hi);
        const char* qp = group_rows(a, a.q, b, sq, hk, ES)(r);
        const char* op = group_rows(a, a.out, b, sq, hk, ES)(r);
        const char* gp = group_rows(a, g.dout, b, sq, hk, ES)(r);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int d = 16 * ks + 8 * h;
            if (d >= a.D) continue;
            q[ks] = frag_of<DT>(qp + d * ES);
            go[ks] = frag_of<DT>(gp + d * ES);
            const Frag<DT> o = frag_of<DT>(op + d * ES);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                dl = fmaf(frag_value<DT>(go[ks], i), frag_value<DT>(o, i), dl);
        }
        const float lse = a.lse[lse_index(a, sq, b, hq, tok)];
        lse2 = lse == -INFINITY ? INFINITY : lse * kLog2eA;
    }
    dl = both_sum(dl);
    if (r < rows && h == 0) delta[(int64_t(b) * a.KV + hk) * all_rows + r] = dl;

    const char* kp = head_of(a.k, packed_k, b, sq.k0, hk, ES);
    const char* vp = head_of(a.v, packed_k, b, sq.k0, hk, ES);
    const int64_t kpitch = a.k.row * ES, vpitch = a.v.row * ES;

    f32x16_t dq[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) zero(dq[i]);
    Scaled<DT> scaled;

    TileLoad<DT, DP, F::KT, F::NT> kl, vl;
    auto k_tile = [&](int st) { return lds + st * 2 * F::SLOTS; };
    auto v_tile = [&](int st) { return lds + (st * 2 + 1) * F::SLOTS; };
    auto block = [&](int k0, int kb, int st) {     // 32 keys
        if (k0 >= hi_max || k0 + 32 <= lo_min) return;
        f32x16_t s, ds;
        zero(s);
        zero(ds);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            s = mma(row_frag<DT, DP>(k_tile(st), kb * 32, ks), q[ks], s);
            ds = mma(row_frag<DT, DP>(v_tile(st), kb * 32, ks), go[ks], ds);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float p = __builtin_amdgcn_exp2f(fmaf(s[i], a.c, -lse2));
            ds[i] = p * (ds[i] - dl);
        }
        if (k0 < lo_max || k0 + 32 > hi_min) {     // some row does not see all
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int j = k0 + 8 * (i / 4) + 4 * h + i % 4;
                if (j < row_lo || j >= row_hi) ds[i] = 0.f;
            }
        }
        scaled.apply(ds, dq);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const Frag<DT> f = results<DT>(ds, t);
#pragma unroll
            for (int i = 0; i < DB; ++i)
                dq[i] = mma(col_frag<DT, DP>(k_tile(st), kb * 32 + 16 * t, i), f, dq[i]);
        }
    };
    const int steps = hi > lo ? (hi - lo + F::KT - 1) / F::KT : 0;
    if (steps > 0) {
        kl.load(kp, kpitch, lo, hi, a.D);
        vl.load(vp, vpitch, lo, hi, a.D);
        kl.store(k_tile(0));
        vl.store(v_tile(0));
        __syncthreads();
        for (int i = 0; i < steps; ++i) {
            const int st = i & 1, k0 = lo + i * F::KT;
            const bool more = i + 1 < steps;
            if (more) kl.load(kp, kpitch, k0 + F::KT, hi, a.D);
            block(k0, 0, st);
            if (more) {
                kl.store(k_tile(st ^ 1));
                vl.load(vp, vpitch, k0 + F::KT, hi, a.D);
            }
#pragma unroll
            for (int kb = 1; kb < KB; ++kb) block(k0 + kb * 32, kb, st);
            if (more) vl.store(v_tile(st ^ 1));
            __syncthreads();
        }
    }
    // rows of a padded batch behind its length are written too, as zeros
    if (packed_q ? r >= rows : r >= all_rows) return;
    char* out = head_of(g.dq, packed_q, b, sq.q0, hq, ES) + int64_t(tok) * g.dq.row * ES;
    const float f = a.scale / scaled.up;
    const bool live = lse2 != INFINITY;            // sees a key
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = 32 * db + 8 * i + 4 * h;
            if (d < a.D) store_scaled<DT>(out, d, dq[db], i, f, live);
        }
}

// ---------------------------------------------------------------------------
// dK and dV

template <int DT, int DP>
struct DkvShape {
    static constexpr int NT = 256, QT = DT == kF32 ? 32 : 64;
    static constexpr int SLOTS = QT * TileShape<DT, DP>::NC;
};

template <int DT, int DP>
__global__ __launch_bounds__(256, 1) void k_attn_dkv(AttnArgs a, AttnGrads g, const float* delta,
                                                     int tiles)
{
    using F = DkvShape<DT, DP>;
    using S = TileShape<DT, DP>;
    constexpr int ES = S::ES, KS = DP / 16, DB = DP / 32, QB = F::QT / 32;
    __shared__ uint4 lds[4 * F::SLOTS];
    __shared__ alignas(16) float info[2][2][F::QT];              // lse * log2(e), delta

    const int lane = threadIdx.x % 64, h = lane / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    uint32_t head, tile;
    head_and_tile(uint32_t(a.B) * a.KV, uint32_t(tiles), head, tile);
    const int b = int(head / uint32_t(a.KV)), hk = int(head % uint32_t(a.KV));
    const Sequence sq = sequence_of(a, b);
    const int all_rows = a.Sq * a.G;
    const int key0 = int(tile) * 128, j0 = key0 + wave * 32, j = j0 + lane % 32;
    const bool packed_k = a.k_starts != nullptr;
    if (packed_k && key0 >= sq.lk) return;

    // rows [lo, hi) that see key x
    const int off = sq.lk - sq.lq;
    auto seen_by = [&](int x, int& lo, int& hi) {
        lo = max(0, x - off - a.right);
        hi = max(lo, min(sq.lq, x - off + a.left + 1));
        lo *= a.G;
        hi *= a.G;
    };
    int lo = 0, hi = 0;                            // the workgroup's keys
    if (key0 < sq.lk) {
        int x;
        seen_by(key0, lo, x);
        seen_by(min(key0 + 128, sq.lk) - 1, x, hi);
    }
    int lo_min = 0, lo_max = 0, hi_min = 0, hi_max = 0;          // the wave's
    if (j0 < sq.lk) {
        seen_by(j0, lo_min, hi_min);
        seen_by(min(j0 + 32, sq.lk) - 1, lo_max, hi_max);
    }
    int key_lo = 0, key_hi = 0;
    Frag<DT> k[KS], v[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        zero(k[ks]);
        zero(v[ks]);
    }
    if (j < sq.lk) {
        seen_by(j, key_lo, key_hi);
        const char* kp = head_of(a.k, packed_k, b, sq.k0, hk, ES) + int64_t(j) * a.k.row * ES;
        const char* vp = head_of(a.v, packed_k, b, sq.k0, hk, ES) + int64_t(j) * a.v.row * ES;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int d = 16 * ks + 8 * h;
            if (d >= a.D) continue;
            k[ks] = frag_of<DT>(kp + d * ES);
            v[ks] = frag_of<DT>(vp + d * ES);
        }
    }
    f32x16_t dk[DB], dv[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) {
        zero(dk[i]);
        zero(dv[i]);
    }
    Scaled<DT> scaled;

    const GroupRows qrows = group_rows(a, a.q, b, sq, hk, ES);
    const GroupRows grows = group_rows(a, g.dout, b, sq, hk, ES);
    TileLoad<DT, DP, F::QT, F::NT> ql, gl;
    float il = 0.f, id = 0.f;                      // of the next tile, one row a thread
    auto q_tile = [&](int st) { return lds + st * 2 * F::SLOTS; };
    auto g_tile = [&](int st) { return lds + (st * 2 + 1) * F::SLOTS; };
    auto fetch_info = [&](int first) {
        const int r = first + int(threadIdx.x);
        il = INFINITY;                             // no row: P = 0
        id = 0.f;
        if (threadIdx.x < F::QT && r < hi) {
            const int t = int(fast_div(uint32_t(r), a.group));
            const float lse = a.lse[lse_index(a, sq, b, hk * a.G + r - t * a.G, t)];
            if (lse != -INFINITY) il = lse * kLog2eA - (DT == kF16 ? kUpP : 0.f);
            id = delta[(int64_t(b) * a.KV + hk) * all_rows + r];
        }
    };
    auto put_info = [&](int st) {
        if (threadIdx.x < F::QT) {
            info[st][0][threadIdx.x] = il;
            info[st][1][threadIdx.x] = id;
        }
    };
    auto block = [&](int r0, int qb, int st) {     // 32 rows
        if (r0 >= hi_max || r0 + 32 <= lo_min) return;
        f32x16_t p, ds;
        zero(p);
        zero(ds);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            p = mma(row_frag<DT, DP>(q_tile(st), qb * 32, ks), k[ks], p);
            ds = mma(row_frag<DT, DP>(g_tile(st), qb * 32, ks), v[ks], ds);
        }
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 ls = *reinterpret_cast<const float4*>(&info[st][0][qb * 32 + 2 * i + 4 * h]);
            const float4 de = *reinterpret_cast<const float4*>(&info[st][1][qb * 32 + 2 * i + 4 * h]);
            const float l4[4] = {ls.x, ls.y, ls.z, ls.w}, d4[4] = {de.x, de.y, de.z, de.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[i + e] = __builtin_amdgcn_exp2f(fmaf(p[i + e], a.c, -l4[e]));
                ds[i + e] = p[i + e] * (ds[i + e] - d4[e]);
            }
        }
        if (r0 < lo_max || r0 + 32 > hi_min) {     // some key is not seen by all
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = r0 + 8 * (i / 4) + 4 * h + i % 4;
                if (r < key_lo || r >= key_hi) p[i] = ds[i] = 0.f;
            }
        }
        scaled.apply(ds, dk);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const Frag<DT> fp = results<DT>(p, t), fs = results<DT>(ds, t);
#pragma unroll
            for (int i = 0; i < DB; ++i) {
                dv[i] = mma(col_frag<DT, DP>(g_tile(st), qb * 32 + 16 * t, i), fp, dv[i]);
                dk[i] = mma(col_frag<DT, DP>(q_tile(st), qb * 32 + 16 * t, i), fs, dk[i]);
            }
        }
    };
    const int steps = hi > lo ? (hi - lo + F::QT - 1) / F::QT : 0;
    if (steps > 0) {
        ql.load_at(qrows, lo, hi, a.D);
        gl.load_at(grows, lo, hi, a.D);
        fetch_info(lo);
        ql.store(q_tile(0));
        gl.store(g_tile(0));
        put_info(0);
        __syncthreads();
        for (int i = 0; i < steps; ++i) {
            const int st = i & 1, r0 = lo + i * F::QT;
            const bool more = i + 1 < steps;
            auto fetch = [&]() {
                ql.load_at(qrows, r0 + F::QT, hi, a.D);
                gl.load_at(grows, r0 + F::QT, hi, a.D);
                fetch_info(r0 + F::QT);
            };
            // float32 has no registers for the next tile over the products, which take 16
            // times as long as loads of the same elements would leave uncovered
            if (more && DT != kF32) fetch();
#pragma unroll
            for (int qb = 0; qb < QB; ++qb) block(r0 + qb * 32, qb, st);
            if (more) {
                if (DT == kF32) fetch();
                ql.store(q_tile(st ^ 1));
                gl.store(g_tile(st ^ 1));
                put_info(st ^ 1);
            }
            __syncthreads();
        }
    }
    if (packed_k ? j >= sq.lk : j >= a.Sk) return;
    char* dkp = head_of(g.dk, packed_k, b, sq.k0, hk, ES) + int64_t(j) * g.dk.row * ES;
    char* dvp = head_of(g.dv, packed_k, b, sq.k0, hk, ES) + int64_t(j) * g.dv.row * ES;
    const float up = DT == kF16 ? 0x1p-10f : 1.f, f = a.scale * up / scaled.up;
    const bool live = key_lo < key_hi;             // is seen
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = 32 * db + 8 * i + 4 * h;
            if (d >= a.D) continue;
            store_scaled<DT>(dkp, d, dk[db], i, f, live);
            store_scaled<DT>(dvp, d, dv[db], i, up, live);
        }
}

}  // namespace

size_t attn_bwd_workspace_bytes(const AttnArgs& a, int64_t)
{
    return size_t(a.B) * size_t(a.KV) * size_t(a.G) * size_t(a.Sq) * 4;        // delta
}

void launch_attn_backward(const AttnArgs& a, const AttnGrads& g, int dtype, int64_t, void* ws,
                          hipStream_t s)
{
    float* delta = static_cast<float*>(ws);
    const int row_tiles = int(ceil_div(int64_t(a.Sq) * a.G, 128)), key_tiles = int(ceil_div(a.Sk, 128));
    const int64_t heads = int64_t(a.B) * a.KV;
    with_dtype(dtype, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        auto go = [&](auto p) {
            constexpr int DP = decltype(p)::value;
            if (row_tiles > 0)
                hipLaunchKernelGGL((k_attn_dq<DT, DP>), dim3(unsigned(heads * row_tiles)),
                                   dim3(256), 0, s, a, g, delta, row_tiles);
            if (key_tiles > 0)
                hipLaunchKernelGGL((k_attn_dkv<DT, DP>), dim3(unsigned(heads * key_tiles)),
                                   dim3(256), 0, s, a, g, delta, key_tiles);
        };
        if (a.D <= 64) go(std::integral_constant<int, 64>{});
        else if (a.D <= 96) go(std::integral_constant<int, 96>{});
        else go(std::integral_constant<int, 128>{});
    });
}

}  // namespace iabn
