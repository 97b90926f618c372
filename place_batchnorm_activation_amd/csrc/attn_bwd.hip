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
// carried times 2^14, and dS times a power of two of each lane's own, found from the
// largest magnitude so far and changed, with the sums, when a larger one would come near
// the type's end.
#include "attn_tile.hpp"

namespace iabn {

namespace {

// f16: binary orders that P, at most 1, is raised by: what is above 2^-28 keeps its digits.  The
// two orders left to the type's end are for the roundings of score and log-sum-exp, which pass
// them where |score| is beyond 2^23 and P means nothing any more.
constexpr int kUpP = 14;

// The factor of dS of a lane's column, a power of two.  It begins where no dS of float16
// tensors overflows float32, and falls to where the largest so far is far inside float16.
template <int DT>
struct Scaled {
    float up = DT == kF16 ? 0x1p60f : 1.f;

    __device__ __forceinline__ float order() const           // log2(up)
    {
        return DT == kF16 ? float(int(__float_as_uint(up) >> 23) - 127) : 0.f;
    }

    // v: values of 32 rows of the column (16 in each half) times up.  Where one comes near
    // float16's end, they and sums (what was made of the column's values so far) are brought
    // to a lower factor; whether any lane's changed.
    template <int N>
    __device__ __forceinline__ bool check(f32x16_t& v, f32x16_t (&sums)[N])
    {
        if constexpr (DT == kF16) {
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(v[i]));
            most = both_max(most);
            const bool change = most > 16384.f;
            if (__any(change)) {
                // the largest in [2^6, 2^7): headroom of 2^7 before the next change
                const int e = int(__float_as_uint(most) >> 23);
                const float f = change ? __uint_as_float(uint32_t(127 + 127 + 6 - e) << 23) : 1.f;
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int i = 0; i < 16; ++i) sums[n][i] *= f;
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] *= f;
                up *= f;
                return true;
            }
        }
        return false;
    }
};

// Results 4i .. 4i + 3 times f at element d of a row; zeros for one that takes no part (its
// column may hold 0 * infinity of other columns' rows).
template <int DT>
__device__ __forceinline__ void store_scaled(char* row, int d, const f32x16_t& v, int i, float f,
                                             bool live)
{
    if (live)
        store4<DT>(row, d, v[4 * i] * f, v[4 * i + 1] * f, v[4 * i + 2] * f, v[4 * i + 3] * f);
    else store4<DT>(row, d, 0.f, 0.f, 0.f, 0.f);
}

// A tile of 128 rows (keys) whose keys (rows) are cut among workgroups, `chunk` each: where a
// tile takes more than one, their shares of its gradients go through the workspace.
struct Parts {
    int parts, chunk;
    float* share;                     // [head][tile][part][dQ, or dK and dV][128][D]
};

template <int N>
__device__ __forceinline__ float* share_of(const Parts& pt, uint32_t head, uint32_t tiles,
                                           uint32_t tile, int part, int D)
{
    return pt.share + ((int64_t(head) * tiles + tile) * pt.parts + part) * N * 128 * D;
}

// The sum of a tile's shares of four elements, in their order.
template <int N>
__device__ __forceinline__ float4 sum_shares(const Parts& pt, uint32_t head, uint32_t tiles,
                                             uint32_t tile, int parts, int D, int at)
{
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
        const float4 u = *reinterpret_cast<const float4*>(
            share_of<N>(pt, head, tiles, tile, p, D) + at);
        v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
    }
    return v;
}

// Keys [lo, hi) that some of rows row0 .. row0 + 127 see.
__device__ __forceinline__ void seen_keys(const AttnArgs& a, const Sequence& s, int row0, int& lo,
                                          int& hi)
{
    const int rows = s.lq * a.G;
    lo = hi = 0;
    if (row0 >= rows) return;
    int x;
    visible(a, s, int(fast_div(uint32_t(row0), a.group)), lo, x);
    visible(a, s, int(fast_div(uint32_t(min(row0 + 128, rows) - 1), a.group)), x, hi);
    hi = max(lo, hi);
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
                                                                          float* delta, Parts pt,
                                                                          int tiles)
{
    using F = DqShape<DT, DP>;
    using S = TileShape<DT, DP>;
    constexpr int ES = S::ES, KS = DP / 16, DB = DP / 32, KB = F::KT / 32;
    __shared__ uint4 space[4 * F::SLOTS];
    char* const lds = reinterpret_cast<char*>(space);

    const int lane = threadIdx.x % 64, h = lane / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    uint32_t head, tile;
    head_and_tile(uint32_t(a.B) * a.KV, uint32_t(tiles), windowed(a), head, tile);
    const int b = int(head / uint32_t(a.KV)), hk = int(head % uint32_t(a.KV));
    tile = uint32_t(tiles) - 1 - tile;             // causal rows with many keys first
    const Sequence sq = sequence_of(a, b);
    const int rows = sq.lq * a.G, all_rows = a.Sq * a.G;
    const int row0 = int(tile) * 128, r0 = row0 + wave * 32, r = r0 + lane % 32;
    const int tok = int(fast_div(uint32_t(r), a.group)), hq = hk * a.G + r - tok * a.G;
    const bool packed_q = a.q_starts != nullptr;

    // the keys that some of the workgroup's rows see, that all of them see, and that some
    // of this wave's
    int lo, hi, all_lo = 0, all_hi = 0, lo_min = 0, hi_max = 0;
    seen_keys(a, sq, row0, lo, hi);
    lo = scalar(lo);
    hi = scalar(hi);
    if (row0 < rows) {
        int x;
        visible(a, sq, int(fast_div(uint32_t(row0), a.group)), x, all_hi);
        visible(a, sq, int(fast_div(uint32_t(min(row0 + 128, rows) - 1), a.group)), all_lo, x);
        all_lo = scalar(all_lo);
        all_hi = scalar(all_hi);
    }
    // this workgroup's part of the keys
    const bool shared = pt.parts > 1 && hi - lo > pt.chunk;
    if (pt.parts > 1) {
        const int64_t first = int64_t(lo) + int64_t(blockIdx.y) * pt.chunk;
        if (blockIdx.y > 0 && first >= hi) return;
        lo = int(first);
        hi = int(min(int64_t(hi), first + pt.chunk));
    }
    if (r0 < rows) {
        int x;
        visible(a, sq, int(fast_div(uint32_t(r0), a.group)), lo_min, x);
        visible(a, sq, int(fast_div(uint32_t(min(r0 + 32, rows) - 1), a.group)), x, hi_max);
        lo_min = scalar(lo_min);
        hi_max = scalar(hi_max);
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
        row_hi = max(row_lo, row_hi);
        const char* qp = group_row(a, a.q, b, sq, hk, r, ES);
        const char* op = group_row(a, a.out, b, sq, hk, r, ES);
        const char* gp = group_row(a, g.dout, b, sq, hk, r, ES);
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
    if (r < rows && h == 0 && blockIdx.y == 0) delta[(int64_t(b) * a.KV + hk) * all_rows + r] = dl;

    using T = Tiles<DT, DP, F::KT, F::NT>;
    const T keys = key_tiles<T>(a, a.k, b, sq, hk, ES), vals = key_tiles<T>(a, a.v, b, sq, hk, ES);
    const RowFrags<DT, DP> rf;
    const ColFrags<DT, DP> cf;

    f32x16_t dq[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) zero(dq[i]);
    Scaled<DT> scaled;
    float base = lse2 - scaled.order();            // P comes times the factor of dS

    auto tile_at = [&](int st, int v) { return lds + (2 * st + v) * F::SLOTS * 16; };
    auto fetch = [&](int i, int st) __attribute__((always_inline)) {
        keys.load(tile_at(st, 0), lo + i * F::KT, hi, a.D);
        vals.load(tile_at(st, 1), lo + i * F::KT, hi, a.D);
    };
    // A tile, 32 keys after another: a block's exponentials among the next one's products, and
    // fragments read ahead of theirs.
    auto step_of = [&](int k0, int st, auto some) __attribute__((always_inline)) {
        const char *K = tile_at(st, 0), *V = tile_at(st, 1);
        f32x16_t s[KB], ds[KB];
        const uint32_t at = uint32_t(k0 + 4 * h - row_lo), n = uint32_t(row_hi - row_lo);
        auto probs = [&](int kb, int from, int to) {             // dS of some of a block
#pragma unroll
            for (int i = from; i < to; ++i) {
                const float p = __builtin_amdgcn_exp2f(fmaf(s[kb][i], a.c, -base));
                ds[kb][i] = p * (ds[kb][i] - dl);
                if (decltype(some)::value && at + uint32_t(kb * 32 + 8 * (i / 4) + i % 4) >= n)
                    ds[kb][i] = 0.f;
            }
        };
        Frag<DT> f[2][2];
        auto read = [&](int g) {
            f[g & 1][0] = rf.read(K, g / KS * 32, g % KS);
            f[g & 1][1] = rf.read(V, g / KS * 32, g % KS);
        };
        read(0);
#pragma unroll
        for (int g = 0; g < KB * KS; ++g) {
            const int kb = g / KS, ks = g % KS;
            if (g + 1 < KB * KS) read(g + 1);
            __builtin_amdgcn_sched_barrier(0);
            if (ks == 0) {
                zero(s[kb]);
                zero(ds[kb]);
            }
            s[kb] = mma(f[g & 1][0], q[ks], s[kb]);
            ds[kb] = mma(f[g & 1][1], go[ks], ds[kb]);
            if (kb > 0) probs(kb - 1, 16 * ks / KS, 16 * (ks + 1) / KS);
        }
        constexpr int CS = DB % 2 == 0 ? 2 : 3, CG = 2 * DB / CS;          // of a block
        Frag<DT> c[2][CS];
        auto read_c = [&](int g) {
#pragma unroll
            for (int i = 0; i < CS; ++i)
                c[g & 1][i] = cf.read(K, (g * CS + i) / DB * 16, (g * CS + i) % DB);
        };
        read_c(0);
        if (KB == 1) probs(0, 0, 16);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            if (scaled.check(ds[kb], dq)) base = lse2 - scaled.order();
            Frag<DT> x = results<DT>(ds[kb], 0);
#pragma unroll
            for (int g = 0; g < CG; ++g) {
                if (kb * CG + g + 1 < KB * CG) read_c(kb * CG + g + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < CS; ++i) {
                    const int t = (g * CS + i) / DB, db = (g * CS + i) % DB;
                    if (db == 0 && t == 1) x = results<DT>(ds[kb], 1);
                    dq[db] = mma(c[(kb * CG + g) & 1][i], x, dq[db]);
                }
                if (KB > 1 && kb == KB - 2) probs(KB - 1, 16 * g / CG, 16 * (g + 1) / CG);
            }
        }
    };
    const int steps = hi > lo ? (hi - lo + F::KT - 1) / F::KT : 0;
    if (steps > 0) {
        if (a.D < DP) {
            clear<F::NT>(lds, 4 * F::SLOTS * 16);
            __syncthreads();
        }
        fetch(0, 0);
        auto step = [&](int i, auto st, auto some) __attribute__((always_inline)) {
            arrived<>();
            __syncthreads();
            if (i + 1 < steps) fetch(i + 1, 1 - st);
            const int k0 = lo + i * F::KT;
            if (!decltype(some)::value || (k0 < hi_max && k0 + F::KT > lo_min))
                step_of(k0, st, some);
        };
        // pairs of tiles that all rows see whole in a loop of their own, as in the forward
        auto whole = [&](int i) {
            return lo + i * F::KT >= all_lo && lo + (i + 1) * F::KT <= min(hi, all_hi);
        };
        for (int i = 0; i < steps;) {
            if ((i & 1) == 0) {
                while (i + 1 < steps && whole(i) && whole(i + 1)) {
                    step(i, std::integral_constant<int, 0>{}, std::false_type{});
                    step(i + 1, std::integral_constant<int, 1>{}, std::false_type{});
                    i += 2;
                }
                if (i >= steps) break;
            }
            step(i, i & 1, std::true_type{});
            ++i;
        }
    }
    if (shared) {
        float* share = share_of<1>(pt, head, uint32_t(tiles), tile, int(blockIdx.y), a.D) +
                       (r - row0) * a.D;
        if (r >= rows) return;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = 32 * db + 8 * i + 4 * h;
                if (d < a.D)
                    store_scaled<kF32>(reinterpret_cast<char*>(share), d, dq[db], i,
                                       a.scale / scaled.up, true);
            }
        return;
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

// Adds the shares of the row tiles whose keys were parted: a thread 4 elements of a row.
template <int DT>
__global__ __launch_bounds__(256) void k_attn_dq_join(AttnArgs a, AttnGrads g, Parts pt, int tiles)
{
    constexpr int ES = DT == kF32 ? 4 : 2;
    const uint32_t head = blockIdx.x / uint32_t(tiles), tile = blockIdx.x % uint32_t(tiles);
    const int b = int(head / uint32_t(a.KV)), hk = int(head % uint32_t(a.KV));
    const Sequence sq = sequence_of(a, b);
    const int row0 = int(tile) * 128, quads = a.D / 4, all_rows = a.Sq * a.G, rows = sq.lq * a.G;
    int lo, hi;
    seen_keys(a, sq, row0, lo, hi);
    if (hi - lo <= pt.chunk) return;
    const int parts = (hi - lo + pt.chunk - 1) / pt.chunk;
    const int end = min(128, (a.q_starts ? rows : all_rows) - row0);
    const int i = int(blockIdx.y) * 256 + int(threadIdx.x);
    if (i < end * quads) {
        const int r = i / quads, d = i % quads * 4;
        const int tok = int(fast_div(uint32_t(row0 + r), a.group));
        const int hq = hk * a.G + row0 + r - tok * a.G;
        // a row that sees no key holds 0 * infinity of its tile's others
        const bool live = row0 + r < rows && a.lse[lse_index(a, sq, b, hq, tok)] != -INFINITY;
        const float4 v = sum_shares<1>(pt, head, uint32_t(tiles), tile, live ? parts : 0, a.D,
                                       r * a.D + d);
        char* out = head_of(g.dq, a.q_starts != nullptr, b, sq.q0, hq, ES) +
                    int64_t(tok) * g.dq.row * ES;
        store4<DT>(out, d, v.x, v.y, v.z, v.w);
    }
}

// ---------------------------------------------------------------------------
// dK and dV

// Rows [lo, hi) of the group that see key x.
__device__ __forceinline__ void seen_by(const AttnArgs& a, const Sequence& s, int x, int& lo,
                                        int& hi)
{
    const int off = s.lk - s.lq;
    lo = max(0, x - off - a.right);
    hi = max(lo, min(s.lq, x - off + a.left + 1));
    lo *= a.G;
    hi *= a.G;
}

template <int DT, int DP>
struct DkvShape {
    static constexpr int NT = 256;
    // 16-bit types keep the values in LDS instead of registers and rows in tiles of 8 KB, so
    // that two workgroups run on a CU
    static constexpr bool VL = DT != kF32;
    static constexpr int QT = DT == kF32 || DP > 64 ? 32 : 64;
    static constexpr int TILE = QT * TileShape<DT, DP>::PITCH;
    static constexpr int VTILE = VL ? 128 * TileShape<DT, DP>::PITCH : 0;
    static constexpr int WAVES = VL ? 2 : 1;
};

template <int DT, int DP>
__global__ __launch_bounds__(256, (DkvShape<DT, DP>::WAVES)) void k_attn_dkv(AttnArgs a,
                                                                            AttnGrads g,
                                                                            const float* delta,
                                                                            Parts pt,
                                                                            int tiles)
{
    using F = DkvShape<DT, DP>;
    using S = TileShape<DT, DP>;
    constexpr int ES = S::ES, KS = DP / 16, DB = DP / 32, QB = F::QT / 32;
    __shared__ uint4 space[(4 * F::TILE + F::VTILE) / 16];
    __shared__ alignas(16) float info[2][2][F::QT];              // lse * log2(e), delta
    char* const lds = reinterpret_cast<char*>(space);

    const int lane = threadIdx.x % 64, h = lane / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    uint32_t head, tile;
    head_and_tile(uint32_t(a.B) * a.KV, uint32_t(tiles), windowed(a), head, tile);
    const int b = int(head / uint32_t(a.KV)), hk = int(head % uint32_t(a.KV));
    const Sequence sq = sequence_of(a, b);
    const int all_rows = a.Sq * a.G;
    const int key0 = int(tile) * 128, j0 = key0 + wave * 32, j = j0 + lane % 32;
    const bool packed_k = a.k_starts != nullptr;
    if (packed_k && key0 >= sq.lk) return;

    // the rows that see some of the workgroup's keys, all of them, and some of this wave's
    int lo = 0, hi = 0, all_lo = 0, all_hi = 0, lo_min = 0, hi_max = 0;
    if (key0 < sq.lk) {
        seen_by(a, sq, key0, lo, all_hi);
        seen_by(a, sq, min(key0 + 128, sq.lk) - 1, all_lo, hi);
        lo = scalar(lo);
        hi = scalar(hi);
        all_lo = scalar(all_lo);
        all_hi = scalar(all_hi);
    }
    if (j0 < sq.lk) {
        int x;
        seen_by(a, sq, j0, lo_min, x);
        seen_by(a, sq, min(j0 + 32, sq.lk) - 1, x, hi_max);
        lo_min = scalar(lo_min);
        hi_max = scalar(hi_max);
    }
    // this workgroup's part of the rows
    bool shared = false;
    if (pt.parts > 1) {
        shared = hi - lo > pt.chunk;
        const int64_t end = int64_t(hi) - int64_t(blockIdx.y) * pt.chunk;
        if (blockIdx.y > 0 && end <= lo) return;
        hi = int(end);
        lo = int(max(int64_t(lo), end - pt.chunk));
    }
    int key_lo = 0, key_hi = 0;
    Frag<DT> k[KS], v[F::VL ? 1 : KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        zero(k[ks]);
        if constexpr (!F::VL) zero(v[ks]);
    }
    if (j < sq.lk) {
        seen_by(a, sq, j, key_lo, key_hi);
        const char* kp = head_of(a.k, packed_k, b, sq.k0, hk, ES) + int64_t(j) * a.k.row * ES;
        const char* vp = head_of(a.v, packed_k, b, sq.k0, hk, ES) + int64_t(j) * a.v.row * ES;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int d = 16 * ks + 8 * h;
            if (d >= a.D) continue;
            k[ks] = frag_of<DT>(kp + d * ES);
            if constexpr (!F::VL) v[ks] = frag_of<DT>(vp + d * ES);
        }
    }
    f32x16_t dk[DB], dv[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) {
        zero(dk[i]);
        zero(dv[i]);
    }
    Scaled<DT> scaled;

    using T = Tiles<DT, DP, F::QT, F::NT>;
    const T qrows = group_tiles<T>(a, a.q, b, sq, hk, ES);
    const T grows = group_tiles<T>(a, g.dout, b, sq, hk, ES);
    const RowFrags<DT, DP> rows_at;
    const ColFrags<DT, DP> cols_at;
    char* const values = lds + 4 * F::TILE;
    float il = 0.f, id = 0.f;                      // of the next tile, one row a thread
    auto tile_at = [&](int st, int v) { return lds + (2 * st + v) * F::TILE; };
    // From the last rows to the first: under a causal mask key tiles begin at different rows, and
    // all of a head's workgroups read the same ones from L2 only if they start at the end.
    const int steps = hi > lo ? (hi - lo + F::QT - 1) / F::QT : 0;
    auto row_of = [&](int i) { return lo + (steps - 1 - i) * F::QT; };
    auto fetch = [&](int i, int st) __attribute__((always_inline)) {
        const int first = row_of(i);
        qrows.load(tile_at(st, 0), first, hi, a.D);
        grows.load(tile_at(st, 1), first, hi, a.D);
        const int r = first + int(threadIdx.x);
        il = INFINITY;                             // no row: P = 0
        id = 0.f;
        if (threadIdx.x < F::QT && r < hi) {
            const int t = int(fast_div(uint32_t(r), a.group));
            const float lse = a.lse[lse_index(a, sq, b, hk * a.G + r - t * a.G, t)];
            if (lse != -INFINITY) il = lse * kLog2eA - (DT == kF16 ? float(kUpP) : 0.f);
            id = delta[(int64_t(b) * a.KV + hk) * all_rows + r];
        }
    };
    auto step_of = [&](int r0, int st, auto some) __attribute__((always_inline)) {
        const char *Q = tile_at(st, 0), *O = tile_at(st, 1);
        const uint32_t n = uint32_t(key_hi - key_lo);
        // the addresses' XORs are made anew each time: kept, they would take the registers
        // that the sums need
        RowFrags<DT, DP> rf = rows_at;
        ColFrags<DT, DP> cf = cols_at;
        asm volatile("" : "+v"(rf.at), "+v"(cf.at));
#pragma unroll
        for (int qb = 0; qb < QB; ++qb) {          // 32 rows after another
            const uint32_t at = uint32_t(r0 + qb * 32 + 4 * h - key_lo);
            f32x16_t p, ds;
            zero(p);
            zero(ds);
            Frag<DT> f[2][2], w[2];
            auto read = [&](int ks) {
                f[ks & 1][0] = rf.read(Q, qb * 32, ks);
                f[ks & 1][1] = rf.read(O, qb * 32, ks);
                if constexpr (F::VL) w[ks & 1] = rf.read(values, wave * 32, ks);
            };
            read(0);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                if (ks + 1 < KS) read(ks + 1);
                __builtin_amdgcn_sched_barrier(0);
                p = mma(f[ks & 1][0], k[ks], p);
                if constexpr (F::VL) ds = mma(f[ks & 1][1], w[ks & 1], ds);
                else ds = mma(f[ks & 1][1], v[ks], ds);
            }
            Frag<DT> c[2][2];
            auto read_c = [&](int i) {             // element block i % DB of 16 rows
                c[i & 1][0] = cf.read(O, qb * 32 + i / DB * 16, i % DB);
                c[i & 1][1] = cf.read(Q, qb * 32 + i / DB * 16, i % DB);
            };
            read_c(0);
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const int at4 = qb * 32 + 2 * i + 4 * h;
                const float4 ls = *reinterpret_cast<const float4*>(&info[st][0][at4]);
                const float4 de = *reinterpret_cast<const float4*>(&info[st][1][at4]);
                const float l4[4] = {ls.x, ls.y, ls.z, ls.w}, d4[4] = {de.x, de.y, de.z, de.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[i + e] = __builtin_amdgcn_exp2f(fmaf(p[i + e], a.c, -l4[e]));
                    const float d = ds[i + e] - d4[e];
                    ds[i + e] = p[i + e] * (DT == kF16 ? d * scaled.up : d);
                    if (decltype(some)::value && at + uint32_t(2 * i + e) >= n)
                        p[i + e] = ds[i + e] = 0.f;
                }
            }
            scaled.check(ds, dk);
            Frag<DT> fp, fs;
#pragma unroll
            for (int i = 0; i < 2 * DB; ++i) {
                const int t = i / DB, db = i % DB;
                if (i + 1 < 2 * DB) read_c(i + 1);
                __builtin_amdgcn_sched_barrier(0);
                if (db == 0) {
                    fp = results<DT>(p, t);
                    fs = results<DT>(ds, t);
                }
                dv[db] = mma(c[i & 1][0], fp, dv[db]);
                dk[db] = mma(c[i & 1][1], fs, dk[db]);
            }
        }
    };
    if (steps > 0) {
        if (a.D < DP) {
            clear<F::NT>(lds, 4 * F::TILE + F::VTILE);
            __syncthreads();
        }
        if constexpr (F::VL) {
            using TV = Tiles<DT, DP, 128, F::NT>;
            key_tiles<TV>(a, a.v, b, sq, hk, ES).load(values, key0, sq.lk, a.D);
        }
        fetch(0, 0);
        auto step = [&](int i, auto st, auto some) __attribute__((always_inline)) {
            if (threadIdx.x < F::QT) {
                info[st][0][threadIdx.x] = il;
                info[st][1][threadIdx.x] = id;
            }
            arrived<>();
            __syncthreads();
            if (i + 1 < steps) fetch(i + 1, 1 - st);
            const int r0 = row_of(i);
            if (!decltype(some)::value || (r0 < hi_max && r0 + F::QT > lo_min))
                step_of(r0, st, some);
        };
        // pairs of tiles whose rows see all keys in a loop of their own, as in the forward
        auto whole = [&](int i) {
            return row_of(i) >= all_lo && row_of(i) + F::QT <= min(hi, all_hi);
        };
        for (int i = 0; i < steps;) {
            if ((i & 1) == 0) {
                while (i + 1 < steps && whole(i) && whole(i + 1)) {
                    step(i, std::integral_constant<int, 0>{}, std::false_type{});
                    step(i + 1, std::integral_constant<int, 1>{}, std::false_type{});
                    i += 2;
                }
                if (i >= steps) break;
            }
            step(i, i & 1, std::true_type{});
            ++i;
        }
    }
    const float up = DT == kF16 ? 1.f / (1 << kUpP) : 1.f, f = a.scale * up / scaled.up;
    if (shared) {
        if (j >= sq.lk) return;
        float* share = share_of<2>(pt, head, uint32_t(tiles), tile, int(blockIdx.y), a.D) +
                       (j - key0) * a.D;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = 32 * db + 8 * i + 4 * h;
                if (d >= a.D) continue;
                char* p = reinterpret_cast<char*>(share);
                store_scaled<kF32>(p, d, dk[db], i, f, true);
                store_scaled<kF32>(p + 512 * a.D, d, dv[db], i, up, true);
            }
        return;
    }
    if (packed_k ? j >= sq.lk : j >= a.Sk) return;
    char* dkp = head_of(g.dk, packed_k, b, sq.k0, hk, ES) + int64_t(j) * g.dk.row * ES;
    char* dvp = head_of(g.dv, packed_k, b, sq.k0, hk, ES) + int64_t(j) * g.dv.row * ES;
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

// Adds the shares of the key tiles whose rows were parted, in their order: a thread 4
// elements of a key.
template <int DT>
__global__ __launch_bounds__(256) void k_attn_dkv_join(AttnArgs a, AttnGrads g, Parts pt,
                                                       int tiles)
{
    constexpr int ES = DT == kF32 ? 4 : 2;
    const uint32_t head = blockIdx.x / uint32_t(tiles), tile = blockIdx.x % uint32_t(tiles);
    const int b = int(head / uint32_t(a.KV)), hk = int(head % uint32_t(a.KV));
    const Sequence sq = sequence_of(a, b);
    const int key0 = int(tile) * 128, quads = a.D / 4;
    if (key0 >= sq.lk) return;
    int lo, hi, x;
    seen_by(a, sq, key0, lo, x);
    seen_by(a, sq, min(key0 + 128, sq.lk) - 1, x, hi);
    if (hi - lo <= pt.chunk) return;
    const int parts = (hi - lo + pt.chunk - 1) / pt.chunk;
    const bool packed_k = a.k_starts != nullptr;
    const int end = min(128, (packed_k ? sq.lk : a.Sk) - key0);
    const int i = int(blockIdx.y) * 256 + int(threadIdx.x), which = int(blockIdx.z);
    if (i < end * quads) {
        const int j = i / quads, d = i % quads * 4;
        seen_by(a, sq, key0 + j, lo, hi);
        const bool live = key0 + j < sq.lk && lo < hi;
        const float4 v = sum_shares<2>(pt, head, uint32_t(tiles), tile, live ? parts : 0, a.D,
                                       (which * 128 + j) * a.D + d);
        const Heads& out = which ? g.dv : g.dk;
        store4<DT>(head_of(out, packed_k, b, sq.k0, hk, ES) + int64_t(key0 + j) * out.row * ES, d,
                   v.x, v.y, v.z, v.w);
    }
}

// Workgroups of the keys that a row tile can see: two for every CU in all, each part at least 128
// keys.
Parts dq_parts(const AttnArgs& a, int64_t cus)
{
    Parts pt{};
    const int64_t wgs = int64_t(a.B) * a.KV * ceil_div(int64_t(a.Sq) * a.G, 128);
    const int64_t want = wgs > 0 && wgs < cus ? ceil_div(2 * cus, wgs) : 1;
    const int64_t keys = seen_most(a, 128 / a.G + 2, a.Sk);
    const int64_t parts = max64(1, min64(want, keys / 128));
    pt.chunk = int(max64(1, ceil_div(ceil_div(keys, parts), 64)) * 64);
    pt.parts = int(max64(1, ceil_div(keys, pt.chunk)));
    return pt;
}

// Workgroups of the rows that can see a key tile: two for every CU in all, and twice as many where
// a mask of one side gives key tiles different numbers of rows, which two resident workgroups a
// CU do not even out (twice 4096 causal tokens of 32 heads on 8: 890 us in one part, 640 in two
// and 28 to join them); each part at least 128 rows, or 256 of the few that a window of two sides
// shows (2 x 4096 tokens, 128 to either side, 4 heads of 64: the backward 33 us in one part, 47
// in three).  Parts of what a window shows instead of all rows: 16384 tokens, the last 1024, 8
// heads on one of 128, 556 us and 356.
Parts dkv_parts(const AttnArgs& a, int64_t cus)
{
    Parts pt{};
    const int64_t wgs = int64_t(a.B) * a.KV * ceil_div(a.Sk, 128);
    const int64_t rows = seen_most(a, 128, a.Sq) * a.G;
    const bool window = a.left < kAttnMaxLen && a.right < kAttnMaxLen;
    const bool uneven = !window && (a.left < kAttnMaxLen || a.right < kAttnMaxLen);
    const int64_t want = wgs > 0 ? ceil_div((uneven ? 4 : 2) * cus, wgs) : 1;
    const int64_t parts = max64(1, min64(want, rows / (window ? 256 : 128)));
    // whole tiles of rows and whole groups
    const int64_t unit = int64_t(64) * a.G;
    const int64_t chunk = max64(1, (ceil_div(rows, parts) + unit / 2) / unit) * unit;
    pt.parts = int(max64(1, ceil_div(rows, chunk)));
    pt.chunk = int(min64(chunk, max64(1, rows)));
    return pt;
}

// delta [B][KV][rows], the shares of dQ, the shares of dK and dV
struct BwdSpace {
    Parts dq, dkv;
    size_t bytes;
};

BwdSpace bwd_space(const AttnArgs& a, int64_t cus, void* ws)
{
    BwdSpace w{dq_parts(a, cus), dkv_parts(a, cus), 0};
    const size_t heads = size_t(a.B) * a.KV, tile = size_t(128) * a.D * 4;
    const int64_t rows = int64_t(a.Sq) * a.G;
    auto take = [&](size_t bytes) {
        char* p = static_cast<char*>(ws) + w.bytes;
        w.bytes += (bytes + 15) / 16 * 16;
        return reinterpret_cast<float*>(p);
    };
    take(heads * size_t(rows) * 4);
    w.dq.share = take(w.dq.parts > 1 ? heads * ceil_div(rows, 128) * w.dq.parts * tile : 0);
    w.dkv.share = take(w.dkv.parts > 1 ? heads * ceil_div(a.Sk, 128) * w.dkv.parts * 2 * tile : 0);
    return w;
}

}  // namespace

size_t attn_bwd_workspace_bytes(const AttnArgs& a, int64_t cus)
{
    return bwd_space(a, cus, nullptr).bytes;
}

void launch_attn_backward(const AttnArgs& a, const AttnGrads& g, int dtype, int64_t cus, void* ws,
                          hipStream_t s)
{
    float* delta = static_cast<float*>(ws);
    const BwdSpace w = bwd_space(a, cus, ws);
    const int row_tiles = int(ceil_div(int64_t(a.Sq) * a.G, 128));
    const int key_tiles = int(ceil_div(a.Sk, 128));
    const int64_t heads = int64_t(a.B) * a.KV;
    const unsigned row_wgs = unsigned(heads * row_tiles), key_wgs = unsigned(heads * key_tiles);
    const unsigned slices = unsigned(ceil_div(128 * (a.D / 4), 256));
    with_dtype(dtype, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        auto go = [&](auto p) {
            constexpr int DP = decltype(p)::value;
            if (row_tiles > 0)
                hipLaunchKernelGGL((k_attn_dq<DT, DP>), dim3(row_wgs, unsigned(w.dq.parts)),
                                   dim3(256), 0, s, a, g, delta, w.dq, row_tiles);
            if (key_tiles > 0)
                hipLaunchKernelGGL((k_attn_dkv<DT, DP>), dim3(key_wgs, unsigned(w.dkv.parts)),
                                   dim3(256), 0, s, a, g, delta, w.dkv, key_tiles);
        };
        if (a.D <= 64) go(std::integral_constant<int, 64>{});
        else if (a.D <= 96) go(std::integral_constant<int, 96>{});
        else go(std::integral_constant<int, 128>{});
        if (row_tiles > 0 && w.dq.parts > 1)
            hipLaunchKernelGGL((k_attn_dq_join<DT>), dim3(row_wgs, slices), dim3(256), 0, s, a, g,
                               w.dq, row_tiles);
        if (key_tiles > 0 && w.dkv.parts > 1)
            hipLaunchKernelGGL((k_attn_dkv_join<DT>), dim3(key_wgs, slices, 2), dim3(256), 0, s, a,
                               g, w.dkv, key_tiles);
    });
}

}  // namespace iabn
