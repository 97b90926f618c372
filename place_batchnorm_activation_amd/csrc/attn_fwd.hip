// Attention forward: out = softmax(scale * q k^T) v over the visible keys, and the rows'
// log-sum-exp for the backward.
//
// One pass over the keys with the running maximum m and sum l of each row:
//   S^T = K Q^T,  P^T = exp(S^T - m),  O^T += V^T P^T,
// O and l scaled by exp(m_old - m_new) when m grows, which is left until it grows by more
// than a factor (Range) that P then stays below; the sums are fp32.  A wave holds 32 rows
// (rows of a key head: attn.hpp) in registers, Q and O^T both; the statistics are scalars of
// the lane, one exchange with the other half of the wave a tile.
//
// P is rounded to the storage type for its product with V, which the matrix units take in one
// type only (in two parts it would keep 16 digits, for half as many products again): half a
// step a term, as the output's own rounding.  l sums it as it was.
//
// Many rows: a workgroup of 4 waves x 32 rows shares the tiles of keys in LDS, two stages,
// the next tile's loads in flight.  At most 32 rows (single tokens): workgroups of one wave,
// three stages, no barriers: what counts there is bytes in flight (96 KB a CU; with 64 KB in
// groups of four waves that share their tiles the same caches were read at 4.6 instead of
// 5.1 TB/s), or of four waves that part the keys and join their shares in LDS (keys_inside).  Few
// workgroups: the keys are cut among several, whose shares (O, m, l in fp32) go through
// the workspace and are joined by a second kernel.
#include "attn_tile.hpp"

namespace iabn {

namespace {
// Binary orders that the running maximum may lag behind, and that P is raised by.  bfloat16 and
// float32 have float32's range.  float16 loses digits below 2^-14 and everything below 2^-25,
// and over long caches with one large score (of a key whose value is near zero) the small
// probabilities are the result: there P is raised as far as the lag leaves room (to 2^15), so that
// what is more than 2^-25 of a row's largest (17.3 below its score) keeps its digits, and the
// next ten orders some of them.  A shorter lag costs more changes of the sums: us for lag and
// raise 8 and 0, 8 and 7, 4 and 11, 2 and 13: 2 x 4096 causal tokens, 32 heads on 8 of 128, 294,
// 294, 295, 298, with scores spread four times as wide 289, 291, 297, 300; 4 x 2048 tokens, 16
// heads of 64, 89.5, 89.4, 89.3, 90.8; single tokens the same.
template <int DT>
struct Range {
    static constexpr float lazy = DT == kF16 ? 4.f : 8.f, up = DT == kF16 ? 11.f : 0.f;

    // log2 of what P = exp2(s c - base) is relative to, for a maximum of m.  float16: rounded up,
    // so that P passes 2^15 at no size of the scores.
    static __device__ __forceinline__ float base(float m, float c)
    {
        if (m == -INFINITY) return 0.f;
        const float b = fmaf(m, c, -up);
        return DT == kF16 ? fmaf(fabsf(b), 0x1p-23f, b) : b;
    }
};

// A row's statistics for its shares and its log-sum-exp: sum exp(S) = 2^x * y.
template <int DT>
__device__ __forceinline__ float2 share_stats(float m, float l, float c)
{
    return make_float2(m == -INFINITY ? -INFINITY : Range<DT>::base(m, c), l);
}
__device__ __forceinline__ float lse_of(float2 st)
{
    return st.y == 0.f ? -INFINITY : (st.x + __builtin_amdgcn_logf(st.y)) * kLn2A;
}

struct FwdSplit {
    int splits, chunk;               // workgroups of the keys, and (at least) keys of each
    float places;                    // 0, or workgroups of a key head that all sequences share
    float* o;                        // [split][row][D]
    float2* ml;                      // [split][row]: share_stats
    int64_t rows;                    // B * KV * Sq * G
    bool inside;                     // parts of the keys are waves of one workgroup
};

// WQ waves of 32 rows, or KW waves with a part of the same rows' keys each.
template <int DT, int DP, int WQ, int KW>
struct FwdShape {
    static constexpr int NT = 64 * WQ;
    static constexpr int KT = WQ == 1 || DT == kF32 ? 32 : 64;   // keys of a tile
    static constexpr int TILE = KT * TileShape<DT, DP>::PITCH;
    static constexpr int STAGES = WQ == 1 && KW == 1 && DT != kF32 ? 3 : 2;
    static constexpr int LDS = STAGES * 2 * TILE;                // of the waves that share it
    static_assert(LDS >= 32 * DP * 4, "a wave's share of the results takes its tiles' place");
    static constexpr int WAVES = WQ == 1 || DT == kF32 ? 1 : 2;  // of a SIMD
};

// Keys of a part with which few rows' sequences of their own lengths take about `places`
// workgroups of a key head in all; every sequence then has parts of one size (k_attn_fwd).  (us
// for one token over 8 caches, 8 key heads of 128, with 16 parts of a fixed size, and with these:
// all of 32768 keys 226, 196; of random lengths up to that 175, 112, and 143 if parts do not move
// on among the CUs (head_and_tile); one of 32768 beside 7 of 200 79, 61; 20 caches of random
// lengths up to 6000 82, 57; 32 of 4096 118, 105.)
__device__ __forceinline__ int even_chunk(const AttnArgs& a, float places)
{
    float all = 0.f;
    for (int i = int(threadIdx.x) % 64; i < a.B; i += 64)
        all += float(min(lane_sequence(a, i).lk, a.left + a.right + a.Sq));
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) all += __shfl_xor(all, x, 64);
    return scalar((int(all / places) + 64) / 64 * 64);
}

// The results of one row, d = d0 .. d0 + 3 of it at a time.
template <int DT>
struct RowOut {
    char* out;                        // NULL: no such row
    float* part;                      // instead of out, its share
    float inv;

    __device__ __forceinline__ void put(int d, float a, float b, float c, float e) const
    {
        if (part) store4<kF32>(reinterpret_cast<char*>(part), d, a, b, c, e);
        else if (inv == 0.f) store4<DT>(out, d, 0.f, 0.f, 0.f, 0.f);       // sees no key
        else store4<DT>(out, d, a * inv, b * inv, c * inv, e * inv);
    }
};

template <int DT, int DP, int WQ, int KW>
__global__ __launch_bounds__(64 * WQ * KW, (FwdShape<DT, DP, WQ, KW>::WAVES)) void k_attn_fwd(
    AttnArgs a, FwdSplit sp, int tiles)
{
    using F = FwdShape<DT, DP, WQ, KW>;
    static_assert(WQ == 1 || KW == 1, "waves for rows or for keys");
    using S = TileShape<DT, DP>;
    constexpr int ES = S::ES, KS = DP / 16, DB = DP / 32, KB = F::KT / 32;
    __shared__ uint4 space[KW * F::LDS / 16];

    const int lane = threadIdx.x % 64, h = lane / 32;
    const int id_wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wave = KW > 1 ? 0 : id_wave, part = KW > 1 ? id_wave : int(blockIdx.y);
    char* const lds = reinterpret_cast<char*>(space) + (KW > 1 ? part * F::LDS : 0);
    uint32_t head, tile;
    head_and_tile(uint32_t(a.B) * a.KV, uint32_t(tiles), windowed(a), head, tile,
                  WQ == 1 ? blockIdx.y : 0);
    const int b = int(head / uint32_t(a.KV)), hk = int(head % uint32_t(a.KV));
    tile = uint32_t(tiles) - 1 - tile;             // causal rows with many keys first
    const Sequence sq = sequence_of(a, b);
    const int rows = sq.lq * a.G, all_rows = a.Sq * a.G;
    const int row0 = int(tile) * 32 * WQ, r0 = row0 + wave * 32, r = r0 + lane % 32;
    const int tok = int(fast_div(uint32_t(r), a.group)), hq = hk * a.G + r - tok * a.G;
    const bool packed_q = a.q_starts != nullptr;

    // the keys that some of the workgroup's rows see, that all of them see, and that some
    // of this wave's
    int lo = 0, hi = 0, all_lo = 0, all_hi = 0;
    if (row0 < rows) {
        visible(a, sq, int(fast_div(uint32_t(row0), a.group)), lo, all_hi);
        visible(a, sq, int(fast_div(uint32_t(min(row0 + 32 * WQ, rows) - 1), a.group)), all_lo, hi);
        lo = scalar(lo);
        hi = scalar(hi);
        all_lo = scalar(all_lo);
        all_hi = scalar(all_hi);
    }
    int lo_min = 0, hi_max = 0;
    if (r0 < rows) {
        int x;
        visible(a, sq, int(fast_div(uint32_t(r0), a.group)), lo_min, x);
        visible(a, sq, int(fast_div(uint32_t(min(r0 + 32, rows) - 1), a.group)), x, hi_max);
        lo_min = scalar(lo_min);
        hi_max = scalar(hi_max);
    }
    int row_lo = 0, row_hi = 0;
    if (r < rows) {
        visible(a, sq, tok, row_lo, row_hi);
        row_hi = max(row_lo, row_hi);
    }

    if (KW > 1 || sp.splits > 1) {                 // this workgroup's, or wave's, part of them
        int chunk = KW > 1 ? (max(0, hi - lo) + 32 * KW - 1) / (32 * KW) * 32 : sp.chunk;
        if (WQ == 1 && KW == 1 && sp.places > 0.f && hi > lo) {
            chunk = max(chunk, even_chunk(a, sp.places));
            const int n = (hi - lo + chunk - 1) / chunk;
            chunk = ((hi - lo + n - 1) / n + 63) / 64 * 64;
        }
        const int64_t first = int64_t(lo) + int64_t(part) * chunk;
        hi = first < hi ? int(min(int64_t(hi), first + chunk)) : lo;
        lo = first < hi ? int(first) : hi;
    }
    const int steps = hi > lo ? (hi - lo + F::KT - 1) / F::KT : 0;

    using T = Tiles<DT, DP, F::KT, F::NT>;
    const T keys = key_tiles<T>(a, a.k, b, sq, hk, ES), vals = key_tiles<T>(a, a.v, b, sq, hk, ES);
    const RowFrags<DT, DP> rf;
    const ColFrags<DT, DP> cf;

    auto tile_at = [&](int st, int v) { return lds + (2 * st + v) * F::TILE; };
    auto fetch = [&](int step, int st) __attribute__((always_inline)) {
        keys.load(tile_at(st, 0), lo + step * F::KT, hi, a.D);
        vals.load(tile_at(st, 1), lo + step * F::KT, hi, a.D);
    };
    if (steps > 0) {
        if (a.D < DP) {
            clear<F::NT>(lds, F::LDS);
            arrived<>();
            if (WQ > 1) __syncthreads();
        }
#pragma unroll
        for (int i = 0; i + 1 < F::STAGES; ++i)
            if (i < steps) fetch(i, i);
    }
    Frag<DT> q[KS];
    {
        const char* p = head_of(a.q, packed_q, b, sq.q0, hq, ES) + int64_t(tok) * a.q.row * ES;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            zero(q[ks]);
            if (r < rows && 16 * ks + 8 * h < a.D) q[ks] = frag_of<DT>(p + (16 * ks + 8 * h) * ES);
        }
    }
    f32x16_t o[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) zero(o[i]);
    float m = -INFINITY, l = 0.f;

    // 32 keys of this wave after another, their fragments read a group ahead of the products
    constexpr int GS = 2, NG = KB * KS / GS, VS = DB % 2 == 0 ? 2 : 3, VG = 2 * KB * DB / VS;
    auto step_of = [&](int k0, int st, auto some) __attribute__((always_inline)) {
        const char *K = tile_at(st, 0), *V = tile_at(st, 1);
        f32x16_t s[KB];
        Frag<DT> f[2][GS];
        auto read = [&](int g) {
#pragma unroll
            for (int i = 0; i < GS; ++i)
                f[g & 1][i] = rf.read(K, (g * GS + i) / KS * 32, (g * GS + i) % KS);
        };
        float mx = -INFINITY;
        const uint32_t at = uint32_t(k0 + 4 * h - row_lo), n = uint32_t(row_hi - row_lo);
        auto finish = [&](int kb) {                // hides keys, finds the largest score
            if (decltype(some)::value) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (at + uint32_t(kb * 32 + 8 * (i / 4) + i % 4) >= n) s[kb][i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[kb][i]);
        };
        read(0);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (g + 1 < NG) read(g + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < GS; ++i) {
                const int kb = (g * GS + i) / KS, ks = (g * GS + i) % KS;
                if (ks == 0) zero(s[kb]);
                s[kb] = mma(f[g & 1][i], q[ks], s[kb]);
                if (ks == 0 && kb > 0) finish(kb - 1);
            }
        }
        finish(KB - 1);
        Frag<DT> vf[2][VS];
        auto read_v = [&](int g) {
#pragma unroll
            for (int i = 0; i < VS; ++i)
                vf[g & 1][i] = cf.read(V, (g * VS + i) / DB * 16, (g * VS + i) % DB);
        };
        read_v(0);
        mx = both_max(mx);
        if (__any((mx - m) * a.c > Range<DT>::lazy)) {
            const float nm = fmaxf(m, mx);
            const float e =
                m == -INFINITY ? 0.f
                               : __builtin_amdgcn_exp2f(Range<DT>::base(m, a.c) -
                                                        Range<DT>::base(nm, a.c));
            m = nm;
            l *= e;
#pragma unroll
            for (int i = 0; i < DB; ++i)
#pragma unroll
                for (int j = 0; j < 16; ++j) o[i][j] *= e;
        }
        const float base = Range<DT>::base(m, a.c);
        auto probs = [&](int t) {                  // of 16 keys
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float e = __builtin_amdgcn_exp2f(fmaf(s[t / 2][t % 2 * 8 + i], a.c, -base));
                s[t / 2][t % 2 * 8 + i] = e;
                l += e;
            }
            return results<DT>(s[t / 2], t % 2);
        };
        Frag<DT> p = probs(0), next{};
#pragma unroll
        for (int g = 0; g < VG; ++g) {
            if (g + 1 < VG) read_v(g + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < VS; ++i) {
                const int t = (g * VS + i) / DB, db = (g * VS + i) % DB;
                if (db == 0 && t > 0) p = next;
                o[db] = mma(vf[g & 1][i], p, o[db]);
                if (db == 0 && t + 1 < 2 * KB) next = probs(t + 1);
            }
        }
    };

    // Step i: its tile is here (the next ones may be on their way), the last one's stage is free
    // for the tile STAGES - 1 ahead.
    auto step = [&](int i, auto st, auto some) __attribute__((always_inline)) {
        if (F::STAGES > 2 && i + 1 < steps) arrived<(F::STAGES - 2) * 2 * T::N>();
        else arrived<0>();
        if (WQ > 1) __syncthreads();
        if (i + F::STAGES - 1 < steps) fetch(i + F::STAGES - 1, (st + F::STAGES - 1) % F::STAGES);
        const int k0 = lo + i * F::KT;
        if (!decltype(some)::value || (k0 < hi_max && k0 + F::KT > lo_min)) step_of(k0, st, some);
    };
    // Runs of tiles that all rows see whole in a loop of their own, without masks and with
    // constant stages.
    auto whole = [&](int i) {
        return lo + i * F::KT >= all_lo && lo + (i + 1) * F::KT <= min(hi, all_hi);
    };
    for (int i = 0; i < steps;) {
        if (i % F::STAGES == 0) {
            while (i + F::STAGES <= steps && whole(i) && whole(i + F::STAGES - 1)) {
                step(i, std::integral_constant<int, 0>{}, std::false_type{});
                step(i + 1, std::integral_constant<int, 1>{}, std::false_type{});
                if constexpr (F::STAGES > 2)
                    step(i + 2, std::integral_constant<int, 2>{}, std::false_type{});
                i += F::STAGES;
            }
            if (i >= steps) break;
        }
        step(i, i % F::STAGES, std::true_type{});
        ++i;
    }
    l = both_sum(l);
    if (r >= rows) {                               // of a tile's other rows' keys
        m = -INFINITY;
        l = 0.f;
    }

    // rows of a padded batch behind its length are written too, as empty ones
    const bool mine = packed_q ? r < rows : r < all_rows;
    RowOut<DT> ro{nullptr, nullptr, 0.f};
    const int64_t id = (int64_t(b) * a.KV + hk) * all_rows + r;
    if (mine) {
        if (sp.splits > 1) ro.part = sp.o + (int64_t(part) * sp.rows + id) * a.D;
        ro.out = head_of(a.out, packed_q, b, sq.q0, hq, ES) + int64_t(tok) * a.out.row * ES;
    }
    auto statistics = [&](float2 st) {
        ro.inv = st.y == 0.f ? 0.f : 1.f / st.y;
        if (!mine || h != 0) return;
        if (sp.splits > 1) sp.ml[int64_t(part) * sp.rows + id] = st;
        else if (a.lse) a.lse[lse_index(a, sq, b, hq, tok)] = lse_of(st);
    };
    auto write = [&](int db, const f32x16_t& v) {
        if (!mine || (sp.splits > 1 && steps == 0)) return;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int d = 32 * db + 8 * g + 4 * h;
            if (d < a.D) ro.put(d, v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
        }
    };
    if constexpr (KW > 1) {
        // the waves' shares, joined in their order: 8 elements of the rows a wave at a time
        __shared__ float2 ml[KW][32];
        float4* const share = reinterpret_cast<float4*>(lds);
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                share[(4 * i + g) * 64 + lane] = make_float4(o[i][4 * g], o[i][4 * g + 1],
                                                             o[i][4 * g + 2], o[i][4 * g + 3]);
        if (h == 0) ml[part][lane] = share_stats<DT>(m, l, a.c);
        __syncthreads();
        float M = -INFINITY, L = 0.f, f[KW];
#pragma unroll
        for (int k = 0; k < KW; ++k) M = fmaxf(M, ml[k][lane % 32].x);
#pragma unroll
        for (int k = 0; k < KW; ++k) {
            const float2 x = ml[k][lane % 32];
            f[k] = x.y == 0.f ? 0.f
                              : __builtin_amdgcn_exp2f(x.x - (M == -INFINITY ? 0.f : M));
            L += x.y * f[k];
        }
        if (part == 0) statistics(make_float2(M, L));
        ro.inv = L == 0.f ? 0.f : 1.f / L;
        for (int u = part; u < a.D / 8; u += KW) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                const float4 s = reinterpret_cast<const float4*>(
                    reinterpret_cast<const char*>(space) + k * F::LDS)[u * 64 + lane];
                if (f[k] != 0.f) {                 // else of a part that shows it no key
                    v.x = fmaf(s.x, f[k], v.x);
                    v.y = fmaf(s.y, f[k], v.y);
                    v.z = fmaf(s.z, f[k], v.z);
                    v.w = fmaf(s.w, f[k], v.w);
                }
            }
            if (mine) ro.put(8 * u + 4 * h, v.x, v.y, v.z, v.w);
        }
    } else {
        statistics(share_stats<DT>(m, l, a.c));
#pragma unroll
        for (int i = 0; i < DB; ++i) write(i, o[i]);
    }
}

// Joins the shares of the key axis.  Few shares: a thread 4 elements of a row, the shares in
// their order.
template <int DT>
__global__ __launch_bounds__(256) void k_attn_join_few(AttnArgs a, FwdSplit sp, int quads)
{
    constexpr int ES = DT == kF32 ? 4 : 2;
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int64_t id = i / quads;
    const int d = int(i % quads) * 4;
    if (id >= sp.rows) return;
    const int all = a.Sq * a.G;
    const int64_t head = id / all;
    const int b = int(head / a.KV), hk = int(head % a.KV), r = int(id % all);
    const Sequence sq = lane_sequence(a, b);
    if (a.q_starts && r >= sq.lq * a.G) return;
    const int tok = int(fast_div(uint32_t(r), a.group)), hq = hk * a.G + r - tok * a.G;
    float M = -INFINITY;
    for (int s = 0; s < sp.splits; ++s) M = fmaxf(M, sp.ml[s * sp.rows + id].x);
    const float ref = M == -INFINITY ? 0.f : M;
    float L = 0.f, v[4] = {};
    for (int s = 0; s < sp.splits; ++s) {
        const float2 x = sp.ml[s * sp.rows + id];
        if (x.y == 0.f) continue;                  // saw no key
        const float f = __builtin_amdgcn_exp2f(x.x - ref);
        const float4 p = *reinterpret_cast<const float4*>(sp.o + (s * sp.rows + id) * a.D + d);
        L += x.y * f;
        v[0] += p.x * f; v[1] += p.y * f; v[2] += p.z * f; v[3] += p.w * f;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    char* out = head_of(a.out, a.q_starts != nullptr, b, sq.q0, hq, ES) +
                int64_t(tok) * a.out.row * ES;
    if (inv == 0.f) store4<DT>(out, d, 0.f, 0.f, 0.f, 0.f);
    else store4<DT>(out, d, v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    if (d == 0 && a.lse) a.lse[lse_index(a, sq, b, hq, tok)] = lse_of(make_float2(M, L));
}

// More: a wave a row, 4 elements a lane, the halves of the wave every other share, eight of
// them in flight.
template <int DT>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, FwdSplit sp)
{
    constexpr int ES = DT == kF32 ? 4 : 2;
    const int64_t id = int64_t(blockIdx.x) * 4 + scalar(int(threadIdx.x / 64));
    if (id >= sp.rows) return;
    const int lane = threadIdx.x % 64, h = lane / 32, d = lane % 32 * 4;
    const int all = a.Sq * a.G;
    const int64_t head = id / all;
    const int b = int(head / a.KV), hk = int(head % a.KV), r = int(id % all);
    const Sequence sq = sequence_of(a, b);
    if (a.q_starts && r >= sq.lq * a.G) return;
    const int tok = int(fast_div(uint32_t(r), a.group)), hq = hk * a.G + r - tok * a.G;
    const float2* ml = sp.ml + id;
    const float* o = sp.o + id * a.D + d;
    float M = -INFINITY;
    for (int s = lane; s < sp.splits; s += 64) M = fmaxf(M, ml[s * sp.rows].x);
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor(M, x, 64));
    const float ref = M == -INFINITY ? 0.f : M;
    float L = 0.f, v[4] = {};
    for (int s0 = 0; s0 < sp.splits; s0 += 64) {   // 64 shares' weights, one a lane
        float f = 0.f;
        if (s0 + lane < sp.splits) {
            const float2 x = ml[(s0 + lane) * sp.rows];
            if (x.y != 0.f) f = __builtin_amdgcn_exp2f(x.x - ref);      // 0: saw no key
            L += x.y * f;
        }
        const int n = min(64, sp.splits - s0);
        for (int s1 = 0; s1 < n; s1 += 16) {
            float4 p[8];
            float w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int s = s1 + 2 * u + h;
                w[u] = __shfl(f, s, 64);           // past the last: 0
                p[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (d < a.D && w[u] != 0.f)
                    p[u] = *reinterpret_cast<const float4*>(o + (s0 + s) * sp.rows * a.D);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                v[0] = fmaf(p[u].x, w[u], v[0]);
                v[1] = fmaf(p[u].y, w[u], v[1]);
                v[2] = fmaf(p[u].z, w[u], v[2]);
                v[3] = fmaf(p[u].w, w[u], v[3]);
            }
        }
    }
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) L += __shfl_xor(L, x, 64);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = both_sum(v[e]);
    if (h == 0 && d < a.D) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        char* out = head_of(a.out, a.q_starts != nullptr, b, sq.q0, hq, ES) +
                    int64_t(tok) * a.out.row * ES;
        if (inv == 0.f) store4<DT>(out, d, 0.f, 0.f, 0.f, 0.f);
        else store4<DT>(out, d, v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    }
    if (lane == 0 && a.lse) a.lse[lse_index(a, sq, b, hq, tok)] = lse_of(make_float2(M, L));
}

// At most 32 rows a key head: the waves share the rows and part the keys.
bool few_rows(const AttnArgs& a) { return int64_t(a.Sq) * a.G <= 32; }

int64_t row_tiles(const AttnArgs& a)
{
    return ceil_div(int64_t(a.Sq) * a.G, few_rows(a) ? 32 : 128);
}

int64_t all_rows(const AttnArgs& a) { return int64_t(a.B) * a.KV * a.Sq * a.G; }

// Whether a few rows' keys are parted among the four waves of one workgroup, which saves the
// shares' way through memory and a launch, rather than among workgroups or not at all.  Two such
// workgroups fit a CU for heads up to 64, else one, with 64 KB of loads in flight.  us among
// workgroups (or in one wave) against inside, 32 heads on 8 of 128:
//   fewer key heads than CUs, short caches: one of 256 keys 12.3, 8.0; of 517 14.6, 11.1; of 1024
//   12.6, 14.5; 8 of 517 15.5, 11.1; 8 of 1024 14.6, 16.1;
//   as many or more, in well filled rounds: 32 of 512 23, 16; of 4096 102, 96; 50 of 1024 55, 40;
//   128 of 1024 113, 106; but 40 of 4096 138, 155, and short ones of many 64 of 512 26, 29.
// Heads of 64: 300 caches of 2000 33, 28; of 200 9.3, 6.6; 30 x 16 of 4000 105, 97.
// Lengths of their own make a workgroup as long as its cache, where parts even them out.
bool keys_inside(const AttnArgs& a, int64_t keys, int64_t wgs, int64_t cus)
{
    const bool lengths = a.k_starts || a.k_lens;
    if (wgs < 2 * cus && keys <= 768) return true;
    if (wgs < cus) return false;
    if (a.D <= 64) return !lengths || wgs >= 2 * cus;
    return !lengths && keys > 768 && 4 * wgs >= 3 * ceil_div(wgs, cus) * cus;
}

// Parts of the keys where the rows' tiles are too few for the card, each at least 128 keys, of
// those that a tile can see.  Many rows: as many workgroups as a CU holds, two (f32 with more
// than 64 elements one).  Few rows: three of the small workgroups fit a CU, and keys of one length come out even
// where all run in one round, or where one would leave a tenth of the places free, in two: for
// one token over 8 caches of 32768, 8 key heads of 128, 12 parts 189 us, 16 (four a CU) 227; 32
// caches of 4096 102, 118; 20 of 6000 in 4 parts 131, 7 108, 9 97.  Lengths of their own are
// known on the device only: it chooses parts that fill nine tenths of a round (even_chunk; half
// a part a sequence for the last ones), or of two where a sequence would have one or two.
// Where each CU has one or two workgroups without parts, a part is at least 512 keys (us without
// and with parts: 40 caches of 4096, 8 heads of 128, 163, 135; of 1024 40, 34).
// (Least keys 64, 128, 256: 8192 of 8 heads of 128 27, 20, 21.  Parts of what a window of 4096
// keys shows instead of the whole cache: 8 caches of 32768 97, 30.)
FwdSplit make_split(const AttnArgs& a, int dtype, int64_t cus)
{
    FwdSplit sp{};
    sp.splits = 1;
    sp.rows = all_rows(a);
    const bool few = few_rows(a);
    const int64_t wgs = int64_t(a.B) * a.KV * row_tiles(a);
    const int64_t keys = seen_most(a, few ? a.Sq : 128 / a.G + 2, a.Sk);    // of a tile
    sp.chunk = int(keys);
    sp.inside = few && dtype != kF32 && keys_inside(a, keys, wgs, cus);
    if (sp.inside) return sp;
    if (wgs == 0 || wgs >= (few ? 2 : 1) * cus) return sp;
    int64_t parts;
    if (!few) {
        parts = ceil_div((dtype == kF32 && a.D > 64 ? 1 : 2) * cus, wgs);
    } else if (a.k_starts || a.k_lens) {
        parts = ceil_div(6 * cus, wgs);
        const float round = 3.f * float(cus) / float(a.KV);
        sp.places = 0.9f * round - 0.5f * float(a.B);
        if (sp.places < 2.f * float(a.B)) sp.places += 0.9f * round;
    } else {
        parts = 3 * cus / wgs;
        if (10 * parts * wgs < 9 * 3 * cus) parts = 6 * cus / wgs;
    }
    const int64_t least = wgs >= cus ? 512 : 128;
    const int64_t chunk = ceil_div(max64(least, ceil_div(keys, min64(parts, 512))), 64) * 64;
    sp.splits = int(max64(1, ceil_div(keys, chunk)));
    sp.chunk = int(chunk);
    return sp;
}

}  // namespace

size_t attn_fwd_workspace_bytes(const AttnArgs& a, int dtype, int64_t cus)
{
    const int64_t splits = make_split(a, dtype, cus).splits;
    return splits > 1 ? size_t(splits) * size_t(all_rows(a)) * size_t(4 * a.D + 8) : 0;
}

void launch_attn_forward(const AttnArgs& a, int dtype, int64_t cus, void* ws, hipStream_t s)
{
    FwdSplit sp = make_split(a, dtype, cus);
    sp.o = static_cast<float*>(ws);
    sp.ml = reinterpret_cast<float2*>(sp.o + sp.splits * sp.rows * a.D);
    const int tiles = int(row_tiles(a));
    const dim3 grid(unsigned(int64_t(a.B) * a.KV * tiles), unsigned(sp.splits));
    with_dtype(dtype, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        auto go = [&](auto p) {
            constexpr int DP = decltype(p)::value;
            if constexpr (DT != kF32) {
                if (sp.inside) {
                    hipLaunchKernelGGL((k_attn_fwd<DT, DP, 1, 4>), grid, dim3(256), 0, s, a, sp,
                                       tiles);
                    return;
                }
            }
            if (few_rows(a))
                hipLaunchKernelGGL((k_attn_fwd<DT, DP, 1, 1>), grid, dim3(64), 0, s, a, sp, tiles);
            else
                hipLaunchKernelGGL((k_attn_fwd<DT, DP, 4, 1>), grid, dim3(256), 0, s, a, sp, tiles);
        };
        if (a.D <= 64) go(std::integral_constant<int, 64>{});
        else if (a.D <= 96) go(std::integral_constant<int, 96>{});
        else go(std::integral_constant<int, 128>{});
        // us for 4 shares of 12324 rows: 6 in order, 12 a wave a row; 16 of 256: 17 against 5
        if (sp.splits > 1 && sp.splits < 8)
            hipLaunchKernelGGL((k_attn_join_few<DT>),
                               dim3(unsigned(ceil_div(sp.rows * (a.D / 4), 256))), dim3(256), 0, s,
                               a, sp, a.D / 4);
        else if (sp.splits > 1)
            hipLaunchKernelGGL((k_attn_join<DT>), dim3(unsigned(ceil_div(sp.rows, 4))), dim3(256),
                               0, s, a, sp);
    });
}

}  // namespace iabn
