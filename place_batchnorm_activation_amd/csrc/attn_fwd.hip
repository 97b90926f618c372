// Attention forward: out = softmax(scale * q k^T) v over the visible keys, and the rows'
// log-sum-exp for the backward.
//
// One pass over the keys with the running maximum m and sum l of each row:
//   S^T = K Q^T,  P^T = exp(S^T - m),  O^T += V^T P^T,
// O and l scaled by exp(m_old - m_new) when m grows, which is left until it grows by more
// than 2^8 (P then stays below 2^8, and the sums are fp32).  A wave holds 32 rows (rows of
// a key head: attn.hpp) in registers, Q and O^T both; the statistics are scalars of the
// lane, one exchange with the other half of the wave a tile.
//
// Many rows: a workgroup of 4 waves x 32 rows shares the tiles of keys in LDS, two stages,
// the next tile's loads in flight.  At most 32 rows (single tokens): the 4 waves take the
// same rows and a quarter of each tile's keys, and their shares are joined in LDS.  Few
// workgroups: the keys are cut among several, whose shares (O, m, l in fp32) go through
// the workspace and are joined in their order by a second kernel.
#include "attn_tile.hpp"

namespace iabn {

namespace {

constexpr float kLazy = 8.f;         // binary orders that the running maximum may lag behind

struct FwdSplit {
    int splits;
    float* o;                        // [split][row][D]
    float2* ml;                      // [split][row]
    int64_t rows;                    // B * KV * Sq * G
};

template <int DT, int DP, int WQ, int WK>
struct FwdShape {
    static constexpr int NT = 64 * WQ * WK;
    static constexpr int KW = WK > 1 || DT == kF32 ? 32 : 64;    // keys of a wave's tile
    static constexpr int KT = KW * WK;
    // a tile in LDS; waves with keys of their own each fill theirs
    static constexpr int ROWS = WK > 1 ? KW : KT, LOADERS = WK > 1 ? 64 : NT;
    static constexpr int TILE = ROWS * TileShape<DT, DP>::PITCH;
    static constexpr int STAGES = WK > 1 && DT == kF32 && DP > 64 ? 1 : 2;       // LDS ends there
    static constexpr int WAVE = WK > 1 ? STAGES * 2 * TILE : 0;  // bytes of a wave
    static constexpr int TILES = WK > 1 ? WK * WAVE : STAGES * 2 * TILE;
    static constexpr int JOIN = WK > 1 ? WK * DP * 32 * 4 + WK * 32 * 8 : 0;
    static constexpr int LDS = TILES > JOIN ? TILES : JOIN;
    static constexpr int WAVES = DT == kF32 || (WK > 1 && DP > 64) ? 1 : 2;      // of a SIMD
};

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

template <int DT, int DP, int WQ, int WK>
__global__ __launch_bounds__(64 * WQ * WK, (FwdShape<DT, DP, WQ, WK>::WAVES)) void k_attn_fwd(
    AttnArgs a, FwdSplit sp, int tiles)
{
    using F = FwdShape<DT, DP, WQ, WK>;
    using S = TileShape<DT, DP>;
    constexpr int ES = S::ES, KS = DP / 16, DB = DP / 32, KB = F::KW / 32;
    __shared__ uint4 space[F::LDS / 16];
    char* const lds = reinterpret_cast<char*>(space);

    const int lane = threadIdx.x % 64, h = lane / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wq = wave % WQ, wk = wave / WQ;
    uint32_t head, tile;
    head_and_tile(uint32_t(a.B) * a.KV, uint32_t(tiles), false, head, tile);
    const int b = int(head / uint32_t(a.KV)), hk = int(head % uint32_t(a.KV));
    tile = uint32_t(tiles) - 1 - tile;             // causal rows with many keys first
    const Sequence sq = sequence_of(a, b);
    const int rows = sq.lq * a.G, all_rows = a.Sq * a.G;
    const int row0 = int(tile) * 32 * WQ, r0 = row0 + wq * 32, r = r0 + lane % 32;
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

    int steps = hi > lo ? (hi - lo + F::KT - 1) / F::KT : 0, step0 = 0;
    if (sp.splits > 1) {
        const int per = (steps + sp.splits - 1) / sp.splits;
        step0 = min(steps, int(blockIdx.y) * per);
        steps = min(steps, step0 + per);
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
    using T = Tiles<DT, DP, F::ROWS, F::LOADERS>;
    const T keys = key_tiles<T>(a, a.k, b, sq, hk, ES), vals = key_tiles<T>(a, a.v, b, sq, hk, ES);
    const RowFrags<DT, DP> rf;
    const ColFrags<DT, DP> cf;

    f32x16_t o[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) zero(o[i]);
    float m = -INFINITY, l = 0.f;

    auto tile_at = [&](int st, int v) { return lds + wk * F::WAVE + (2 * st + v) * F::TILE; };
    auto fetch = [&](int step, int st) __attribute__((always_inline)) {
        const int first = lo + step * F::KT + (WK > 1 ? wk * F::KW : 0);
        keys.load(tile_at(st, 0), first, hi, a.D);
        vals.load(tile_at(st, 1), first, hi, a.D);
    };
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
        if (__any((mx - m) * a.c > kLazy)) {
            const float nm = fmaxf(m, mx);
            const float e = __builtin_amdgcn_exp2f((m - (nm == -INFINITY ? 0.f : nm)) * a.c);
            m = nm;
            l *= e;
#pragma unroll
            for (int i = 0; i < DB; ++i)
#pragma unroll
                for (int j = 0; j < 16; ++j) o[i][j] *= e;
        }
        const float base = m == -INFINITY ? 0.f : m * a.c;
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

    if (step0 < steps) {
        if (a.D < DP) {
            clear<F::NT>(lds, F::TILES);
            __syncthreads();
        }
        fetch(step0, 0);
        auto step = [&](int i, auto st, auto some) __attribute__((always_inline)) {
            arrived();
            if (WK == 1) __syncthreads();          // here, and the other stage read by all
            if (F::STAGES == 2 && i + 1 < steps) fetch(i + 1, 1 - st);
            const int k0 = lo + i * F::KT + wk * F::KW;          // of this wave
            if (!decltype(some)::value || (k0 < hi_max && k0 + F::KW > lo_min))
                step_of(k0, st, some);
            if (F::STAGES == 1 && i + 1 < steps) {
                arrived();
                fetch(i + 1, 0);
            }
        };
        // Pairs of tiles that all rows see whole in a loop of their own, without masks and with
        // constant stages.
        const int first = lo + (WK > 1 ? wk * F::KW : 0);
        auto whole = [&](int i) {
            return first + i * F::KT >= all_lo && first + i * F::KT + (WK > 1 ? F::KW : F::KT) <= all_hi;
        };
        for (int i = step0; i < steps;) {
            if (F::STAGES == 2 && ((i - step0) & 1) == 0) {
                while (i + 1 < steps && whole(i) && whole(i + 1)) {
                    step(i, std::integral_constant<int, 0>{}, std::false_type{});
                    step(i + 1, std::integral_constant<int, 1>{}, std::false_type{});
                    i += 2;
                }
                if (i >= steps) break;
            }
            step(i, F::STAGES == 2 ? (i - step0) & 1 : 0, std::true_type{});
            ++i;
        }
        __syncthreads();
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
        if (sp.splits > 1) ro.part = sp.o + (int64_t(blockIdx.y) * sp.rows + id) * a.D;
        ro.out = head_of(a.out, packed_q, b, sq.q0, hq, ES) + int64_t(tok) * a.out.row * ES;
    }
    auto statistics = [&](float m_, float l_) {
        ro.inv = l_ == 0.f ? 0.f : 1.f / l_;
        if (!mine || h != 0) return;
        if (sp.splits > 1) {
            sp.ml[int64_t(blockIdx.y) * sp.rows + id] = make_float2(m_, l_);
        } else if (a.lse) {
            const float lse = l_ == 0.f ? -INFINITY : (m_ * a.c + __builtin_amdgcn_logf(l_)) * kLn2A;
            a.lse[lse_index(a, sq, b, hq, tok)] = lse;
        }
    };
    auto write = [&](int db, const f32x16_t& v) {
        if (!mine) return;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int d = 32 * db + 8 * g + 4 * h;
            if (d < a.D) ro.put(d, v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
        }
    };
    if constexpr (WK == 1) {
        statistics(m, l);
#pragma unroll
        for (int i = 0; i < DB; ++i) write(i, o[i]);
    } else {
        // the tiles have been read by all waves: their place holds the shares
        float* share = reinterpret_cast<float*>(lds);            // [wave][db][16][64]
        float2* ml = reinterpret_cast<float2*>(share + WK * DB * 16 * 64);
        if (h == 0) ml[wk * 32 + lane] = make_float2(m, l);
        __syncthreads();
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int k = 0; k < WK; ++k) M = fmaxf(M, ml[k * 32 + lane % 32].x);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int k = 0; k < WK; ++k) {
            const float2 x = ml[k * 32 + lane % 32];
            L += x.y * __builtin_amdgcn_exp2f((x.x - ref) * a.c);
        }
        const float f = __builtin_amdgcn_exp2f((m - ref) * a.c);
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) share[((wk * DB + i) * 16 + e) * 64 + lane] = o[i][e] * f;
        __syncthreads();
        if (wk < DB) {
            f32x16_t v;
            zero(v);
#pragma unroll
            for (int k = 0; k < WK; ++k)
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] += share[((k * DB + wk) * 16 + e) * 64 + lane];
            statistics(M, L);                                    // every wave the same
            write(wk, v);
        }
    }
}

// Joins the shares of the key axis, in their order: a thread 4 elements of a row.
template <int DT>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, FwdSplit sp, int quads)
{
    constexpr int ES = DT == kF32 ? 4 : 2;
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int64_t id = i / quads;
    const int d = int(i % quads) * 4;
    if (id >= sp.rows) return;
    const int all_rows = a.Sq * a.G;
    const int64_t head = id / all_rows;
    const int b = int(head / a.KV), hk = int(head % a.KV), r = int(id % all_rows);
    const Sequence sq = sequence_of(a, b);
    if (a.q_starts && r >= sq.lq * a.G) return;
    const int tok = int(fast_div(uint32_t(r), a.group)), hq = hk * a.G + r - tok * a.G;
    float M = -INFINITY;
    for (int s = 0; s < sp.splits; ++s) M = fmaxf(M, sp.ml[s * sp.rows + id].x);
    const float ref = M == -INFINITY ? 0.f : M;
    float L = 0.f, v[4] = {};
    for (int s = 0; s < sp.splits; ++s) {
        const float2 x = sp.ml[s * sp.rows + id];
        const float f = __builtin_amdgcn_exp2f((x.x - ref) * a.c);
        const float4 p = *reinterpret_cast<const float4*>(sp.o + (s * sp.rows + id) * a.D + d);
        L += x.y * f;
        v[0] += p.x * f; v[1] += p.y * f; v[2] += p.z * f; v[3] += p.w * f;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    char* out = head_of(a.out, a.q_starts != nullptr, b, sq.q0, hq, ES) +
                int64_t(tok) * a.out.row * ES;
    if (inv == 0.f) store4<DT>(out, d, 0.f, 0.f, 0.f, 0.f);
    else store4<DT>(out, d, v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    if (d == 0 && a.lse) {
        const float lse = L == 0.f ? -INFINITY : (M * a.c + __builtin_amdgcn_logf(L)) * kLn2A;
        a.lse[lse_index(a, sq, b, hq, tok)] = lse;
    }
}

// At most 32 rows a key head: the waves share the rows and part the keys.
bool few_rows(const AttnArgs& a) { return int64_t(a.Sq) * a.G <= 32; }

int64_t row_tiles(const AttnArgs& a)
{
    return ceil_div(int64_t(a.Sq) * a.G, few_rows(a) ? 32 : 128);
}

int64_t all_rows(const AttnArgs& a) { return int64_t(a.B) * a.KV * a.Sq * a.G; }

}  // namespace

// Two workgroups a CU, each at least 256 keys.
int attn_fwd_splits(const AttnArgs& a, int64_t cus)
{
    const int64_t wgs = int64_t(a.B) * a.KV * row_tiles(a);
    if (wgs >= cus || wgs == 0) return 1;
    return int(max64(1, min64(min64(ceil_div(2 * cus, wgs), ceil_div(a.Sk, 256)), 512)));
}

size_t attn_fwd_workspace_bytes(const AttnArgs& a, int64_t cus)
{
    const int64_t splits = attn_fwd_splits(a, cus);
    return splits > 1 ? size_t(splits) * size_t(all_rows(a)) * size_t(4 * a.D + 8) : 0;
}

void launch_attn_forward(const AttnArgs& a, int dtype, int64_t cus, void* ws, hipStream_t s)
{
    FwdSplit sp{};
    sp.splits = attn_fwd_splits(a, cus);
    sp.rows = all_rows(a);
    sp.o = static_cast<float*>(ws);
    sp.ml = reinterpret_cast<float2*>(sp.o + sp.splits * sp.rows * a.D);
    const int tiles = int(row_tiles(a));
    const dim3 grid(unsigned(int64_t(a.B) * a.KV * tiles), unsigned(sp.splits));
    with_dtype(dtype, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        auto go = [&](auto p) {
            constexpr int DP = decltype(p)::value;
            if (few_rows(a))
                hipLaunchKernelGGL((k_attn_fwd<DT, DP, 1, 4>), grid, dim3(256), 0, s, a, sp, tiles);
            else
                hipLaunchKernelGGL((k_attn_fwd<DT, DP, 4, 1>), grid, dim3(256), 0, s, a, sp, tiles);
        };
        if (a.D <= 64) go(std::integral_constant<int, 64>{});
        else if (a.D <= 96) go(std::integral_constant<int, 96>{});
        else go(std::integral_constant<int, 128>{});
        if (sp.splits > 1) {
            const int quads = a.D / 4;
            hipLaunchKernelGGL((k_attn_join<DT>), dim3(unsigned(ceil_div(sp.rows * quads, 256))),
                               dim3(256), 0, s, a, sp, quads);
        }
    });
}

}  // namespace iabn
