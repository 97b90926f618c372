// Rotary positions with several axes: pair p of every head of a token turns by
//
//   angle = position[token][axis[p]] * inv_freq[p],
//   (a, b) -> (a cos - b sin, b cos + a sin),
//
// a and b the elements p and p + n (halves) or 2p and 2p + 1 (interleaved) of a head whose
// first 2n elements turn; the rest is copied.  The gradient is the turn by the negative
// angle.
//
// Positions reach 2^31, where an angle in float32 is off by whole turns: the angle is
// formed in float64 and reduced to a part of a turn there; its sine and cosine are
// float32.  They cost a wave about 1600 cycles for 8 pairs a lane and are shared by the
// heads that a thread takes: a thread has 8 pairs (one 16-byte access a half for 16-bit
// types) of every eighth head of a token, so that a wave covers whole rows of heads, and
// the angles are a quarter of the time that the card's memory needs for the same heads.
// Few tokens: a head a thread, for the launch's latency.
#include "attn.hpp"
#include "attn_tile.hpp"

namespace iabn {

namespace {

constexpr double kTurns = 0.159154943091895335769;   // 1 / (2 pi)

template <int POS>
__device__ __forceinline__ double position(const void* p, int64_t i)
{
    if constexpr (POS == kPosI32) return double(static_cast<const int32_t*>(p)[i]);
    else if constexpr (POS == kPosI64) return double(static_cast<const int64_t*>(p)[i]);
    else return double(static_cast<const float*>(p)[i]);
}

struct RotarySplit {
    int slices;                       // threads that share a token's heads
    int turn, copy;                   // threads of a head: 8 pairs each, 8 of the rest each
    FastDiv dslices, dchunks;
    int64_t token0;
    uint32_t count;                   // threads of this launch
};

template <int DT, int POS, bool INTER, bool WHOLE>
__global__ __launch_bounds__(kThreads) void k_rotary(RotaryArgs a, RotarySplit sp)
{
    constexpr int ES = DT == kF32 ? 4 : 2;
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= sp.count) return;
    const uint32_t chunks = uint32_t(sp.turn + sp.copy);
    const uint32_t j = fast_div(i, sp.dchunks), chunk = i - j * chunks;
    const uint32_t tk = fast_div(j, sp.dslices), slice = j - tk * uint32_t(sp.slices);
    const int64_t token = sp.token0 + tk, b = token / a.S, row = token - b * a.S;
    const int n = a.pairs, H = a.heads[0] + a.heads[1];

    auto x_of = [&](int h) {
        const bool second = h >= a.heads[0];
        const Heads& t = second ? a.x[1] : a.x[0];
        return t.p + (b * t.batch + row * t.row + int64_t(second ? h - a.heads[0] : h) * t.head) * ES;
    };
    auto y_of = [&](int h) {
        const bool second = h >= a.heads[0];
        const Heads& t = second ? a.y[1] : a.y[0];
        return t.p + (b * t.batch + row * t.row + int64_t(second ? h - a.heads[0] : h) * t.head) * ES;
    };

    if (chunk >= uint32_t(sp.turn)) {                    // what does not turn
        const uint32_t c = 8 * (chunk - uint32_t(sp.turn));
        for (int h = int(slice); h < H; h += sp.slices) {
            float v[8];
            widen8<DT>(load8<DT, false>(x_of(h) + 2 * n * ES, c, a.D - 2 * n), v);
            store8<DT, false>(y_of(h) + 2 * n * ES, c, a.D - 2 * n, v);
        }
        return;
    }
    const int p0 = 8 * int(chunk);
    float co[8], si[8];
    const int64_t at = b * a.pos_batch + row * a.pos_row;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int p = min(p0 + e, n - 1);
        const int axis = a.axis ? min(max(a.axis[p], 0), a.axes - 1) : 0;
        double t = position<POS>(a.positions, at + axis) * a.inv_freq[p] * kTurns;
        t -= rint(t);
        sincospif(2.f * float(t), &si[e], &co[e]);
        si[e] *= a.sign;
    }
    // the two vectors of 8 that hold the pairs, in rows that end with what turns
    const uint32_t c0 = INTER ? 2 * p0 : p0, c1 = INTER ? 2 * p0 + 8 : p0;
    const int C = INTER ? 2 * n : n, second = INTER ? 0 : n * ES;
    auto turn = [&](int h, const Raw8<DT>& r0, const Raw8<DT>& r1) {
        float u[8], v[8], f[8], g[8];
        widen8<DT>(r0, u);
        widen8<DT>(r1, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = INTER ? (e < 4 ? u[2 * e % 8] : v[2 * e % 8]) : u[e];
            const float y = INTER ? (e < 4 ? u[2 * e % 8 + 1] : v[2 * e % 8 + 1]) : v[e];
            const float nx = fmaf(x, co[e], -(y * si[e])), ny = fmaf(y, co[e], x * si[e]);
            if (INTER) {
                if (e < 4) { f[2 * e % 8] = nx; f[2 * e % 8 + 1] = ny; }
                else { g[2 * e % 8] = nx; g[2 * e % 8 + 1] = ny; }
            } else {
                f[e] = nx;
                g[e] = ny;
            }
        }
        char* y = y_of(h);
        store8<DT, WHOLE>(y, c0, C, f);
        store8<DT, WHOLE>(y + second, c1, C, g);
    };
    // four heads' loads in flight
    int h = int(slice);
    for (; h + 3 * sp.slices < H; h += 4 * sp.slices) {
        Raw8<DT> r[4][2];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const char* x = x_of(h + u * sp.slices);
            r[u][0] = load8<DT, WHOLE>(x, c0, C);
            r[u][1] = load8<DT, WHOLE>(x + second, c1, C);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) turn(h + u * sp.slices, r[u][0], r[u][1]);
    }
    for (; h < H; h += sp.slices) {
        const char* x = x_of(h);
        const Raw8<DT> r0 = load8<DT, WHOLE>(x, c0, C), r1 = load8<DT, WHOLE>(x + second, c1, C);
        turn(h, r0, r1);
    }
}

bool in_place(const RotaryArgs& a)
{
    for (int t = 0; t < 2; ++t)
        if (a.heads[t] > 0 && a.x[t].p != a.y[t].p) return false;
    return true;
}

}  // namespace

void launch_rotary(const RotaryArgs& a, int dtype, int64_t cus, hipStream_t s)
{
    RotarySplit sp{};
    const int H = a.heads[0] + a.heads[1];
    const int64_t tokens = a.B * a.S;
    sp.turn = int(ceil_div(a.pairs, 8));
    sp.copy = in_place(a) ? 0 : int(ceil_div(a.D - 2 * a.pairs, 8));
    const int64_t chunks = sp.turn + sp.copy;
    // eighths of the heads, unless the tokens alone would not fill the card
    sp.slices = tokens * chunks * 8 >= cus * 2048 ? int(min64(8, H)) : H;
    sp.dslices = make_fast_div(uint32_t(sp.slices));
    sp.dchunks = make_fast_div(uint32_t(chunks));
    const int64_t per = chunks * sp.slices, step = max64(1, ((int64_t(1) << 31) - 1) / per);
    for (sp.token0 = 0; sp.token0 < tokens; sp.token0 += step) {
        sp.count = uint32_t(min64(step, tokens - sp.token0) * per);
        const dim3 grid(unsigned(ceil_div(sp.count, kThreads)));
        with_dtype(dtype, [&](auto d) {
            constexpr int DT = decltype(d)::value;
            auto go = [&](auto pos, auto inter, auto whole) {
                hipLaunchKernelGGL((k_rotary<DT, decltype(pos)::value, decltype(inter)::value,
                                             decltype(whole)::value>),
                                   grid, dim3(kThreads), 0, s, a, sp);
            };
            auto shape = [&](auto pos) {
                with_whole(a.pairs, [&](auto whole) {
                    if (a.interleaved) go(pos, std::true_type{}, whole);
                    else go(pos, std::false_type{}, whole);
                });
            };
            if (a.pos_type == kPosI32) shape(std::integral_constant<int, kPosI32>{});
            else if (a.pos_type == kPosI64) shape(std::integral_constant<int, kPosI64>{});
            else shape(std::integral_constant<int, kPosF32>{});
        });
    }
}

}  // namespace iabn
