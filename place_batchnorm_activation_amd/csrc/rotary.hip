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

// cos and sin of pair p at position i (counted in coordinates).
template <int POS>
__device__ __forceinline__ void turn_of(const RotaryArgs& a, int64_t i, int p, float& co, float& si)
{
    double t = position<POS>(a.positions, i) * a.inv_freq[p] * kTurns;
    t -= rint(t);
    sincospif(2.f * float(t), &si, &co);
    si *= a.sign;
}

struct RotarySplit {
    int slices;                       // threads that share a token's heads
    int turn, copy;                   // threads of a head: 8 pairs each, 8 of the rest each
    bool in_place;
    FastDiv dslices, dchunks, drows;
    int64_t b0;                       // the first token's sequence, and row in it (below 2^30,
    uint32_t row0;                    // as the tokens of a launch are)
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
    const uint32_t r0 = sp.row0 + tk, db = fast_div(r0, sp.drows);
    const int64_t b = sp.b0 + db, row = r0 - db * uint32_t(a.S);
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
    // A ragged last chunk begins early, inside the row: its loads stay wide, and what belongs to
    // the chunk before it is written twice with the same values, or in place (where that one's
    // thread may have turned it) not written.
    const int own = 8 * int(chunk), p0 = WHOLE ? own : min(own, n - 8), skip = own - p0;
    float co[8], si[8];
    const int64_t at = b * a.pos_batch + row * a.pos_row;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int p = p0 + e, axis = a.axis ? min(max(a.axis[p], 0), a.axes - 1) : 0;
        turn_of<POS>(a, at + axis, p, co[e], si[e]);
    }
    // the two vectors of 8 elements that hold the pairs
    const int c0 = INTER ? 2 * p0 : p0, c1 = INTER ? 2 * p0 + 8 : n + p0;
    auto put = [&](char* y, int first, const float (&v)[8], int from) {
        if (WHOLE || from <= 0 || !sp.in_place) {
            store8<DT, true>(y + first * ES, 0, 8, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e >= from) {
                    if constexpr (DT == kF32) reinterpret_cast<float*>(y)[first + e] = v[e];
                    else reinterpret_cast<uint16_t*>(y)[first + e] = pack1<DT>(v[e]);
                }
        }
    };
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
        put(y, c0, f, INTER ? 2 * skip : skip);
        put(y, c1, g, INTER ? 2 * skip - 8 : skip);
    };
    auto load = [&](const char* x, int first) { return load8<DT, true>(x + first * ES, 0, 8); };
    // four heads' loads in flight
    int h = int(slice);
    for (; h + 3 * sp.slices < H; h += 4 * sp.slices) {
        Raw8<DT> r[4][2];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const char* x = x_of(h + u * sp.slices);
            r[u][0] = load(x, c0);
            r[u][1] = load(x, c1);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) turn(h + u * sp.slices, r[u][0], r[u][1]);
    }
    for (; h < H; h += sp.slices) {
        const char* x = x_of(h);
        const Raw8<DT> r0 = load(x, c0), r1 = load(x, c1);
        turn(h, r0, r1);
    }
}

// Fewer than 8 pairs: a thread one pair of a head.
template <int DT, int POS, bool INTER>
__global__ __launch_bounds__(kThreads) void k_rotary_few(RotaryArgs a, RotarySplit sp)
{
    constexpr int ES = DT == kF32 ? 4 : 2;
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= sp.count) return;
    const uint32_t per = uint32_t(a.pairs + (sp.copy ? a.D - 2 * a.pairs : 0));
    const uint32_t j = fast_div(i, sp.dchunks), p = i - j * per;
    const uint32_t tk = fast_div(j, sp.dslices);
    const int h = int(j - tk * uint32_t(sp.slices)), n = a.pairs;
    const uint32_t r0 = sp.row0 + tk, db = fast_div(r0, sp.drows);
    const int64_t b = sp.b0 + db, row = r0 - db * uint32_t(a.S);
    const bool second = h >= a.heads[0];
    const Heads& tx = second ? a.x[1] : a.x[0];
    const Heads& ty = second ? a.y[1] : a.y[0];
    const int hh = second ? h - a.heads[0] : h;
    const char* x = tx.p + (b * tx.batch + row * tx.row + int64_t(hh) * tx.head) * ES;
    char* y = ty.p + (b * ty.batch + row * ty.row + int64_t(hh) * ty.head) * ES;
    auto get = [&](int d) {
        if constexpr (DT == kF32) return reinterpret_cast<const float*>(x)[d];
        else return unpack1<DT>(reinterpret_cast<const uint16_t*>(x)[d]);
    };
    auto put = [&](int d, float v) {
        if constexpr (DT == kF32) reinterpret_cast<float*>(y)[d] = v;
        else reinterpret_cast<uint16_t*>(y)[d] = pack1<DT>(v);
    };
    if (int(p) >= n) {
        put(n + int(p), get(n + int(p)));
        return;
    }
    float co, si;
    const int axis = a.axis ? min(max(a.axis[p], 0), a.axes - 1) : 0;
    turn_of<POS>(a, b * a.pos_batch + row * a.pos_row + axis, int(p), co, si);
    const int d0 = INTER ? 2 * int(p) : int(p), d1 = INTER ? d0 + 1 : n + int(p);
    const float u = get(d0), v = get(d1);
    put(d0, fmaf(u, co, -(v * si)));
    put(d1, fmaf(v, co, u * si));
}

bool all_in_place(const RotaryArgs& a)
{
    for (int t = 0; t < 2; ++t)
        if (a.heads[t] > 0 && a.x[t].p != a.y[t].p) return false;
    return true;
}

bool any_in_place(const RotaryArgs& a)
{
    for (int t = 0; t < 2; ++t)
        if (a.heads[t] > 0 && a.x[t].p == a.y[t].p) return true;
    return false;
}

}  // namespace

void launch_rotary(const RotaryArgs& a, int dtype, int64_t cus, hipStream_t s)
{
    RotarySplit sp{};
    const int H = a.heads[0] + a.heads[1];
    const int64_t tokens = a.B * a.S;
    const bool few = a.pairs < 8, inside = any_in_place(a);
    sp.in_place = inside;
    sp.turn = int(ceil_div(a.pairs, 8));
    sp.copy = all_in_place(a) ? 0 : int(ceil_div(a.D - 2 * a.pairs, 8));
    const int64_t chunks = few ? a.pairs + (sp.copy ? a.D - 2 * a.pairs : 0) : sp.turn + sp.copy;
    // Eighths of the heads, unless that leaves fewer than two waves a SIMD (3 x 1369 tokens of 24
    // heads of 72, f32: 17 us, 22 with a head a thread).
    sp.slices = !few && tokens * chunks * 8 >= cus * 512 ? int(min64(8, H)) : H;
    sp.dslices = make_fast_div(uint32_t(sp.slices));
    sp.dchunks = make_fast_div(uint32_t(chunks));
    sp.drows = make_fast_div(uint32_t(a.S));
    const int64_t per = chunks * sp.slices;
    const int64_t step = max64(1, min64(int64_t(1) << 30, ((int64_t(1) << 31) - 1) / per));
    for (int64_t first = 0; first < tokens; first += step) {
        sp.b0 = first / a.S;
        sp.row0 = uint32_t(first % a.S);
        sp.count = uint32_t(min64(step, tokens - first) * per);
        const dim3 grid(unsigned(ceil_div(sp.count, kThreads)));
        with_dtype(dtype, [&](auto d) {
            constexpr int DT = decltype(d)::value;
            auto go = [&](auto pos, auto inter, auto whole) {
                hipLaunchKernelGGL((k_rotary<DT, decltype(pos)::value, decltype(inter)::value,
                                             decltype(whole)::value>),
                                   grid, dim3(kThreads), 0, s, a, sp);
            };
            auto shape = [&](auto pos) {
                if (few) {
                    if (a.interleaved)
                        hipLaunchKernelGGL((k_rotary_few<DT, decltype(pos)::value, true>), grid,
                                           dim3(kThreads), 0, s, a, sp);
                    else
                        hipLaunchKernelGGL((k_rotary_few<DT, decltype(pos)::value, false>), grid,
                                           dim3(kThreads), 0, s, a, sp);
                    return;
                }
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
