// Device helpers of the attention kernels: sequences, tiles of rows in LDS and the
// fragments that the matrix instructions take from them.
//
// Products are 32 x 32 x 16 on the matrix units: a lane holds 8 consecutive elements of
// the summed index of one row (operand A, row lane % 32) or column (operand B), those of
// half lane / 32, and of the result the elements of column lane % 32 in rows
// 8 * (r / 4) + 4 * (lane / 32) + r % 4, r = 0 .. 15.  Scores are formed transposed
// (keys x queries, or queries x keys where a wave owns keys), so that a lane's results
// belong to one query (key): its statistics are scalars of the lane, and the results,
// converted, are as they lie the operand B of the next product, whose summed index is
// what the rows were.  That product's operand A, the transpose of a tile that lies in LDS row by
// row, comes through the transposing LDS reads.
//
// float32 takes the same fragments of 8 elements through eight 32 x 32 x 2 instructions.
#pragma once

#include <hip/hip_runtime.h>

#include "attn.hpp"
#include "rows.hpp"

namespace iabn {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr float kLog2eA = 1.44269504088896341f;
constexpr float kLn2A = 0.693147180559945309f;

// A problem's sequence: rows of q and k, and where they begin.  Starts and lengths are
// the caller's device data: whatever they hold, no row outside the tensors results.
struct Sequence {
    int64_t q0, k0;
    int lq, lk;
};

__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t lo, int64_t hi)
{
    return v < lo ? lo : v > hi ? hi : v;
}

__device__ __forceinline__ void sequence_side(const int32_t* starts, const int32_t* lens, int b,
                                              int64_t rows, int most, int64_t& first, int& len)
{
    first = 0;
    len = most;
    if (starts) {
        first = clamp64(starts[b], 0, rows);
        const int64_t n = clamp64(int64_t(starts[b + 1]) - first, 0, most);
        len = int(dmin(n, rows - first));
    } else if (lens) {
        len = int(clamp64(lens[b], 0, most));
    }
}

// The same in every lane, and in scalar registers.
__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ Sequence lane_sequence(const AttnArgs& a, int b)
{
    Sequence s;
    sequence_side(a.q_starts, a.q_lens, b, a.q_rows, a.Sq, s.q0, s.lq);
    sequence_side(a.k_starts, a.k_lens, b, a.k_rows, a.Sk, s.k0, s.lk);
    return s;
}

// b the same in all lanes
__device__ __forceinline__ Sequence sequence_of(const AttnArgs& a, int b)
{
    Sequence s = lane_sequence(a, b);
    s.q0 = uint32_t(scalar(int(s.q0)));            // starts are below 2^31
    s.k0 = uint32_t(scalar(int(s.k0)));
    s.lq = scalar(s.lq);
    s.lk = scalar(s.lk);
    return s;
}

// Keys [lo, hi) that query token t sees.
__device__ __forceinline__ void visible(const AttnArgs& a, const Sequence& s, int t, int& lo,
                                        int& hi)
{
    const int at = t + s.lk - s.lq;
    lo = max(0, at - a.left);
    hi = min(s.lk, at + a.right + 1);
}

__device__ __forceinline__ bool windowed(const AttnArgs& a)
{
    return a.left < kAttnMaxLen || a.right < kAttnMaxLen;
}

// First address of head h of sequence b.
__device__ __forceinline__ char* head_of(const Heads& t, bool packed, int b, int64_t first, int h,
                                         int es)
{
    return t.p + ((packed ? 0 : b * t.batch) + first * t.row + h * t.head) * es;
}

// ---------------------------------------------------------------------------
// fragments and products

template <int DT>
struct Frag {
    uint32_t w[DT == kF32 ? 8 : 4];
};

template <int DT>
__device__ __forceinline__ f32x16_t mma(const Frag<DT>& a, const Frag<DT>& b, f32x16_t c)
{
    if constexpr (DT == kBF16) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    } else if constexpr (DT == kF16) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a),
                                                      __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.w[i]),
                                                     __uint_as_float(b.w[i]), c, 0, 0, 0);
        return c;
    }
}

template <int DT>
__device__ __forceinline__ void zero(Frag<DT>& f)
{
#pragma unroll
    for (uint32_t& w : f.w) w = 0u;
}

__device__ __forceinline__ void zero(f32x16_t& v)
{
#pragma unroll
    for (int r = 0; r < 16; ++r) v[r] = 0.f;
}

// Results 8i .. 8i + 7 of a product, as the next one's operand B (rounded to DT).
template <int DT>
__device__ __forceinline__ Frag<DT> results(const f32x16_t& v, int i)
{
    Frag<DT> f;
#pragma unroll
    for (int j = 0; j < (DT == kF32 ? 8 : 4); ++j) {
        if constexpr (DT == kF32) f.w[j] = __float_as_uint(v[8 * i + j]);
        else f.w[j] = pack2<DT>(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
    }
    return f;
}

// Eight elements of a row from global memory (any alignment of one element).
template <int DT>
__device__ __forceinline__ Frag<DT> frag_of(const char* p)
{
    Frag<DT> f;
#pragma unroll
    for (int i = 0; i < (DT == kF32 ? 2 : 1); ++i) {
        const uint4 q = load16_any(p + 16 * i);
        f.w[4 * i] = q.x; f.w[4 * i + 1] = q.y; f.w[4 * i + 2] = q.z; f.w[4 * i + 3] = q.w;
    }
    return f;
}

template <int DT>
__device__ __forceinline__ float frag_value(const Frag<DT>& f, int i)
{
    if constexpr (DT == kF32) return __uint_as_float(f.w[i]);
    else return unpack1<DT>(uint16_t(f.w[i / 2] >> (16 * (i & 1))));
}

// The largest, and the sum, of both halves' values of a column, in both.
__device__ __forceinline__ float both_max(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float both_sum(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// ---------------------------------------------------------------------------
// tiles of rows in LDS

__device__ __forceinline__ uint32_t lds_address(const char* p)
{
    return uint32_t(uintptr_t((const __attribute__((address_space(3))) char*)p));
}

// 16 bytes a lane from base + offset to LDS, lane l's to dst + 16 * l (dst the same in all
// lanes).  In assembly, since the compiler would wait for it before any other access to
// LDS; the wait is arrived()'s.  (The compiler warns of a clobbered m0, which it reserves: it
// never keeps a value there, but an m0 that it set for instructions of its own it sets again
// behind a statement that names it.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void to_lds(const char* base, uint32_t offset, uint32_t dst)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "s"(dst), "v"(offset), "s"(base)
                 : "m0", "memory");
}
#pragma clang diagnostic pop

// DP: the head's elements as the kernel counts them, a multiple of 32 (those past D are
// zeros).  Rows are NC 16-byte chunks apart, a power of two; chunk c of row r lies at
// place c XOR a mix of r, so that
//   - 16 lanes that read one chunk of 16 neighbouring rows meet 16 different bank quads,
//   - 32 lanes that read 64 bytes of each of 4 neighbouring rows (a transposing read)
//     cover all 64 banks.
// (No bank conflicts by the counters.)  A lane's reads of a tile are then one address XOR
// constants plus constants.
template <int DT, int DP>
struct TileShape {
    static constexpr int ES = DT == kF32 ? 4 : 2;
    static constexpr int E = 16 / ES;                            // elements of a chunk
    static constexpr int USED = DP / E;                          // chunks of a row
    static constexpr int NC = (DP <= 64 ? 64 : 128) / E;
    static constexpr int PITCH = NC * 16;                        // bytes
    static_assert(DP % 32 == 0 && DP <= 128, "head sizes");

    static __device__ __forceinline__ uint32_t mix(uint32_t r)
    {
        if constexpr (NC == 8) return ((r & 2) << 1) | ((r >> 2) & 3);
        else if constexpr (DT == kF32) return ((r & 7) << 1) | ((r >> 3) & 1);
        else return ((r & 3) << 2) | ((r >> 2) & 3);
    }
    static __device__ __forceinline__ uint32_t place(uint32_t r, uint32_t c)
    {
        return r * PITCH + 16 * (c ^ mix(r));
    }
};

// Rows of a head, or of a group of heads (attn.hpp), in global memory, and how NT threads
// take ROWS of them to LDS: thread t has place t % NC of row t / NC of each pass of PER rows.
//
// Whole tiles of aligned rows go there directly, without registers, each wave writing the
// 64 chunks from a scalar place on: the mix is undone in the addresses that the lanes read.
// The caller waits for them (arrived()).  Everything else (the end of a sequence, rows not
// at 16-byte distances) goes through registers before load() returns; rows from `end` on
// and elements from D on are zeros there.  (Elements from D on of direct tiles are not
// written at all: clear() the stages first.)
template <int DT, int DP, int ROWS, int NT>
struct Tiles {
    using S = TileShape<DT, DP>;
    static constexpr int PER = NT / S::NC, N = ROWS / PER;
    static_assert(NT % S::NC == 0 && ROWS % PER == 0, "threads for a tile");

    const char* p;                    // the (first query) head
    int64_t row, head;                // bytes
    FastDiv group;
    int G;
    uint32_t offset;                  // of this thread's row within a pass
    bool direct;

    __device__ __forceinline__ Tiles(const char* p_, int64_t row_, int64_t head_, FastDiv group_,
                                     int G_)
        : p(p_), row(row_), head(head_), group(group_), G(G_), offset(0)
    {
        const int64_t most = row * (PER / G + 1) + head * G;     // of a pass's offsets
        direct = PER % G == 0 && most < (int64_t(1) << 31) &&
                 ((reinterpret_cast<uintptr_t>(p) | uintptr_t(row) | uintptr_t(head)) & 15) == 0;
        if (direct) {
            const uint32_t r = threadIdx.x % NT / S::NC, t = G == 1 ? r : fast_div(r, group);
            offset = t * uint32_t(row) + (r - t * G) * uint32_t(head);
        }
    }

    // rows first .. first + ROWS - 1, first a multiple of the group, D elements of each
    __device__ __forceinline__ void load(char* tile, int first, int end, int D) const
    {
        const uint32_t th = threadIdx.x % NT, c = th % S::NC, r = th / S::NC;
        if (direct && first + ROWS <= end) {
            const int tok = G == 1 ? first : scalar(int(fast_div(uint32_t(first), group)));
            const char* base = p + int64_t(tok) * row;
            const uint32_t dst = uint32_t(scalar(int(lds_address(tile) + th / 64 * 1024)));
            const int64_t pass = PER / G * row;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t chunk = c ^ S::mix(r + i * PER);
                if (int(chunk) * S::E < D)
                    to_lds(base + i * pass, offset + 16 * chunk, dst + i * NT * 16);
            }
            return;
        }
        uint4 q[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = first + int(r) + i * PER;
            q[i] = make_uint4(0, 0, 0, 0);
            if (int(c) * S::E < D && at < end) {
                const int t = G == 1 ? at : int(fast_div(uint32_t(at), group));
                q[i] = load16_any(p + t * row + int64_t(at - t * G) * head + c * 16);
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (S::USED == S::NC || c < S::USED)
                *reinterpret_cast<uint4*>(tile + S::place(r + i * PER, c)) = q[i];
    }
};

// Zeros in `bytes` (a multiple of 16) of LDS.
template <int NT>
__device__ __forceinline__ void clear(char* p, int bytes)
{
    for (int i = int(threadIdx.x) % NT * 16; i < bytes; i += NT * 16)
        *reinterpret_cast<uint4*>(p + i) = make_uint4(0, 0, 0, 0);
}

// All but the last LEFT direct loads of this wave have arrived (loads return in their
// order), and every read of LDS has returned, so that a direct load may take its place.
template <int LEFT = 0>
__device__ __forceinline__ void arrived()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LEFT) : "memory");
}

// A lane's operand A of rows row0 .. row0 + 31 at elements 16 * ks .. 16 * ks + 15, row0 a
// multiple of 16: at(lane) once, then read.
template <int DT, int DP>
struct RowFrags {
    using S = TileShape<DT, DP>;
    uint32_t at;

    __device__ __forceinline__ RowFrags()
    {
        const uint32_t lane = threadIdx.x % 64, h = lane / 32;
        at = S::place(lane % 32, DT == kF32 ? 2 * h : h);
    }
    __device__ __forceinline__ Frag<DT> read(const char* tile, int row0, int ks) const
    {
        Frag<DT> f;
#pragma unroll
        for (int i = 0; i < (DT == kF32 ? 2 : 1); ++i) {
            const uint32_t x = at ^ uint32_t(DT == kF32 ? 64 * ks + 16 * i : 32 * ks);
            const uint4 q = *reinterpret_cast<const uint4*>(tile + row0 * S::PITCH + x);
            f.w[4 * i] = q.x; f.w[4 * i + 1] = q.y; f.w[4 * i + 2] = q.z; f.w[4 * i + 3] = q.w;
        }
        return f;
    }
};

// A lane's operand A of the transposed tile: elements 32 * db .. 32 * db + 31, summed over
// the 16 rows from row0 (a multiple of 16) in the order in which a lane holds a product's
// results: element i of half h is row row0 + 8 * (i / 4) + 4 * h + i % 4.
template <int DT, int DP>
struct ColFrags {
    using S = TileShape<DT, DP>;
    uint32_t at;

    __device__ __forceinline__ ColFrags()
    {
        const uint32_t lane = threadIdx.x % 64, h = lane / 32, l = lane % 16;
        if constexpr (DT == kF32)
            at = S::place(4 * h, (lane % 32) / 4) + 4 * (lane % 4);
        else          // 16 lanes read 16 columns of 4 rows, 4 columns each, and get one column's 4
            at = S::place(4 * h + l / 4, ((lane / 16) & 1) * 2 + (l % 4) / 2) + 8 * (l % 2);
    }
    __device__ __forceinline__ Frag<DT> read(const char* tile, int row0, int db) const
    {
        Frag<DT> f;
        if constexpr (DT == kF32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t x = at ^ uint32_t(128 * db + 32 * (i % 4) + 16 * (i / 4));
                f.w[i] = *reinterpret_cast<const uint32_t*>(
                    tile + (row0 + 8 * (i / 4) + i % 4) * S::PITCH + x);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t x = at ^ uint32_t(64 * db + 32 * j);
                const char* p = tile + (row0 + 8 * j) * S::PITCH + x;
                const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4_t*)p);
                const uint2 u = __builtin_bit_cast(uint2, v);
                f.w[2 * j] = u.x;
                f.w[2 * j + 1] = u.y;
            }
        }
        return f;
    }
};

// Four consecutive elements d .. d + 3 of a row, rounded.
template <int DT>
__device__ __forceinline__ void store4(char* row, int d, float a, float b, float c, float e)
{
    if constexpr (DT == kF32) {
        const u32x4_any_t w = {__float_as_uint(a), __float_as_uint(b), __float_as_uint(c),
                               __float_as_uint(e)};
        *reinterpret_cast<u32x4_any_t*>(row + 4 * d) = w;
    } else {
        const u32x2_any_t w = {pack2<DT>(a, b), pack2<DT>(c, e)};
        *reinterpret_cast<u32x2_any_t*>(row + 2 * d) = w;
    }
}

// A row of a key head's group (attn.hpp) in global memory, and tiles of such rows.
__device__ __forceinline__ const char* group_row(const AttnArgs& a, const Heads& t, int b,
                                                 const Sequence& s, int hk, int r, int es)
{
    const int tok = int(fast_div(uint32_t(r), a.group));
    return head_of(t, a.q_starts != nullptr, b, s.q0, hk * a.G + r - tok * a.G, es) +
           int64_t(tok) * t.row * es;
}

template <class T>
__device__ __forceinline__ T group_tiles(const AttnArgs& a, const Heads& t, int b,
                                         const Sequence& s, int hk, int es)
{
    return T(head_of(t, a.q_starts != nullptr, b, s.q0, hk * a.G, es), t.row * es, t.head * es,
             a.group, a.G);
}

template <class T>
__device__ __forceinline__ T key_tiles(const AttnArgs& a, const Heads& t, int b, const Sequence& s,
                                       int hk, int es)
{
    return T(head_of(t, a.k_starts != nullptr, b, s.k0, hk, es), t.row * es, 0, FastDiv{}, 1);
}

// The place of a row's log-sum-exp.
__device__ __forceinline__ int64_t lse_index(const AttnArgs& a, const Sequence& s, int b, int hq,
                                             int tok)
{
    return a.q_starts ? int64_t(hq) * a.q_rows + s.q0 + tok
                      : (int64_t(b) * a.KV * a.G + hq) * a.Sq + tok;
}

// Which workgroup of a key head, and which key head, blockIdx.x stands for: consecutive
// workgroups go to the 8 XCDs in turn, so where the heads divide by 8 all workgroups of
// one run on one XCD, whose L2 then holds its keys once.  An XCD takes its heads one after
// another, or (across) their first tiles before their second ones: under a causal mask
// tiles differ in their work, and the long ones of all heads come first so that none of them
// ends alone.  (us, head by head against across: 13 packed causal sequences of up to 2048 tokens,
// 16 heads of 64: forward 93, 76, dQ 125, 107; twice 4096 tokens of 32 heads on 8, dK and dV: 850,
// 640.  Without a mask, also of different lengths, across is slower: 16 of up to 1024 tokens, 32
// heads of 128: forward 197, 202.)
//
// part: of those that blockIdx.y counts.  An XCD deals its workgroups to four groups of CUs in
// turn, whatever their work; sequences of different lengths, whose parts would meet the same CUs
// again and again, move on by one with each part.  (One token over 8 caches of up to 32768: see
// even_chunk in attn_fwd.hip.)
__device__ __forceinline__ void head_and_tile(uint32_t heads, uint32_t tiles, bool across,
                                              uint32_t& head, uint32_t& tile, uint32_t part = 0)
{
    const uint32_t xcds = heads % 8 == 0 ? 8 : 1;
    const uint32_t x = blockIdx.x % xcds;
    uint32_t i = blockIdx.x / xcds;
    if (part > 0) i = (i + part) % (heads / xcds * tiles);
    if (across) {
        tile = i / (heads / xcds);
        head = x + xcds * (i % (heads / xcds));
    } else {
        head = x + xcds * (i / tiles);
        tile = i % tiles;
    }
}

}  // namespace iabn
