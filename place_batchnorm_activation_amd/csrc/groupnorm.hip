// Group norm with an activation, channels last: a sample's rows (pixels) of C channels,
// groups of C / G neighbouring ones.
//
//   xhat = (x - mean) * rstd over the pixels and channels of a group of a sample,
//   z = w_c xhat + b_c,  y = act(z);
//   dz = act'(z) dy,  dw_c = sum dz xhat,  db_c = sum dz,
//   dx = rstd (w dz - <w dz> - xhat <w dz xhat>),  <.> the mean over the group.
//
// Bound by memory.  A thread keeps 8 channels and walks rows, so that what belongs to a
// channel (weight, statistics, sums) stays in its registers and every access is a row's
// run of 16 bytes a lane, whatever the groups' width.
//
// Large maps: sums over runs of rows, a workgroup each, for each channel; a small kernel
// finishes them for the groups; an elementwise pass.  Two reads of x (three passes over
// x and dy in the backward), the second of which the 256 MB cache serves where the map
// fits it.  Small maps: one workgroup a group and sample reads it twice, the second time
// from its L2, in one launch.
//
// Statistics: a thread's rows about its own first value in fp32, joined as mean and sum of
// squares about it, the mean from the chunk's first value on (a mean far from zero takes no
// digits from the variance), the chunks in fp64.  Gradients' sums: fp32 within a workgroup,
// fp64 over them.  All in a fixed order.
#include <hip/hip_runtime.h>

#include "acts.hpp"
#include "gnorm.hpp"
#include "rows.hpp"

namespace iabn {

namespace {

constexpr int kGnThreads = 256;
constexpr int kBlockC = kGnThreads * kRowV;        // channels of a workgroup

// act(z) and act'(z).  SiLU without the gated unit's care for the ends (glu_act): z is a norm's
// output, finite where its group is, and s = 1/(1 + e^-z) reaches 0 and 1 by itself.  (Six
// operations less an element: the sums' pass is as near to the vector units' rate as to the
// memory's.)
template <int ACT>
__device__ __forceinline__ void gn_act(float z, float param, float& f, float& d)
{
    if constexpr (ACT == kGnIdentity) {
        f = z;
        d = 1.f;
    } else if constexpr (ACT == kGnLeaky) {
        f = z >= 0.f ? z : z * param;
        d = z >= 0.f ? 1.f : param;
        if (z != z) f = d = z;
    } else if constexpr (ACT == kGnSilu) {
        const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * z));
        f = z * s;
        d = s * fmaf(z, 1.f - s, 1.f);
    } else {
        glu_act<ACT>(z, f, d);
    }
}

// How a workgroup of rows lies over the tensor.
struct GnGrid {
    int64_t chunk;                    // rows of a workgroup
    int chunks, blocks;               // workgroups of a sample: along its rows, its channels
    FastDiv width;                    // by C / G
    int64_t n0;                       // first sample of the launch
};

// A thread's place: 8 channels from c on, rows first, first + step, ... of its chunk.
struct Place {
    int c, nv;                        // nv: valid channels, 0 none
    int lane, lanes;                  // row lanes of the workgroup
    int64_t row0, row1;
};

__device__ __forceinline__ Place place_of(const GnArgs& a, const GnGrid& gr)
{
    Place p;
    const int c0 = int(blockIdx.z) * kBlockC;
    const int vecs = (min(int(a.C) - c0, kBlockC) + kRowV - 1) / kRowV;
    p.lanes = kGnThreads / vecs;
    p.lane = int(threadIdx.x) / vecs;
    p.c = c0 + (int(threadIdx.x) - p.lane * vecs) * kRowV;
    p.nv = p.lane < p.lanes ? valid8(p.c, int(a.C)) : 0;
    p.row0 = int64_t(blockIdx.x) * gr.chunk;
    p.row1 = dmin(p.row0 + gr.chunk, a.HW);
    return p;
}

template <int DT>
__device__ __forceinline__ const char* sample_row(const void* t, int64_t ld, const GnArgs& a,
                                                  int64_t n, int64_t row)
{
    return row_ptr<DT>(t, n * a.HW + row, ld);
}

// What a channel's elementwise pass needs: z = (x - mean) * a + b, a = rstd * w.
struct Channel {
    float mean[8], rstd[8], a[8], b[8];
    int group[8];
};

template <bool WHOLE>
__device__ __forceinline__ void load_channels(const GnArgs& a, FastDiv width, int64_t n, int c,
                                              int nv, Channel& ch)
{
    load_cols<WHOLE>(a.weight, uint32_t(c), int(a.C), 1.f, ch.a);
    load_cols<WHOLE>(a.bias, uint32_t(c), int(a.C), 0.f, ch.b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        ch.group[e] = e < nv ? int(fast_div(uint32_t(c + e), width)) : int(a.G) - 1;
        const float2 st = reinterpret_cast<const float2*>(a.stats)[n * a.G + ch.group[e]];
        ch.mean[e] = st.x;
        ch.rstd[e] = st.y;
        ch.a[e] *= st.y;
    }
}

// The row lanes' pairs of each channel, joined in their order: out[c] of the block.
template <class Join>
__device__ __forceinline__ void join_lanes(const Place& p, const float (&s)[8],
                                           const float (&t)[8], float2* out, int C, Join&& join)
{
    __shared__ float2 all[kGnThreads * kRowV];
    const int c0 = int(blockIdx.z) * kBlockC, cols = min(C - c0, kBlockC);
    const int wide = (cols + kRowV - 1) / kRowV * kRowV;          // lanes * wide <= 256 * 8
    if (p.nv > 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) all[p.lane * wide + p.c - c0 + e] = make_float2(s[e], t[e]);
    }
    __syncthreads();
    for (int c = int(threadIdx.x); c < cols; c += kGnThreads) {
        float2 v = all[c];
        for (int l = 1; l < p.lanes; ++l) join(v, all[l * wide + c], l);
        out[c0 + c] = v;
    }
}

// part[n][chunk][c]: the mean of the chunk's rows, less its first, and the sum of squares about
// the mean.
template <int DT, bool WHOLE>
__global__ __launch_bounds__(kGnThreads) void k_gn_stats(GnArgs a, GnGrid gr, float2* part)
{
    const int64_t n = gr.n0 + blockIdx.y;
    const Place p = place_of(a, gr);
    const int C = int(a.C);
    const int rows = int(p.row1 - p.row0);
    auto count = [&](int lane) { return lane < rows ? (rows - lane + p.lanes - 1) / p.lanes : 0; };
    float s[8] = {}, t[8] = {};
    if (p.nv > 0 && p.lane < rows) {
        // sums about the thread's first value, which take no digits from the squares; means
        // from the chunk's first value, which keeps those of means far from zero
        float pivot[8], first[8];
        int64_t row = p.row0 + p.lane;
        widen8<DT>(load8<DT, WHOLE>(sample_row<DT>(a.x, a.ldx, a, n, p.row0), uint32_t(p.c), C), first);
        widen8<DT>(load8<DT, WHOLE>(sample_row<DT>(a.x, a.ldx, a, n, row), uint32_t(p.c), C), pivot);
        row += p.lanes;
        auto add = [&](const Raw8<DT>& r) {
            float v[8];
            widen8<DT>(r, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = v[e] - pivot[e];
                s[e] += d;
                t[e] = fmaf(d, d, t[e]);
            }
        };
        for (; row + 3 * p.lanes < p.row1; row += 4 * p.lanes) {
            Raw8<DT> r[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                r[u] = load8<DT, WHOLE>(sample_row<DT>(a.x, a.ldx, a, n, row + u * p.lanes),
                                        uint32_t(p.c), C);
#pragma unroll
            for (int u = 0; u < 4; ++u) add(r[u]);
        }
        for (; row < p.row1; row += p.lanes)
            add(load8<DT, WHOLE>(sample_row<DT>(a.x, a.ldx, a, n, row), uint32_t(p.c), C));
        const float inv = 1.f / float(count(p.lane));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q = fmaf(-s[e] * inv, s[e], t[e]);
            t[e] = q < 0.f ? 0.f : q;
            s[e] = fmaf(s[e], inv, pivot[e] - first[e]);
        }
    }
    join_lanes(p, s, t, part + (n * gr.chunks + blockIdx.x) * a.C, C,
               [&](float2& v, const float2& o, int l) {
        const int nb = count(l);
        if (nb == 0) return;
        // rows of the lanes before: whole rounds of them, and of the last round min(l, rest)
        const int na = rows / p.lanes * l + min(l, rows % p.lanes);
        const float f = float(nb) / float(na + nb), d = o.x - v.x;
        v.x = fmaf(d, f, v.x);
        v.y += o.y + d * d * float(na) * f;
    });
}

// The sum over a workgroup, in every thread.
template <int NT>
__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double all[NT / 64];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    __syncthreads();
    if (threadIdx.x % 64 == 0) all[threadIdx.x / 64] = v;
    __syncthreads();
    double s = 0.;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) s += all[i];
    return s;
}

// Statistics of a group from its channels' moments in each chunk; one workgroup a group.
template <int DT>
__global__ __launch_bounds__(kGnThreads) void k_gn_finish(GnArgs a, GnGrid gr, const float2* part)
{
    const int64_t g = blockIdx.x, n = gr.n0 + blockIdx.y, cg = a.C / a.G, c0 = g * cg;
    const float2* p = part + n * gr.chunks * a.C + c0;
    const double M = double(a.HW) * double(cg);
    const uint32_t all = uint32_t(cg) * uint32_t(gr.chunks);      // below 2^31: C and chunks are
    const char* x0 = sample_row<DT>(a.x, a.ldx, a, n, 0);
    const int64_t step = gr.chunk * a.ldx * (DT == kF32 ? 4 : 2);
    auto rows = [&](uint32_t i) { return double(dmin(gr.chunk, a.HW - i * gr.chunk)); };
    // the k-th channel mean, and its sum of squares
    auto value = [&](uint32_t k, uint32_t& i, float& m2) {
        i = fast_div(k, gr.width);
        const uint32_t c = k - i * uint32_t(cg);
        const float2 v = p[i * a.C + c];
        m2 = v.y;
        const char* row = x0 + i * step;
        float first;
        if constexpr (DT == kF32) first = reinterpret_cast<const float*>(row)[c0 + c];
        else first = unpack1<DT>(reinterpret_cast<const uint16_t*>(row)[c0 + c]);
        return double(first) + double(v.x);
    };
    double mean = 0., var = 0.;
#pragma unroll 4
    for (uint32_t k = threadIdx.x; k < all; k += kGnThreads) {
        uint32_t i;
        float m2;
        const double v = value(k, i, m2);
        mean += v * rows(i);
    }
    mean = block_sum<kGnThreads>(mean) / M;
#pragma unroll 4
    for (uint32_t k = threadIdx.x; k < all; k += kGnThreads) {
        uint32_t i;
        float m2;
        const double d = value(k, i, m2) - mean;
        var += double(m2) + d * d * rows(i);
    }
    var = block_sum<kGnThreads>(var) / M;
    if (threadIdx.x == 0)
        reinterpret_cast<float2*>(a.stats)[n * a.G + g] =
            make_float2(float(mean), float(1. / sqrt(var + double(a.eps))));
}

template <int DT, int ACT, bool WHOLE>
__global__ __launch_bounds__(kGnThreads) void k_gn_apply(GnArgs a, GnGrid gr)
{
    const int64_t n = gr.n0 + blockIdx.y;
    const Place p = place_of(a, gr);
    const int C = int(a.C);
    if (p.nv == 0) return;
    Channel ch;
    load_channels<WHOLE>(a, gr.width, n, p.c, p.nv, ch);
    auto one = [&](const Raw8<DT>& r, int64_t row) {
        float v[8], d;
        widen8<DT>(r, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            gn_act<ACT>(fmaf(v[e] - ch.mean[e], ch.a[e], ch.b[e]), a.param, v[e], d);
        store8<DT, WHOLE>(sample_row<DT>(a.out, a.ldo, a, n, row), uint32_t(p.c), C, v);
    };
    int64_t row = p.row0 + p.lane;
    for (; row + 3 * p.lanes < p.row1; row += 4 * p.lanes) {
        Raw8<DT> r[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            r[u] = load8<DT, WHOLE>(sample_row<DT>(a.x, a.ldx, a, n, row + u * p.lanes),
                                    uint32_t(p.c), C);
#pragma unroll
        for (int u = 0; u < 4; ++u) one(r[u], row + u * p.lanes);
    }
    for (; row < p.row1; row += p.lanes)
        one(load8<DT, WHOLE>(sample_row<DT>(a.x, a.ldx, a, n, row), uint32_t(p.c), C), row);
}

// x - mean and dz of 8 channels.
template <int DT, int ACT>
__device__ __forceinline__ void gn_grad(const Raw8<DT>& rx, const Raw8<DT>& rg, const Channel& ch,
                                        float param, float (&x)[8], float (&dz)[8])
{
    float g[8], f, d;
    widen8<DT>(rx, x);
    widen8<DT>(rg, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] -= ch.mean[e];
        gn_act<ACT>(fmaf(x[e], ch.a[e], ch.b[e]), param, f, d);
        dz[e] = g[e] * d;
    }
}

// dx = rstd (w dz - <w dz> - xhat <w dz xhat>) as a dz - k - (x - mean) m.
__device__ __forceinline__ void gn_dx(const Channel& ch, const float (&k)[8], const float (&m)[8],
                                      const float (&x)[8], float (&dz)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) dz[e] = fmaf(ch.a[e], dz[e], -fmaf(x[e], m[e], k[e]));
}

// part[n][chunk][c]: sums of dz and of dz * xhat.
template <int DT, int ACT, bool WHOLE>
__global__ __launch_bounds__(kGnThreads) void k_gn_sums(GnArgs a, GnGrid gr, float2* part)
{
    const int64_t n = gr.n0 + blockIdx.y;
    const Place p = place_of(a, gr);
    const int C = int(a.C);
    float s[8] = {}, t[8] = {};
    if (p.nv > 0) {
        Channel ch;
        load_channels<WHOLE>(a, gr.width, n, p.c, p.nv, ch);
        auto add = [&](const Raw8<DT>& rx, const Raw8<DT>& rg) {
            float x[8], dz[8];
            gn_grad<DT, ACT>(rx, rg, ch, a.param, x, dz);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[e] += dz[e];
                t[e] = fmaf(dz[e], x[e], t[e]);
            }
        };
        int64_t row = p.row0 + p.lane;
        constexpr int R = DT == kF32 ? 2 : 4;      // rows in flight
        for (; row + (R - 1) * p.lanes < p.row1; row += R * p.lanes) {
            Raw8<DT> rx[R], rg[R];
#pragma unroll
            for (int u = 0; u < R; ++u) {
                rx[u] = load8<DT, WHOLE>(sample_row<DT>(a.x, a.ldx, a, n, row + u * p.lanes),
                                         uint32_t(p.c), C);
                rg[u] = load8<DT, WHOLE>(sample_row<DT>(a.dy, a.lddy, a, n, row + u * p.lanes),
                                         uint32_t(p.c), C);
            }
#pragma unroll
            for (int u = 0; u < R; ++u) add(rx[u], rg[u]);
        }
        for (; row < p.row1; row += p.lanes)
            add(load8<DT, WHOLE>(sample_row<DT>(a.x, a.ldx, a, n, row), uint32_t(p.c), C),
                load8<DT, WHOLE>(sample_row<DT>(a.dy, a.lddy, a, n, row), uint32_t(p.c), C));
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] *= ch.rstd[e];
    }
    join_lanes(p, s, t, part + (n * gr.chunks + blockIdx.x) * a.C, C,
               [](float2& v, const float2& o, int) {
        v.x += o.x;
        v.y += o.y;
    });
}

// sums[n][c] over the chunks, and coef[n][g] = (<w dz>, <w dz xhat>).
__global__ __launch_bounds__(kGnThreads) void k_gn_finish_sums(GnArgs a, GnGrid gr,
                                                              const float2* part, float2* sums,
                                                              float2* coef)
{
    const int64_t g = blockIdx.x, n = gr.n0 + blockIdx.y, cg = a.C / a.G, c0 = g * cg;
    __shared__ double2 all[kGnThreads];
    double u = 0., v = 0.;
    for (int64_t cb = 0; cb < cg; cb += kGnThreads) {             // 256 channels at a time
        const int wide = int(dmin(cg - cb, kGnThreads)), lanes = kGnThreads / wide;
        const int lane = int(threadIdx.x) / wide, c = int(threadIdx.x) - lane * wide;
        double s = 0., t = 0.;
        if (lane < lanes) {
            const float2* p = part + n * gr.chunks * a.C + c0 + cb + c;
#pragma unroll 4
            for (int i = lane; i < gr.chunks; i += lanes) {
                const float2 x = p[i * a.C];
                s += double(x.x);
                t += double(x.y);
            }
        }
        __syncthreads();
        all[threadIdx.x] = make_double2(s, t);
        __syncthreads();
        if (lane == 0) {
            for (int l = 1; l < lanes; ++l) {
                s += all[l * wide + c].x;
                t += all[l * wide + c].y;
            }
            const double w = a.weight ? double(a.weight[c0 + cb + c]) : 1.;
            sums[n * a.C + c0 + cb + c] = make_float2(float(s), float(t));
            u += w * s;
            v += w * t;
        }
    }
    const double M = double(a.HW) * double(cg);
    u = block_sum<kGnThreads>(u) / M;
    v = block_sum<kGnThreads>(v) / M;
    if (threadIdx.x == 0) coef[n * a.G + g] = make_float2(float(u), float(v));
}

// dw and db: the samples' sums, in their order.
__device__ __forceinline__ void add_samples(const GnArgs& a, const float2* sums, int64_t c)
{
    if (c >= a.C) return;
    double s = 0., t = 0.;
#pragma unroll 4
    for (int64_t n = 0; n < a.N; ++n) {
        const float2 v = sums[n * a.C + c];
        s += double(v.x);
        t += double(v.y);
    }
    if (a.dbias) a.dbias[c] = float(s);
    if (a.dweight) a.dweight[c] = float(t);
}

__global__ __launch_bounds__(kGnThreads) void k_gn_dparams(GnArgs a, const float2* sums)
{
    add_samples(a, sums, int64_t(blockIdx.x) * kGnThreads + threadIdx.x);
}

template <int DT, int ACT, bool WHOLE>
__global__ __launch_bounds__(kGnThreads) void k_gn_dx(GnArgs a, GnGrid gr, const float2* coef,
                                                       const float2* sums)
{
    if (int(blockIdx.x) >= gr.chunks) {            // behind the rows: dw and db
        if (blockIdx.y == 0 && blockIdx.z == 0)
            add_samples(a, sums, int64_t(int(blockIdx.x) - gr.chunks) * kGnThreads + threadIdx.x);
        return;
    }
    const int64_t n = gr.n0 + blockIdx.y;
    const Place p = place_of(a, gr);
    const int C = int(a.C);
    if (p.nv == 0) return;
    Channel ch;
    load_channels<WHOLE>(a, gr.width, n, p.c, p.nv, ch);
    float k[8], m[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float2 v = coef[n * a.G + ch.group[e]];
        k[e] = v.x * ch.rstd[e];
        m[e] = v.y * ch.rstd[e] * ch.rstd[e];
    }
    auto one = [&](const Raw8<DT>& rx, const Raw8<DT>& rg, int64_t row) {
        float x[8], dz[8];
        gn_grad<DT, ACT>(rx, rg, ch, a.param, x, dz);
        gn_dx(ch, k, m, x, dz);
        store8<DT, WHOLE>(sample_row<DT>(a.out, a.ldo, a, n, row), uint32_t(p.c), C, dz);
    };
    int64_t row = p.row0 + p.lane;
    for (; row + p.lanes < p.row1; row += 2 * p.lanes) {
        Raw8<DT> rx[2], rg[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            rx[u] = load8<DT, WHOLE>(sample_row<DT>(a.x, a.ldx, a, n, row + u * p.lanes),
                                     uint32_t(p.c), C);
            rg[u] = load8<DT, WHOLE>(sample_row<DT>(a.dy, a.lddy, a, n, row + u * p.lanes),
                                     uint32_t(p.c), C);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) one(rx[u], rg[u], row + u * p.lanes);
    }
    for (; row < p.row1; row += p.lanes)
        one(load8<DT, WHOLE>(sample_row<DT>(a.x, a.ldx, a, n, row), uint32_t(p.c), C),
            load8<DT, WHOLE>(sample_row<DT>(a.dy, a.lddy, a, n, row), uint32_t(p.c), C), row);
}

// ---------------------------------------------------------------------------
// small maps: a workgroup a sample's group, which it reads twice

constexpr int kGroupThreads = 512;

// Workgroups go to the 8 XCDs in turn; neighbouring groups share memory lines, so each XCD
// takes a run of them.
__device__ __forceinline__ void group_of(const GnArgs& a, int64_t& n, int64_t& g)
{
    const uint32_t per = gridDim.x / 8;
    const uint32_t i = gridDim.x % 8 == 0 ? blockIdx.x % 8 * per + blockIdx.x / 8 : blockIdx.x;
    n = i / uint32_t(a.G);
    g = i % uint32_t(a.G);
}

struct GroupPlace {
    int c, nv, lane, lanes;
};

__device__ __forceinline__ GroupPlace group_place(int cg)
{
    const int vecs = (cg + kRowV - 1) / kRowV;
    GroupPlace p;
    p.lanes = kGroupThreads / vecs;
    p.lane = int(threadIdx.x) / vecs;
    p.c = (int(threadIdx.x) - p.lane * vecs) * kRowV;
    p.nv = p.lane < p.lanes ? valid8(p.c, cg) : 0;
    return p;
}

template <int DT, int ACT, bool WHOLE>
__global__ __launch_bounds__(kGroupThreads) void k_gn_group(GnArgs a)
{
    constexpr int ES = DT == kF32 ? 4 : 2;
    int64_t n, g;
    group_of(a, n, g);
    const int cg = int(a.C / a.G), HW = int(a.HW);
    const int64_t c0 = g * cg;
    const GroupPlace p = group_place(cg);
    auto load = [&](int row) {
        return load8<DT, WHOLE>(sample_row<DT>(a.x, a.ldx, a, n, row) + c0 * ES, uint32_t(p.c), cg);
    };
    // a thread's rows about its first one, as in k_gn_stats
    float pivot[8] = {}, mean[8] = {};             // mean: from the pivot
    double sum = 0., m2 = 0.;
    const int count = p.nv > 0 && p.lane < HW ? (HW - p.lane + p.lanes - 1) / p.lanes : 0;
    if (count > 0) {
        float t[8] = {};
        widen8<DT>(load(p.lane), pivot);
        auto add = [&](const Raw8<DT>& r) {
            float v[8];
            widen8<DT>(r, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = v[e] - pivot[e];
                mean[e] += d;
                t[e] = fmaf(d, d, t[e]);
            }
        };
        int row = p.lane + p.lanes;
        for (; row + 3 * p.lanes < HW; row += 4 * p.lanes) {
            Raw8<DT> r[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) r[u] = load(row + u * p.lanes);
#pragma unroll
            for (int u = 0; u < 4; ++u) add(r[u]);
        }
        for (; row < HW; row += p.lanes) add(load(row));
        const float inv = 1.f / float(count);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e >= p.nv) continue;
            const float q = fmaf(-mean[e] * inv, mean[e], t[e]);
            mean[e] *= inv;
            m2 += double(q < 0.f ? 0.f : q);
            sum += (double(pivot[e]) + double(mean[e])) * count;
        }
    }
    const double M = double(HW) * cg;
    sum = block_sum<kGroupThreads>(sum) / M;
    if (count > 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double d = double(pivot[e]) - sum + double(mean[e]);
            if (e < p.nv) m2 += d * d * count;
        }
    }
    const double var = block_sum<kGroupThreads>(m2) / M;
    const float mu = float(sum), rstd = float(1. / sqrt(var + double(a.eps)));
    if (threadIdx.x == 0 && a.stats)
        reinterpret_cast<float2*>(a.stats)[n * a.G + g] = make_float2(mu, rstd);
    if (p.nv == 0) return;
    float w[8], b[8], d;
    load_cols<WHOLE>(a.weight ? a.weight + c0 : nullptr, uint32_t(p.c), cg, 1.f, w);
    load_cols<WHOLE>(a.bias ? a.bias + c0 : nullptr, uint32_t(p.c), cg, 0.f, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= rstd;
    auto put = [&](const Raw8<DT>& r, int row) {
        float v[8];
        widen8<DT>(r, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) gn_act<ACT>(fmaf(v[e] - mu, w[e], b[e]), a.param, v[e], d);
        store8<DT, WHOLE>(sample_row<DT>(a.out, a.ldo, a, n, row) + c0 * ES, uint32_t(p.c), cg, v);
    };
    int row = p.lane;
    for (; row + 3 * p.lanes < HW; row += 4 * p.lanes) {
        Raw8<DT> r[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) r[u] = load(row + u * p.lanes);
#pragma unroll
        for (int u = 0; u < 4; ++u) put(r[u], row + u * p.lanes);
    }
    for (; row < HW; row += p.lanes) put(load(row), row);
}

// sums[n][c] for dw and db, and dx.
template <int DT, int ACT, bool WHOLE>
__global__ __launch_bounds__(kGroupThreads) void k_gn_group_grad(GnArgs a, float2* sums)
{
    constexpr int ES = DT == kF32 ? 4 : 2;
    __shared__ float2 all[kGroupThreads * kRowV];
    int64_t n, g;
    group_of(a, n, g);
    const int cg = int(a.C / a.G), HW = int(a.HW);
    const int64_t c0 = g * cg;
    const GroupPlace p = group_place(cg);
    const float2 st = reinterpret_cast<const float2*>(a.stats)[n * a.G + g];
    Channel ch;
    load_cols<WHOLE>(a.weight ? a.weight + c0 : nullptr, uint32_t(p.c), cg, 1.f, ch.a);
    load_cols<WHOLE>(a.bias ? a.bias + c0 : nullptr, uint32_t(p.c), cg, 0.f, ch.b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        ch.mean[e] = st.x;
        ch.a[e] *= st.y;
    }
    auto load = [&](const void* t, int64_t ld, int row) {
        return load8<DT, WHOLE>(sample_row<DT>(t, ld, a, n, row) + c0 * ES, uint32_t(p.c), cg);
    };
    const int wide = (cg + kRowV - 1) / kRowV * kRowV;
    if (p.nv > 0) {
        float s[8] = {}, t[8] = {}, x[8], dz[8];
        auto add = [&](const Raw8<DT>& rx, const Raw8<DT>& rg) {
            gn_grad<DT, ACT>(rx, rg, ch, a.param, x, dz);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[e] += dz[e];
                t[e] = fmaf(dz[e], x[e], t[e]);
            }
        };
        int row = p.lane;
        for (; row + p.lanes < HW; row += 2 * p.lanes) {
            const Raw8<DT> x0 = load(a.x, a.ldx, row), g0 = load(a.dy, a.lddy, row);
            const Raw8<DT> x1 = load(a.x, a.ldx, row + p.lanes);
            const Raw8<DT> g1 = load(a.dy, a.lddy, row + p.lanes);
            add(x0, g0);
            add(x1, g1);
        }
        for (; row < HW; row += p.lanes) add(load(a.x, a.ldx, row), load(a.dy, a.lddy, row));
#pragma unroll
        for (int e = 0; e < 8; ++e) all[p.lane * wide + p.c + e] = make_float2(s[e], t[e] * st.y);
    }
    __syncthreads();
    // a channel's lanes: runs of them by one thread each, the runs by the channel's own
    const int runs = max(1, min(p.lanes, kGroupThreads / wide)), per = (p.lanes + runs - 1) / runs;
    const int run = int(threadIdx.x) / wide, rc = int(threadIdx.x) - run * wide;
    float2 part = make_float2(0.f, 0.f);
    if (run < runs) {
#pragma unroll 4
        for (int l = run * per; l < min(run * per + per, p.lanes); ++l) {
            part.x += all[l * wide + rc].x;
            part.y += all[l * wide + rc].y;
        }
    }
    __syncthreads();
    if (run < runs) all[run * wide + rc] = part;
    __syncthreads();
    double u = 0., v = 0.;
    if (const int c = int(threadIdx.x); c < cg) {
        double s = 0., t = 0.;
        for (int l = 0; l < runs; ++l) {
            s += double(all[l * wide + c].x);
            t += double(all[l * wide + c].y);
        }
        const double w = a.weight ? double(a.weight[c0 + c]) : 1.;
        sums[n * a.C + c0 + c] = make_float2(float(s), float(t));
        u += w * s;
        v += w * t;
    }
    const double M = double(HW) * cg;
    u = block_sum<kGroupThreads>(u) / M;
    v = block_sum<kGroupThreads>(v) / M;
    if (p.nv == 0 || !a.out) return;
    float k[8], m[8], x[8], dz[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        k[e] = float(u) * st.y;
        m[e] = float(v) * st.y * st.y;
    }
    auto put = [&](const Raw8<DT>& rx, const Raw8<DT>& rg, int row) {
        gn_grad<DT, ACT>(rx, rg, ch, a.param, x, dz);
        gn_dx(ch, k, m, x, dz);
        store8<DT, WHOLE>(sample_row<DT>(a.out, a.ldo, a, n, row) + c0 * ES, uint32_t(p.c), cg, dz);
    };
    int row = p.lane;
    for (; row + p.lanes < HW; row += 2 * p.lanes) {
        const Raw8<DT> x0 = load(a.x, a.ldx, row), g0 = load(a.dy, a.lddy, row);
        const Raw8<DT> x1 = load(a.x, a.ldx, row + p.lanes), g1 = load(a.dy, a.lddy, row + p.lanes);
        put(x0, g0, row);
        put(x1, g1, row + p.lanes);
    }
    for (; row < HW; row += p.lanes) put(load(a.x, a.ldx, row), load(a.dy, a.lddy, row), row);
}

// Whether a workgroup a group takes the map: up to 1024 of them (four a CU), whose elements, in
// whole vectors and twice where the last one is ragged, are few.  us, one workgroup a group
// against many, forward and backward, bf16: 8 x 32^2 x 512 in 32 groups 9 against 15, 14
// against 19; 2 x 48^2 x 512 11, 15, 20, 19; 2 x 64^2 x 512 15, 17, 28, 19; 1 x 64^2 x 320 21,
// 17, 38, 19; 64 x 32^2 x 256 (2048 groups) 31, 27, 72, 46.  Ragged groups: 3 x 1073 x 150 in
// 10 groups of 15 (17168 elements, twice) 12, 18, 18, 23; 3 x 2146 17, 18, 29, 23; 3 x 4000 30,
// 19, 56, 23; 16 x 600 x 360 in 30 of 12 (9600) 11, 15, 19, 20; 16 x 1200 18, 18, 27, 24.
bool small_map(int64_t N, int64_t HW, int64_t C, int64_t G, int64_t most)
{
    const int64_t cg = C / G, wide = ceil_div(cg, kRowV) * kRowV;
    return cg >= kRowV && cg <= kGroupThreads && N * G <= 1024 &&
           HW * wide * (cg % kRowV ? 2 : 1) <= most;
}

constexpr int64_t kSmallForward = 1 << 16, kSmallBackward = 36000;

// Workgroups of rows: four a CU where the rows give them, each at least 8 rows a lane.
GnGrid make_grid(int64_t N, int64_t HW, int64_t C, int64_t G, int64_t cus)
{
    GnGrid gr{};
    gr.width = make_fast_div(uint32_t(C / G));
    gr.blocks = int(ceil_div(C, kBlockC));
    const int64_t lanes = max64(1, kGnThreads / ceil_div(min64(C, kBlockC), kRowV));
    const int64_t want = max64(1, ceil_div(4 * cus, N * gr.blocks));
    gr.chunk = max64(8 * lanes, ceil_div(HW, want));
    gr.chunks = int(ceil_div(HW, gr.chunk));
    return gr;
}

constexpr int64_t kMostSamples = 32768;            // of a grid's second extent

// Calls f(grid of a run of samples, its workgroups of rows, its groups).
template <class F>
void each_samples(const GnArgs& a, GnGrid gr, F&& f)
{
    for (gr.n0 = 0; gr.n0 < a.N; gr.n0 += kMostSamples) {
        const unsigned n = unsigned(min64(kMostSamples, a.N - gr.n0));
        f(gr, dim3(unsigned(gr.chunks), n, unsigned(gr.blocks)), dim3(unsigned(a.G), n));
    }
}

// Calls f(std::integral_constant<int, ACT>).
template <class F>
void with_gn_act(int act, F&& f)
{
    switch (act) {
    case kGnSilu: f(std::integral_constant<int, kGnSilu>{}); break;
    case kGnGelu: f(std::integral_constant<int, kGnGelu>{}); break;
    case kGnGeluTanh: f(std::integral_constant<int, kGnGeluTanh>{}); break;
    case kGnIdentity: f(std::integral_constant<int, kGnIdentity>{}); break;
    case kGnLeaky: f(std::integral_constant<int, kGnLeaky>{}); break;
    default: break;
    }
}

}  // namespace

// part [N][chunks][C], sums [N][C], coef [N][G] (float2 each); the forward's statistics
// where the caller wants none take sums' place.
size_t gn_workspace_bytes(int64_t N, int64_t HW, int64_t C, int64_t G, int64_t cus)
{
    const GnGrid gr = make_grid(N, HW, C, G, cus);
    return size_t(N) * 8 * (size_t(gr.chunks) * size_t(C) + size_t(C) + size_t(G));
}

void launch_gn_forward(const GnArgs& a0, int dtype, int64_t cus, void* ws, hipStream_t s)
{
    GnArgs a = a0;
    if (small_map(a.N, a.HW, a.C, a.G, kSmallForward)) {
        with_dtype(dtype, [&](auto d) {
            with_whole(a.C / a.G, [&](auto wh) {
                with_gn_act(a.act, [&](auto act) {
                    hipLaunchKernelGGL((k_gn_group<decltype(d)::value, decltype(act)::value,
                                                   decltype(wh)::value>),
                                       dim3(unsigned(a.N * a.G)), dim3(kGroupThreads), 0, s, a);
                });
            });
        });
        return;
    }
    const GnGrid gr = make_grid(a.N, a.HW, a.C, a.G, cus);
    float2* part = static_cast<float2*>(ws);
    if (!a.stats) a.stats = reinterpret_cast<float*>(part + a.N * gr.chunks * a.C);
    with_dtype(dtype, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        with_whole(a.C, [&](auto wh) {
            constexpr bool W = decltype(wh)::value;
            each_samples(a, gr, [&](const GnGrid& g, dim3 grid, dim3 groups) {
                hipLaunchKernelGGL((k_gn_stats<DT, W>), grid, dim3(kGnThreads), 0, s, a, g, part);
                hipLaunchKernelGGL((k_gn_finish<DT>), groups, dim3(kGnThreads), 0, s, a, g, part);
                with_gn_act(a.act, [&](auto act) {
                    hipLaunchKernelGGL((k_gn_apply<DT, decltype(act)::value, W>), grid,
                                       dim3(kGnThreads), 0, s, a, g);
                });
            });
        });
    });
}

void launch_gn_backward(const GnArgs& a, int dtype, int64_t cus, void* ws, hipStream_t s)
{
    auto params = [&](const float2* sums, int64_t n) {
        GnArgs b = a;
        b.N = n;
        if (a.dweight || a.dbias)
            hipLaunchKernelGGL(k_gn_dparams, dim3(unsigned(ceil_div(a.C, kGnThreads))),
                               dim3(kGnThreads), 0, s, b, sums);
    };
    if (a.N == 0 || a.HW == 0) return params(nullptr, 0);         // zeros
    if (small_map(a.N, a.HW, a.C, a.G, kSmallBackward)) {
        float2* sums = static_cast<float2*>(ws);
        with_dtype(dtype, [&](auto d) {
            with_whole(a.C / a.G, [&](auto wh) {
                with_gn_act(a.act, [&](auto act) {
                    hipLaunchKernelGGL((k_gn_group_grad<decltype(d)::value, decltype(act)::value,
                                                        decltype(wh)::value>),
                                       dim3(unsigned(a.N * a.G)), dim3(kGroupThreads), 0, s, a, sums);
                });
            });
        });
        return params(sums, a.N);
    }
    const GnGrid gr = make_grid(a.N, a.HW, a.C, a.G, cus);
    float2* part = static_cast<float2*>(ws);
    float2* sums = part + a.N * gr.chunks * a.C;
    float2* coef = sums + a.N * a.C;
    // dw and db by workgroups of the last pass, unless they replace the vectors that it reads or
    // the samples take several launches
    const bool fold = a.out && (a.dweight || a.dbias) && a.dweight != a.weight &&
                      a.dbias != a.bias && a.N <= kMostSamples;
    with_dtype(dtype, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        with_whole(a.C, [&](auto wh) {
            constexpr bool W = decltype(wh)::value;
            with_gn_act(a.act, [&](auto act) {
                constexpr int A = decltype(act)::value;
                each_samples(a, gr, [&](const GnGrid& g, dim3 grid, dim3 groups) {
                    hipLaunchKernelGGL((k_gn_sums<DT, A, W>), grid, dim3(kGnThreads), 0, s, a, g,
                                       part);
                    hipLaunchKernelGGL(k_gn_finish_sums, groups, dim3(kGnThreads), 0, s, a, g,
                                       part, sums, coef);
                    if (a.out) {
                        dim3 wide = grid;
                        if (fold) wide.x += unsigned(ceil_div(a.C, kGnThreads));
                        hipLaunchKernelGGL((k_gn_dx<DT, A, W>), wide, dim3(kGnThreads), 0, s, a, g,
                                           coef, sums);
                    }
                });
            });
        });
    });
    if (!fold) params(sums, a.N);
}

}  // namespace iabn
