// Group norm over a row's channels with an activation or gate, and its gradients.
//
// Bound by HBM: the forward reads x (and z) and writes out, the backward reads x, dout (and z) and
// writes dx (and dz), each once. A group lives in the registers of LPG lanes of one warp (NV
// 16-byte vectors a lane), so the statistics are a few shuffles, the deviations are squared from
// registers (no E[x^2] - mean^2 cancellation) and nothing is read twice. Groups too large, or rows
// not 16-byte aligned, take one CTA per group with scalar loads. Statistics, sums and arithmetic
// are fp32; each output is rounded once. bf16, 8192 rows of 4096 channels in groups of 64, centred and
// gated: forward 40.4 us (5.0 TB/s; a copy reaches 6.4), backward 80 us (4.2 TB/s). No unit is full in either (an
// instruction is issued in 62 and 53 % of the cycles, the FMA pipe busy in half of them): the registers hold 32
// and 16 warps an SM, which wait for their loads and for one another's results.
//
// Backward, with xh = (x - mean) r, y = xh w + b, s = act(z) or act(y):
//     dy = dout s (gate) or dout act'(y),  dz = dout y act'(z),  g = dy w,
//     dx = r (g - xh mean(g xh) - mean(g) [centred]),  dw = sum_rows dy xh,  db = sum_rows dy.
// Threads keep their columns and walk down the rows, so dw and db are summed in registers; a CTA's
// shares go to the workspace and a second launch adds them in a fixed order.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "m3_common.cuh"
#include "m3_internal.h"
#include "m3_sm100.cuh"
#include "m3_vec.cuh"

namespace m3 {
namespace {

// A tensor [batch][rows][G][D] by its strides, in elements.
struct GnTensor {
    void* p;
    int64_t batch, row, group;
};
struct GnParams {
    uint32_t rows, inner;                   // rows in all, and of each batch entry
    int C, G, D;
    GnTensor x, z, out, dout, dx, dz;
    const float *w, *b;
    float *dw, *db;
    float* part;                            // backward: [shares][2][C]
    uint32_t share_rows;                    // rows of one share
    int shares;
    float eps;
};

// A group's first element. T may be const.
template <typename T>
__device__ __forceinline__ T* at(const GnTensor& t, const GnParams& p, uint32_t row, int group) {
    const uint32_t b = p.inner == p.rows ? 0u : row / p.inner;
    return static_cast<T*>(t.p) + b * t.batch + static_cast<int64_t>(row - b * p.inner) * t.row + group * t.group;
}

constexpr int kThreads = 256;

// 1 / (1 + e^-v); e^-v = inf gives 0. The approximate divide is within 2 units in the last place.
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }
template <bool kSilu>
__device__ __forceinline__ float act(float v) { return kSilu ? v * sigmoid(v) : v; }
// act(v) and its slope
template <bool kSilu>
__device__ __forceinline__ void act_slope(float v, float* a, float* da) {
    if (!kSilu) { *a = v; *da = 1.f; return; }
    const float s = sigmoid(v);
    *a = v * s;
    *da = s * fmaf(v, 1.f - s, 1.f);
}
template <bool kSilu>
__device__ __forceinline__ float2 act2(const float2& v) { return kSilu ? mul2(v, sigmoid2(v)) : v; }
template <bool kSilu>
__device__ __forceinline__ void act_slope2(const float2& v, float2* a, float2* da) {
    if (!kSilu) { *a = v; *da = both(1.f); return; }
    const float2 s = sigmoid2(v);
    *a = mul2(v, s);
    *da = fma2(*a, fma2(s, both(-1.f), both(1.f)), s);      // s (1 + v (1 - s))
}

// the sum over the LPG lanes that hold a group
template <int LPG>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LPG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// v becomes the group's deviations from the mean (or stays, without centring); returns
// 1 / sqrt(var + eps). Vectors beyond the group's end hold zeros and keep them.
template <int LPG, int NV, int N, bool kCenter>
__device__ __forceinline__ float stats(float2 (&v)[NV][N], const bool (&in)[NV], float inv, float eps) {
    if (kCenter) {
        float2 s = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) s = add2(s, v[i][e]);
        const float m = group_sum<LPG>(s.x + s.y) * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float2 mi = both(in[i] ? -m : 0.f);
#pragma unroll
            for (int e = 0; e < N; ++e) v[i][e] = add2(v[i][e], mi);
        }
    }
    float2 q = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) q = fma2(v[i][e], v[i][e], q);
    return rsqrtf(fmaf(group_sum<LPG>(q.x + q.y), inv, eps));
}

// The row walk of both directions. A CTA's threads lie side by side over gx whole groups and, where
// those are narrower than the CTA, over nry rows; they keep their columns (and so the weights) and
// walk down the share's rows, the next row's loads in flight while one is worked on (two rows ahead
// measured the same within 3 %).
template <typename T, int LPG, int NV>
struct Walk {
    static constexpr int N = 2 * Vec<T>::N;     // elements of a vector
    int lane, ry, nry, group, c0;
    uint32_t row, r1, turns;
    bool col_ok, in[NV];
    __device__ __forceinline__ Walk(const GnParams& p, int gx) {
        lane = threadIdx.x % LPG;
        const int grp = threadIdx.x / LPG;
        nry = (kThreads / LPG) / gx;
        ry = grp / gx;
        group = blockIdx.x * gx + grp % gx;
        col_ok = group < p.G && ry < nry;
        c0 = group * p.D;
        const uint32_t r0 = blockIdx.y * p.share_rows;
        r1 = min(r0 + p.share_rows, p.rows);
        row = r0 + ry;
        turns = (r1 - r0 + nry - 1) / nry;      // the same for every thread: the shuffles need whole warps
#pragma unroll
        for (int i = 0; i < NV; ++i) in[i] = col_ok && (i * LPG + lane) * N < p.D;
    }
    __device__ __forceinline__ int col(int i) const { return (i * LPG + lane) * N; }
    // this thread's vectors of one row, zeros where it has none
    __device__ __forceinline__ void fetch(const GnParams& p, const GnTensor& t, uint32_t r, uint4 (&raw)[NV]) const {
        const bool live = col_ok && r < r1;
        const T* src = live ? at<const T>(t, p, r, group) : nullptr;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            raw[i] = live && in[i] ? __ldcs(reinterpret_cast<const uint4*>(src + col(i))) : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void weights(const float* src, float other, float2 (&w)[NV][N / 2]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
                const float* at = src + c0 + col(i) + 2 * e;
                w[i][e] = src && in[i] ? make_float2(__ldg(at), __ldg(at + 1)) : both(other);
            }
    }
};

template <typename T, int LPG, int NV, bool kCenter, bool kSilu, bool kGate>
__global__ void __launch_bounds__(kThreads) gn_fwd_kernel(const GnParams p, int gx) {
    constexpr int N = Vec<T>::N;
    Walk<T, LPG, NV> k(p, gx);
    uint4 rx[NV], rz[NV];
    k.fetch(p, p.x, k.row, rx);
    if (kGate) k.fetch(p, p.z, k.row, rz);
    float2 w[NV][N], b[NV][N];
    k.weights(p.w, 1.f, w);
    k.weights(p.b, 0.f, b);
    const float inv = 1.f / p.D;
    for (uint32_t t = 0; t < k.turns; ++t, k.row += k.nry) {
        float2 v[NV][N], g[NV][N];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Vec<T>::unpack(rx[i], v[i]);
            if (kGate) Vec<T>::unpack(rz[i], g[i]);
        }
        k.fetch(p, p.x, k.row + k.nry, rx);
        if (kGate) k.fetch(p, p.z, k.row + k.nry, rz);
        const float r = stats<LPG, NV, N, kCenter>(v, k.in, inv, p.eps);
        if (!(k.col_ok && k.row < k.r1)) continue;
        T* out = at<T>(p.out, p, k.row, k.group);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!k.in[i]) continue;
            float2 o[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float2 y = fma2(mul2(v[i][e], both(r)), w[i][e], b[i][e]);
                o[e] = kGate ? mul2(y, act2<kSilu>(g[i][e])) : act2<kSilu>(y);
            }
            Vec<T>::store(out + k.col(i), o);
        }
    }
}

template <typename T, int LPG, int NV, bool kCenter, bool kSilu, bool kGate>
__global__ void __launch_bounds__(kThreads) gn_bwd_kernel(const GnParams p, int gx) {
    constexpr int N = Vec<T>::N;
    extern __shared__ float s_part[];
    sm100::grid_dep_launch_dependents();
    Walk<T, LPG, NV> k(p, gx);
    uint4 rx[NV], rz[NV], rd[NV];
    k.fetch(p, p.x, k.row, rx);
    k.fetch(p, p.dout, k.row, rd);
    if (kGate) k.fetch(p, p.z, k.row, rz);
    float2 w[NV][N], b[NV][N], dw[NV][N], db[NV][N];
    k.weights(p.w, 1.f, w);
    k.weights(p.b, 0.f, b);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) dw[i][e] = db[i][e] = both(0.f);
    const float inv = 1.f / p.D;
    for (uint32_t t = 0; t < k.turns; ++t, k.row += k.nry) {
        float2 v[NV][N], dy[NV][N], z[NV][N];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Vec<T>::unpack(rx[i], v[i]);
            Vec<T>::unpack(rd[i], dy[i]);
            if (kGate) Vec<T>::unpack(rz[i], z[i]);
        }
        const uint32_t row = k.row;
        const bool live = k.col_ok && row < k.r1;
        k.fetch(p, p.x, row + k.nry, rx);
        k.fetch(p, p.dout, row + k.nry, rd);
        if (kGate) k.fetch(p, p.z, row + k.nry, rz);
        float r = stats<LPG, NV, N, kCenter>(v, k.in, inv, p.eps);
        r = live ? r : 0.f;         // with eps = 0 an absent row's would be infinite
        float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                v[i][e] = mul2(v[i][e], both(r));
                const float2 y = fma2(v[i][e], w[i][e], b[i][e]), d = dy[i][e];
                float2 a, da;
                act_slope2<kSilu>(kGate ? z[i][e] : y, &a, &da);
                if (kGate) z[i][e] = mul2(mul2(d, y), da);      // dz
                const float2 g = mul2(d, kGate ? a : da);       // (absent elements have dout = 0)
                dw[i][e] = fma2(g, v[i][e], dw[i][e]);
                db[i][e] = add2(db[i][e], g);
                dy[i][e] = mul2(g, w[i][e]);
                s1 = fma2(dy[i][e], v[i][e], s1);
                s2 = add2(s2, dy[i][e]);
            }
        }
        const float m1 = -group_sum<LPG>(s1.x + s1.y) * inv, m2 = kCenter ? -group_sum<LPG>(s2.x + s2.y) * inv : 0.f;
        if (!live) continue;
        T* dx = at<T>(p.dx, p, row, k.group);
        T* dz = kGate ? at<T>(p.dz, p, row, k.group) : nullptr;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!k.in[i]) continue;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                float2 g = fma2(v[i][e], both(m1), dy[i][e]);
                if (kCenter) g = add2(g, both(m2));
                dy[i][e] = mul2(g, both(r));
            }
            Vec<T>::store(dx + k.col(i), dy[i]);
            if (kGate) Vec<T>::store(dz + k.col(i), z[i]);
        }
    }
    if (!p.dw && !p.db) return;
    // the CTA's rows are added group row by group row
    const int width = gx * p.D;
    float* sw = s_part;
    float* sb = s_part + width;
    for (int y = 0; y < k.nry; ++y) {
        if (k.ry == y) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!k.in[i]) continue;
                const int c = (k.group - blockIdx.x * gx) * p.D + k.col(i);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    float2 *tw = reinterpret_cast<float2*>(sw + c) + e, *tb = reinterpret_cast<float2*>(sb + c) + e;
                    *tw = y ? add2(*tw, dw[i][e]) : dw[i][e];
                    *tb = y ? add2(*tb, db[i][e]) : db[i][e];
                }
            }
        }
        __syncthreads();
    }
    const int col0 = blockIdx.x * width;
    float* part = p.shares > 1 ? p.part + static_cast<int64_t>(blockIdx.y) * 2 * p.C : nullptr;
    float *ow = part ? part : p.dw, *ob = part ? part + p.C : p.db;     // a single share is the sum
    for (int c = threadIdx.x; c < width && col0 + c < p.C; c += kThreads) {
        if (ow) ow[col0 + c] = sw[c];
        if (ob) ob[col0 + c] = sb[c];
    }
}

// dweight and dbias: the shares of one column added in order by 32 threads, then those by a tree
__global__ void __launch_bounds__(1024) gn_shares_kernel(const GnParams p) {
    __shared__ float s[32][33];
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + cx;   // of 2 C columns
    sm100::grid_dep_wait();     // may have started while the shares were formed
    float sum = 0.f;
    if (c < 2 * static_cast<int64_t>(p.C))
#pragma unroll 4
        for (int k = ry; k < p.shares; k += 32) sum += __ldcg(p.part + static_cast<int64_t>(k) * 2 * p.C + c);
    s[ry][cx] = sum;
    __syncthreads();
    // warp ry takes column ry
    sum = warp_sum(s[cx][ry]);
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + ry;
    if (cx == 0 && col < 2 * static_cast<int64_t>(p.C)) {
        float* dst = col < p.C ? p.dw : p.db;
        if (dst) dst[col < p.C ? col : col - p.C] = sum;
    }
}

// ---- any group size and alignment: one CTA per group, scalar loads

__device__ __forceinline__ float block_sum(float v, float* s) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) v += s[i];
    return v;
}

template <typename T, bool kCenter, bool kSilu, bool kGate>
__global__ void __launch_bounds__(kThreads) gn_fwd_any_kernel(const GnParams p) {
    __shared__ float s[kThreads / 32];
    const uint32_t row = blockIdx.x / p.G;
    const int group = static_cast<int>(blockIdx.x - row * p.G), c0 = group * p.D;
    const T* x = at<const T>(p.x, p, row, group);
    const T* z = kGate ? at<const T>(p.z, p, row, group) : nullptr;
    T* out = at<T>(p.out, p, row, group);
    float m = 0.f, q = 0.f;
    if (kCenter) {
        for (int d = threadIdx.x; d < p.D; d += kThreads) m += to_f(x[d]);
        m = block_sum(m, s) / p.D;
    }
    for (int d = threadIdx.x; d < p.D; d += kThreads) {
        const float v = to_f(x[d]) - m;
        q = fmaf(v, v, q);
    }
    const float r = rsqrtf(block_sum(q, s) / p.D + p.eps);
    for (int d = threadIdx.x; d < p.D; d += kThreads) {
        const float y = fmaf((to_f(x[d]) - m) * r, p.w ? p.w[c0 + d] : 1.f, p.b ? p.b[c0 + d] : 0.f);
        out[d] = from_f<T>(kGate ? y * act<kSilu>(to_f(z[d])) : act<kSilu>(y));
    }
}

// one CTA per (share, group): its rows in turn; the columns' sums stay in the share's row of the
// workspace, which only this CTA's thread of that column touches
template <typename T, bool kCenter, bool kSilu, bool kGate>
__global__ void __launch_bounds__(kThreads) gn_bwd_any_kernel(const GnParams p) {
    __shared__ float s[kThreads / 32];
    sm100::grid_dep_launch_dependents();
    const uint32_t share = blockIdx.x / p.G;
    const int group = static_cast<int>(blockIdx.x - share * p.G), c0 = group * p.D;
    const uint32_t r0 = share * p.share_rows;
    const uint32_t r1 = min(r0 + p.share_rows, p.rows);
    float* part = p.shares > 1 ? p.part + static_cast<int64_t>(share) * 2 * p.C : nullptr;
    float *ow = part ? part : p.dw, *ob = part ? part + p.C : p.db;     // a single share is the sum
    if (ow) ow += c0;
    if (ob) ob += c0;
    for (int d = threadIdx.x; d < p.D; d += kThreads) {
        if (ow) ow[d] = 0.f;
        if (ob) ob[d] = 0.f;
    }
    for (uint32_t row = r0; row < r1; ++row) {
        const T* x = at<const T>(p.x, p, row, group);
        const T* dout = at<const T>(p.dout, p, row, group);
        const T* z = kGate ? at<const T>(p.z, p, row, group) : nullptr;
        T* dx = at<T>(p.dx, p, row, group);
        T* dz = kGate ? at<T>(p.dz, p, row, group) : nullptr;
        float m = 0.f, q = 0.f;
        if (kCenter) {
            for (int d = threadIdx.x; d < p.D; d += kThreads) m += to_f(x[d]);
            m = block_sum(m, s) / p.D;
        }
        for (int d = threadIdx.x; d < p.D; d += kThreads) {
            const float v = to_f(x[d]) - m;
            q = fmaf(v, v, q);
        }
        const float r = rsqrtf(block_sum(q, s) / p.D + p.eps);
        float s1 = 0.f, s2 = 0.f;
        for (int pass = 0; pass < 2; ++pass) {
            for (int d = threadIdx.x; d < p.D; d += kThreads) {
                const float xh = (to_f(x[d]) - m) * r, w = p.w ? p.w[c0 + d] : 1.f;
                const float y = fmaf(xh, w, p.b ? p.b[c0 + d] : 0.f), dd = to_f(dout[d]);
                float a, da;
                act_slope<kSilu>(kGate ? to_f(z[d]) : y, &a, &da);
                const float dy = kGate ? dd * a : dd * da, g = dy * w;
                if (pass == 0) {
                    s1 = fmaf(g, xh, s1);
                    s2 += g;
                    if (ow) ow[d] = fmaf(dy, xh, ow[d]);
                    if (ob) ob[d] += dy;
                } else {
                    // this thread alone reads and writes element d from here on: dx may be x or dout
                    dx[d] = from_f<T>(r * (g - xh * s1 - s2));
                    if (kGate) dz[d] = from_f<T>(dd * y * da);
                }
            }
            if (pass == 0) {
                s1 = block_sum(s1, s) / p.D;
                s2 = kCenter ? block_sum(s2, s) / p.D : 0.f;
            }
        }
    }
}

// ---- dispatch

template <bool kC, bool kS, bool kG>
struct Flags {
    static constexpr bool C = kC, S = kS, Z = kG;
};
template <typename F>
auto with_flags(uint32_t flags, bool gate, F&& f) {
    const bool c = flags & M3_GN_CENTER, s = flags & M3_GN_SILU;
    if (c) {
        if (s) return gate ? f(Flags<true, true, true>{}) : f(Flags<true, true, false>{});
        return gate ? f(Flags<true, false, true>{}) : f(Flags<true, false, false>{});
    }
    if (s) return gate ? f(Flags<false, true, true>{}) : f(Flags<false, true, false>{});
    return gate ? f(Flags<false, false, true>{}) : f(Flags<false, false, false>{});
}

template <int L, int V>
struct Shape {
    static constexpr int LPG = L, NV = V;
};
// lanes and vectors per group: the fewest lanes (from 4) that hold it in one vector each, then
// more vectors; the caller has checked that 32 * 4 vectors are enough
template <typename F>
auto with_shape(int vecs, F&& f) {
    if (vecs <= 4) return f(Shape<4, 1>{});
    if (vecs <= 8) return f(Shape<8, 1>{});
    if (vecs <= 16) return f(Shape<16, 1>{});
    if (vecs <= 32) return f(Shape<32, 1>{});
    if (vecs <= 64) return f(Shape<32, 2>{});
    return f(Shape<32, 4>{});
}

bool ok16(const GnTensor& t, int es) {
    return !t.p || ((reinterpret_cast<uintptr_t>(t.p) | static_cast<uintptr_t>(t.batch * es) |
                     static_cast<uintptr_t>(t.row * es) | static_cast<uintptr_t>(t.group * es)) & 15u) == 0;
}

// 16-byte vectors of a group, or 0 where the vector form does not apply
template <typename T>
int vector_count(const GnParams& p) {
    constexpr int N = 2 * Vec<T>::N, es = sizeof(T);
    if (p.D % N != 0 || p.D / N > 128) return 0;
    const bool ok = ok16(p.x, es) && ok16(p.z, es) && ok16(p.out, es) && ok16(p.dout, es) && ok16(p.dx, es) && ok16(p.dz, es);
    return ok ? p.D / N : 0;
}

// Shares of the rows: as many as give every SM `per_sm` CTAs, at most one per (CTA's) row. Where shares are
// added up afterwards, one of up to four rows (a second launch costs more than the rows).
int64_t share_count(int64_t rows, int64_t per_row_ctas, int per_sm, bool added) {
    if (added && rows <= 4) return 1;
    const int64_t want = (per_sm * static_cast<int64_t>(device_sm_count()) + per_row_ctas - 1) / per_row_ctas;
    return rows < want ? (rows > 0 ? rows : 1) : want;
}
// One wave of CTAs: what the registers let an SM hold of this kernel, asked of the runtime once, up to the
// most that pays (16 an SM forward: 46.1 us against 40.1 for 8192 x 4096 bf16 in groups of 64) and, in the
// backward, that the workspace is laid out for. 8192 x 4096, gated / not, where the count was another:
// four where one fits (bf16 forward, groups of 1024) 52.3 / 46.1 us against 43.0 / 37.0, two where one fits
// (bf16 backward, groups of 512) 88.8 / 76.7 against 84.3 / 72.1, one where two fit (fp32 backward, groups of
// 256, gated) 139 against 112. The exception is the gated bf16 backward of groups of 1024, which spills: two
// where one fits 114, one 120.
// Above kBwdPerSm CTAs an SM, shares of the backward keep kShareRows rows or more: shorter ones cost more in
// their sums (two rows each against six: 777 x 1920 fp32 gated 12.3 against 11.9 us, bf16 ungated 12.3
// against 11.1; 4000 x 512 fp32 gated 14.5 against 13.2, bf16 ungated 12.4 against 11.5; 300 x 1920 fp32 8.3 against 8.7).
constexpr int kFwdPerSm = 4, kBwdPerSm = 2, kBwdMostF32 = 4, kBwdMostBf16 = 3, kShareRows = 6;
template <typename T>
constexpr int bwd_most() { return sizeof(T) == 4 ? kBwdMostF32 : kBwdMostBf16; }
template <typename K>
int resident_ctas(K* kernel, size_t smem, int most) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, smem) != cudaSuccess || n < 1) n = 1;
    return n < most ? n : most;
}
// the most shares any form of the backward takes
int64_t max_shares(int64_t rows, bool bf16) { return share_count(rows, 1, bf16 ? kBwdMostBf16 : kBwdMostF32, true); }

constexpr int kMostSums = 32768;        // bytes of a CTA's column sums
// Groups side by side in a CTA: as many as its threads and their column sums' room hold, the row's groups
// spread evenly over the slabs.
int groups_per_cta(const GnParams& p, int per) {
    const int columns = kMostSums / (2 * sizeof(float)), most = per < columns / p.D ? per : columns / p.D;
    const int slabs = (p.G + most - 1) / most;
    return (p.G + slabs - 1) / slabs;
}

// The walk's grid (per_sm CTAs an SM, or down to `least` where shares get short): fills in the shares.
dim3 walk_grid(GnParams& p, int gx, int per, int per_sm, int least, bool added) {
    const int nry = per / gx;
    const unsigned slabs = static_cast<unsigned>((p.G + gx - 1) / gx);
    const int64_t turns = (p.rows + nry - 1) / nry;
    int64_t n = share_count(turns, slabs, per_sm, added);
    if (least < per_sm && n > turns / kShareRows) {
        const int64_t few = share_count(turns, slabs, least, added);
        n = few > turns / kShareRows ? few : turns / kShareRows;
    }
    p.share_rows = static_cast<uint32_t>((turns + n - 1) / n * nry);
    p.shares = static_cast<int>((p.rows + p.share_rows - 1) / p.share_rows);
    return dim3(slabs, static_cast<unsigned>(p.shares));    // up to 2^16 slabs: more than gridDim.y holds
}

template <typename T>
cudaError_t launch_fwd(GnParams p, uint32_t flags, cudaStream_t s) {
    const int vecs = vector_count<T>(p);
    with_flags(flags, p.z.p != nullptr, [&](auto f) {
        using F = decltype(f);
        if (vecs == 0) {
            gn_fwd_any_kernel<T, F::C, F::S, F::Z><<<p.rows * static_cast<unsigned>(p.G), kThreads, 0, s>>>(p);
            return 0;
        }
        return with_shape(vecs, [&](auto sh) {
            using S = decltype(sh);
            constexpr int per = kThreads / S::LPG;
            const int gx = groups_per_cta(p, per);
            auto* const kernel = gn_fwd_kernel<T, S::LPG, S::NV, F::C, F::S, F::Z>;
            static const int per_sm = resident_ctas(kernel, 0, kFwdPerSm);
            const dim3 grid = walk_grid(p, gx, per, per_sm, per_sm, false);
            kernel<<<grid, kThreads, 0, s>>>(p, gx);
            return 0;
        });
    });
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd(GnParams p, uint32_t flags, cudaStream_t s) {
    const int vecs = vector_count<T>(p);
    with_flags(flags, p.z.p != nullptr, [&](auto f) {
        using F = decltype(f);
        if (vecs == 0) {
            const int64_t n = share_count(p.rows, p.G, kBwdPerSm, true);
            p.share_rows = static_cast<uint32_t>((p.rows + n - 1) / n);
            p.shares = static_cast<int>((p.rows + p.share_rows - 1) / p.share_rows);
            gn_bwd_any_kernel<T, F::C, F::S, F::Z><<<static_cast<unsigned>(p.shares * static_cast<int64_t>(p.G)), kThreads, 0, s>>>(p);
            return 0;
        }
        return with_shape(vecs, [&](auto sh) {
            using S = decltype(sh);
            constexpr int per = kThreads / S::LPG;
            const int gx = groups_per_cta(p, per);
            auto* const kernel = gn_bwd_kernel<T, S::LPG, S::NV, F::C, F::S, F::Z>;
            static const int per_sm = resident_ctas(kernel, kMostSums, bwd_most<T>());
            const dim3 grid = walk_grid(p, gx, per, per_sm, kBwdPerSm, true);
            const size_t smem = static_cast<size_t>(gx) * p.D * 2 * sizeof(float);
            kernel<<<grid, kThreads, smem, s>>>(p, gx);
            return 0;
        });
    });
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.shares == 1 || (!p.dw && !p.db)) return e;
    return launch_after_rms(gn_shares_kernel, static_cast<unsigned>((2 * static_cast<int64_t>(p.C) + 31) / 32), 1024, 0, s, p);
}

m3_status err(m3_status st, const char* fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return set_error(st, msg);
}

m3_status check(const m3_group_norm_dims* d) {
    if (!d) return err(M3_ERR_INVALID_ARG, "dims is NULL");
    if (d->in_dtype != M3_F32 && d->in_dtype != M3_BF16)
        return err(M3_ERR_INVALID_ARG, "in_dtype %d is not M3_F32 or M3_BF16", d->in_dtype);
    if (d->batch < 0 || d->rows < 0) return err(M3_ERR_INVALID_ARG, "batch and rows must be >= 0");
    if (d->channels < 1 || d->groups < 1 || d->channels % d->groups != 0)
        return err(M3_ERR_INVALID_ARG, "channels (%lld) must be a positive multiple of groups (%lld)",
                   (long long)d->channels, (long long)d->groups);
    if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return err(M3_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (d->flags & ~(M3_GN_CENTER | M3_GN_SILU))
        return err(M3_ERR_INVALID_ARG, "unknown bits in flags (0x%x)", (unsigned)d->flags);
    // (row, group) pairs are counted in 32 bits
    const int64_t lim = 0x7fffffffLL - kThreads;
    if (d->channels > (int64_t(1) << 24) || (d->batch > 0 && d->rows > lim / d->batch) ||
        (d->batch > 0 && d->rows > 0 && d->groups > lim / (d->batch * d->rows)))
        return err(M3_ERR_UNSUPPORTED, "batch * rows * groups exceeds 2^31");
    return M3_OK;
}

m3_status check_ptr(const void* q, int64_t align, const char* name, bool need) {
    if (!q) return need ? err(M3_ERR_INVALID_ARG, "%s is NULL", name) : M3_OK;
    if (reinterpret_cast<uintptr_t>(q) % static_cast<uintptr_t>(align) != 0)
        return err(M3_ERR_INVALID_ARG, "%s is not aligned to its element size", name);
    return M3_OK;
}

m3_status check_view(const m3_view* v, int es, const char* name, bool need) {
    return check_ptr(v ? v->data : nullptr, es, name, need);
}

GnTensor tensor(const m3_view* v) {
    return v && v->data ? GnTensor{v->data, v->batch, v->token, v->head} : GnTensor{};
}

// Rows (and groups) of an output that share elements through equal strides.
m3_status check_out(const m3_view* v, const m3_group_norm_dims* d, const char* name) {
    const int64_t D = d->channels / d->groups;
    const int64_t g = v->head < 0 ? -v->head : v->head, r = v->token < 0 ? -v->token : v->token;
    if ((d->groups > 1 && g < D) || (d->rows > 1 && r < D) || (d->batch > 1 && v->batch == 0))
        return err(M3_ERR_INVALID_ARG, "%s: rows or groups overlap", name);
    return M3_OK;
}

// An output that begins where another tensor does: allowed for the ones named, by the same strides.
m3_status check_shared(const m3_view* out, const m3_view* t, const m3_group_norm_dims* d, bool allowed,
                       const char* name, const char* other) {
    if (!out || !t || !out->data || out->data != t->data) return M3_OK;
    const bool same = (d->batch == 1 || out->batch == t->batch) && (d->rows == 1 || out->token == t->token) &&
                      (d->groups == 1 || out->head == t->head);
    if (allowed && same) return M3_OK;
    return err(M3_ERR_INVALID_ARG, allowed ? "%s is %s by other strides" : "%s is %s", name, other);
}

// The gradients of weight and bias, and any output, begin at no other tensor's address.
struct Named {
    const void* p;
    const char* name;
};
template <int I>
m3_status check_apart(const Named& out, const Named (&others)[I]) {
    for (const Named& o : others)
        if (out.p && out.p == o.p) return err(M3_ERR_INVALID_ARG, "%s is %s", out.name, o.name);
    return M3_OK;
}

GnParams make_params(const m3_group_norm_dims* d, const m3_view* x, const m3_view* z, const float* w, const float* b) {
    GnParams p{};
    p.rows = static_cast<uint32_t>(d->batch * d->rows);
    p.inner = static_cast<uint32_t>(d->rows);
    p.C = static_cast<int>(d->channels);
    p.G = static_cast<int>(d->groups);
    p.D = p.C / p.G;
    p.eps = d->eps;
    p.x = tensor(x);
    p.z = tensor(z);
    p.w = w;
    p.b = b;
    return p;
}

}  // namespace
}  // namespace m3

using namespace m3;

extern "C" {

m3_status m3_group_norm_fwd(const m3_group_norm_dims* dims, const m3_view* x, const m3_view* z,
                            const float* weight, const float* bias, const m3_view* out, void* stream) {
    set_error(M3_OK, "");
    m3_status st = check(dims);
    if (st != M3_OK) return st;
    const bool bf16 = dims->in_dtype == M3_BF16;
    const int es = bf16 ? 2 : 4;
    const bool any = dims->batch > 0 && dims->rows > 0;
    if ((st = check_view(x, es, "x", any)) != M3_OK || (st = check_view(z, es, "z", false)) != M3_OK ||
        (st = check_ptr(weight, 4, "weight", false)) != M3_OK || (st = check_ptr(bias, 4, "bias", false)) != M3_OK ||
        (st = check_view(out, es, "out", any)) != M3_OK)
        return st;
    if (!any) return M3_OK;
    if ((st = check_out(out, dims, "out")) != M3_OK || (st = check_shared(out, x, dims, true, "out", "x")) != M3_OK ||
        (st = check_shared(out, z, dims, true, "out", "z")) != M3_OK ||
        (st = check_apart({out->data, "out"}, {{weight, "weight"}, {bias, "bias"}})) != M3_OK)
        return st;
    GnParams p = make_params(dims, x, z, weight, bias);
    p.out = tensor(out);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = bf16 ? launch_fwd<__nv_bfloat16>(p, dims->flags, s) : launch_fwd<float>(p, dims->flags, s);
    return e == cudaSuccess ? M3_OK : err(M3_ERR_CUDA, "group norm launch: %s", cudaGetErrorString(e));
}

size_t m3_group_norm_bwd_workspace_bytes(const m3_group_norm_dims* dims) {
    if (check(dims) != M3_OK) return 0;
    const int64_t shares = max_shares(dims->batch * dims->rows, dims->in_dtype == M3_BF16);
    const size_t n = shares > 1 ? static_cast<size_t>(shares) * 2 * static_cast<size_t>(dims->channels) * 4 : 0;
    return (n + 255) / 256 * 256;
}

m3_status m3_group_norm_bwd(const m3_group_norm_dims* dims, const m3_view* x, const m3_view* z, const float* weight,
                            const float* bias, const m3_view* dout, const m3_view* dx, const m3_view* dz,
                            float* dweight, float* dbias, void* workspace, size_t ws_bytes, void* stream) {
    set_error(M3_OK, "");
    m3_status st = check(dims);
    if (st != M3_OK) return st;
    const bool bf16 = dims->in_dtype == M3_BF16;
    const int es = bf16 ? 2 : 4;
    const bool any = dims->batch > 0 && dims->rows > 0, gate = z && z->data;
    if ((st = check_view(x, es, "x", any)) != M3_OK || (st = check_view(z, es, "z", false)) != M3_OK ||
        (st = check_view(dout, es, "dout", any)) != M3_OK || (st = check_view(dx, es, "dx", any)) != M3_OK ||
        (st = check_view(dz, es, "dz", any && gate)) != M3_OK ||
        (st = check_ptr(weight, 4, "weight", false)) != M3_OK || (st = check_ptr(bias, 4, "bias", false)) != M3_OK ||
        (st = check_ptr(dweight, 4, "dweight", false)) != M3_OK || (st = check_ptr(dbias, 4, "dbias", false)) != M3_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!any) {
        cudaError_t e = cudaSuccess;
        if (dweight) e = cudaMemsetAsync(dweight, 0, dims->channels * 4, s);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, dims->channels * 4, s);
        return e == cudaSuccess ? M3_OK : err(M3_ERR_CUDA, "empty gradient: %s", cudaGetErrorString(e));
    }
    if ((st = check_out(dx, dims, "dx")) != M3_OK || (gate && (st = check_out(dz, dims, "dz")) != M3_OK)) return st;
    if ((st = check_shared(dx, x, dims, true, "dx", "x")) != M3_OK ||
        (st = check_shared(dx, dout, dims, true, "dx", "dout")) != M3_OK ||
        (st = check_shared(dx, z, dims, false, "dx", "z")) != M3_OK)
        return st;
    if (gate && ((st = check_shared(dz, z, dims, true, "dz", "z")) != M3_OK ||
                 (st = check_shared(dz, x, dims, false, "dz", "x")) != M3_OK ||
                 (st = check_shared(dz, dout, dims, false, "dz", "dout")) != M3_OK ||
                 (st = check_shared(dz, dx, dims, false, "dz", "dx")) != M3_OK))
        return st;
    const void *pz = gate ? z->data : nullptr, *pdz = gate ? dz->data : nullptr;
    const Named params[] = {{weight, "weight"}, {bias, "bias"}};
    const Named all[] = {{x->data, "x"}, {pz, "z"}, {dout->data, "dout"}, {weight, "weight"}, {bias, "bias"},
                         {dx->data, "dx"}, {pdz, "dz"}};
    if ((st = check_apart({dx->data, "dx"}, params)) != M3_OK || (st = check_apart({pdz, "dz"}, params)) != M3_OK ||
        (st = check_apart({dweight, "dweight"}, all)) != M3_OK || (st = check_apart({dbias, "dbias"}, all)) != M3_OK ||
        (st = check_apart({dbias, "dbias"}, {{dweight, "dweight"}})) != M3_OK)
        return st;
    const size_t need = m3_group_norm_bwd_workspace_bytes(dims);
    if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || ws_bytes < need))
        return err(M3_ERR_INVALID_ARG, "workspace: NULL, misaligned or below %zu bytes", need);
    GnParams p = make_params(dims, x, z, weight, bias);
    p.dout = tensor(dout);
    p.dx = tensor(dx);
    p.dz = gate ? tensor(dz) : GnTensor{};
    p.dw = dweight;
    p.db = dbias;
    p.part = static_cast<float*>(workspace);
    const cudaError_t e = bf16 ? launch_bwd<__nv_bfloat16>(p, dims->flags, s) : launch_bwd<float>(p, dims->flags, s);
    return e == cudaSuccess ? M3_OK : err(M3_ERR_CUDA, "group norm backward launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
