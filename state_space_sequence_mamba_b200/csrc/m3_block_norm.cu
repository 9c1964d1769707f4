// The norms before and after a block with its gate and residual, and their gradients:
//     n = post(y),  h = x + alpha n act(z),  out = pre(h)
//
// Bound by HBM: the forward reads y, x, z and writes h, out, the backward reads those inputs, dh and dout
// and writes dy, dx, dz, each once. A row lies in the registers of a team of W warps (NV 16-byte vectors
// a lane), so h goes from its residual into the second norm's statistics without a trip through memory, and the
// deviations are squared from registers. Teams walk over rows, the next row's loads in flight. Rows too
// wide, or not 16-byte aligned, take one CTA each with scalar loads.
//
// Backward, with yh = (y - mean) ry, hh = (h - mean) rh, n = yh w1 + b1 and go = dout w2:
//     d  = dh + rh (go - hh mean(go hh) - mean(go) [layer]),     dx = d
//     dz = alpha d n act'(z),  e = alpha d act(z),  g = e w1
//     dy = ry (g - yh mean(g yh) - mean(g) [layer])
//     dw2 = sum dout hh,  db2 = sum dout,  dw1 = sum e yh,  db1 = sum e
// A team's column sums lie in its shared memory, each thread's in its own places; a CTA's are written to the
// workspace and a second launch adds them in a fixed order.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "m3_common.cuh"
#include "m3_internal.h"
#include "m3_linattn.h"
#include "m3_sm100.cuh"
#include "m3_vec.cuh"

namespace m3 {
namespace {

struct BnTensor {
    void* p;
    int64_t batch, row;         // strides in elements
};
enum Norm { kNone = 0, kRms = 1, kLayer = 2 };
enum Act { kIdentity = 0, kSigmoid = 1, kSilu = 2 };
struct BnParams {
    uint32_t rows, inner;       // rows in all, and of each batch entry
    int C, post, pre, act;
    BnTensor y, x, z, h, out, dh, dout, dy, dx, dz;
    const float *w1, *b1, *w2, *b2;
    int sums;                   // backward: which of dw1, db1, dw2, db2 are wanted (bits), and how many
    int nsums;
    float* part;                // [CTAs][nsums][C]
    float alpha, eps;
};

template <typename T>
__device__ __forceinline__ T* at(const BnTensor& t, const BnParams& p, uint32_t row) {
    const uint32_t b = p.inner == p.rows ? 0u : row / p.inner;
    return static_cast<T*>(t.p) + b * t.batch + static_cast<int64_t>(row - b * p.inner) * t.row;
}

// N elements of TR where a 16-byte vector of the block's type has N: as bits, and as pairs of floats
template <typename TR, int N>
struct Part {
    static constexpr int Q = N * static_cast<int>(sizeof(TR)) / 16;     // 16-byte words
    uint4 w[Q];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < Q; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void load(const TR* p) {
#pragma unroll
        for (int i = 0; i < Q; ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void unpack(float2 (&f)[N / 2]) const {
#pragma unroll
        for (int i = 0; i < Q; ++i) Vec<TR>::unpack(w[i], f + i * Vec<TR>::N);
    }
    static __device__ __forceinline__ void store(TR* p, const float2 (&f)[N / 2]) {
#pragma unroll
        for (int i = 0; i < Q; ++i) Vec<TR>::store(p + i * 2 * Vec<TR>::N, f + i * Vec<TR>::N);
    }
};

__device__ __forceinline__ float2 act2(int act, const float2& z) {
    if (act == kIdentity) return z;
    const float2 s = sigmoid2(z);
    return act == kSigmoid ? s : mul2(z, s);
}
__device__ __forceinline__ void act_slope2(int act, const float2& z, float2* a, float2* da) {
    if (act == kIdentity) {
        *a = z;
        *da = both(1.f);
        return;
    }
    const float2 s = sigmoid2(z), t = fma2(s, both(-1.f), both(1.f));
    if (act == kSigmoid) {
        *a = s;
        *da = mul2(s, t);
    } else {
        *a = mul2(z, s);
        *da = fma2(*a, t, s);       // s (1 + z (1 - s))
    }
}

// A team: W warps that hold one row. Its sums go through shared memory, in turn through one of two places, so
// that one barrier a sum is enough.
template <int W, int kTeams>
struct Team {
    float2 (*s)[kTeams][W];
    int team, warp, lane, turn = 0;
    __device__ __forceinline__ explicit Team(float2 (*places)[kTeams][W]) : s(places) {
        team = threadIdx.x / (32 * W);
        warp = (threadIdx.x / 32) % W;
        lane = threadIdx.x & 31;
    }
    __device__ __forceinline__ float2 sum(float2 v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float2 u = make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o));
            v = add2(v, u);
        }
        if (W == 1) return v;
        if (lane == 0) s[turn][team][warp] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(32 * W) : "memory");
        v = s[turn][team][0];
#pragma unroll
        for (int w = 1; w < W; ++w) v = add2(v, s[turn][team][w]);
        turn ^= 1;
        return v;
    }
    __device__ __forceinline__ float sum(float v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (W == 1) return v;
        if (lane == 0) s[turn][team][warp].x = v;
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(32 * W) : "memory");
        v = s[turn][team][0].x;
#pragma unroll
        for (int w = 1; w < W; ++w) v += s[turn][team][w].x;
        turn ^= 1;
        return v;
    }
};

// v becomes its deviations over the root of its variance (or v over its root mean square); returns the factor.
// Elements beyond the row hold zeros and keep them.
template <int NV, int H, typename T>
__device__ __forceinline__ float normalise(T& team, float2 (&v)[NV][H], const bool (&in)[NV], int kind, float inv, float eps) {
    if (kind == kNone) return 1.f;
    if (kind == kLayer) {
        float2 s = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < H; ++e) s = add2(s, v[i][e]);
        const float m = team.sum(s.x + s.y) * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float2 mi = both(in[i] ? -m : 0.f);
#pragma unroll
            for (int e = 0; e < H; ++e) v[i][e] = add2(v[i][e], mi);
        }
    }
    float2 q = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < H; ++e) q = fma2(v[i][e], v[i][e], q);
    const float r = rsqrtf(fmaf(team.sum(q.x + q.y), inv, eps));
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < H; ++e) v[i][e] = in[i] ? mul2(v[i][e], both(r)) : both(0.f);
    return r;
}

// a channel's parameters, or `other` without any
template <int H>
__device__ __forceinline__ void params(const float* w, int c, bool in, float other, float2 (&f)[H]) {
#pragma unroll
    for (int e = 0; e < H; ++e) f[e] = w && in ? make_float2(__ldg(w + c + 2 * e), __ldg(w + c + 2 * e + 1)) : both(other);
}

template <int W>
constexpr int block_threads() { return 32 * (W > 8 ? W : 8); }

template <typename T, typename TR, int W, int NV>
__global__ void __launch_bounds__(block_threads<W>()) bn_fwd_kernel(const __grid_constant__ BnParams p) {
    constexpr int N = 16 / sizeof(T), H = N / 2, kTeams = block_threads<W>() / (32 * W);
    __shared__ float2 s_sum[2][kTeams][W];
    Team<W, kTeams> team(s_sum);
    const int t = threadIdx.x % (32 * W);
    int c[NV];
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        c[i] = (i * 32 * W + t) * N;
        in[i] = c[i] < p.C;
    }
    const float inv = 1.f / p.C;
    Part<T, N> ry[NV], rz[NV];
    Part<TR, N> rx[NV];
    const auto fetch = [&](uint32_t row) {
        const bool live = row < p.rows;
        const T* y = live ? at<const T>(p.y, p, row) : nullptr;
        const T* z = live && p.z.p ? at<const T>(p.z, p, row) : nullptr;
        const TR* x = live ? at<const TR>(p.x, p, row) : nullptr;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            ry[i].zero();
            rx[i].zero();
            rz[i].zero();
            if (!live || !in[i]) continue;
            ry[i].load(y + c[i]);
            rx[i].load(x + c[i]);
            if (z) rz[i].load(z + c[i]);
        }
    };
    const uint32_t step = gridDim.x * kTeams;
    uint32_t row = blockIdx.x * kTeams + team.team;
    fetch(row);
    for (; row < p.rows; row += step) {
        float2 v[NV][H], x[NV][H], z[NV][H];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            ry[i].unpack(v[i]);
            rx[i].unpack(x[i]);
            rz[i].unpack(z[i]);
        }
        fetch(row + step);
        normalise(team, v, in, p.post, inv, p.eps);
        TR* h = at<TR>(p.h, p, row);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float2 w[H], b[H];
            params(p.w1, c[i], in[i], 1.f, w);
            params(p.b1, c[i], in[i], 0.f, b);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                float2 n = mul2(fma2(v[i][e], w[e], b[e]), both(p.alpha));
                if (p.z.p) n = mul2(n, act2(p.act, z[i][e]));
                v[i][e] = add2(x[i][e], n);
            }
            if (in[i]) Part<TR, N>::store(h + c[i], v[i]);
        }
        if (p.pre == kNone) continue;
        normalise(team, v, in, p.pre, inv, p.eps);
        T* out = at<T>(p.out, p, row);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float2 w[H], b[H];
            params(p.w2, c[i], in[i], 1.f, w);
            params(p.b2, c[i], in[i], 0.f, b);
#pragma unroll
            for (int e = 0; e < H; ++e) v[i][e] = fma2(v[i][e], w[e], b[e]);
            if (in[i]) Part<T, N>::store(out + c[i], v[i]);
        }
    }
}

// A thread's columns in a team's sums: vector i, quarter q (two pairs) of thread t of the team lie side by side
// with the other threads'.
template <int W, int NV, int Q>
__device__ __forceinline__ float4* place(float* s, int sum, int i, int q, int t) {
    return reinterpret_cast<float4*>(s) + ((sum * NV + i) * Q + q) * (32 * W) + t;
}

template <typename T, typename TR, int W, int NV>
__global__ void __launch_bounds__(block_threads<W>()) bn_bwd_kernel(const __grid_constant__ BnParams p) {
    constexpr int N = 16 / sizeof(T), H = N / 2, Q = N / 4, kTeams = block_threads<W>() / (32 * W);
    __shared__ float2 s_sum[2][kTeams][W];
    extern __shared__ float4 s_cols[];      // [teams][nsums][NV][Q][32 W]
    sm100::grid_dep_launch_dependents();
    Team<W, kTeams> team(s_sum);
    const int t = threadIdx.x % (32 * W);
    float* cols = reinterpret_cast<float*>(s_cols) + static_cast<size_t>(team.team) * p.nsums * NV * N * 32 * W;
    for (int i = 0; i < p.nsums * NV * Q; ++i) reinterpret_cast<float4*>(cols)[i * 32 * W + t] = make_float4(0.f, 0.f, 0.f, 0.f);
    int c[NV];
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        c[i] = (i * 32 * W + t) * N;
        in[i] = c[i] < p.C;
    }
    // which of the wanted sums is which
    const int i0 = 0, i1 = i0 + (p.sums & 1), i2 = i1 + (p.sums >> 1 & 1), i3 = i2 + (p.sums >> 2 & 1);
    const auto add = [&](int sum, int i, const float2 (&v)[H]) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            float4* a = place<W, NV, Q>(cols, sum, i, q, t);
            float4 o = *a;
            const float2 lo = add2(make_float2(o.x, o.y), v[2 * q]), hi = add2(make_float2(o.z, o.w), v[2 * q + 1]);
            *a = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
    };
    const float inv = 1.f / p.C;
    Part<T, N> ry[NV], rz[NV], ro[NV];
    Part<TR, N> rx[NV], rd[NV];
    const auto fetch = [&](uint32_t row) {
        const bool live = row < p.rows;
        const T* y = live ? at<const T>(p.y, p, row) : nullptr;
        const T* z = live && p.z.p ? at<const T>(p.z, p, row) : nullptr;
        const T* o = live && p.pre != kNone ? at<const T>(p.dout, p, row) : nullptr;
        const TR* x = live ? at<const TR>(p.x, p, row) : nullptr;
        const TR* d = live && p.dh.p ? at<const TR>(p.dh, p, row) : nullptr;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            ry[i].zero();
            rx[i].zero();
            rz[i].zero();
            ro[i].zero();
            rd[i].zero();
            if (!live || !in[i]) continue;
            ry[i].load(y + c[i]);
            rx[i].load(x + c[i]);
            if (z) rz[i].load(z + c[i]);
            if (o) ro[i].load(o + c[i]);
            if (d) rd[i].load(d + c[i]);
        }
    };
    const uint32_t step = gridDim.x * kTeams;
    for (uint32_t row = blockIdx.x * kTeams + team.team; row < p.rows; row += step) {
        fetch(row);
        float2 v[NV][H], d[NV][H];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            ry[i].unpack(v[i]);
            rd[i].unpack(d[i]);
        }
        const float r1 = normalise(team, v, in, p.post, inv, p.eps);
        if (p.pre != kNone) {
            float2 h[NV][H];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 w[H], b[H], x[H], z[H];
                params(p.w1, c[i], in[i], 1.f, w);
                params(p.b1, c[i], in[i], 0.f, b);
                rx[i].unpack(x);
                rz[i].unpack(z);
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    float2 n = mul2(fma2(v[i][e], w[e], b[e]), both(p.alpha));
                    if (p.z.p) n = mul2(n, act2(p.act, z[e]));
                    h[i][e] = add2(x[e], n);
                }
            }
            const float r2 = normalise(team, h, in, p.pre, inv, p.eps);
            float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 w[H], o[H], u[H];
                params(p.w2, c[i], in[i], 1.f, w);
                ro[i].unpack(o);
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    u[e] = mul2(o[e], h[i][e]);
                    s1 = fma2(u[e], w[e], s1);
                    s2 = fma2(o[e], w[e], s2);
                }
                if (in[i] && (p.sums & 4)) add(i2, i, u);
                if (in[i] && (p.sums & 8)) add(i3, i, o);
            }
            const float2 s = team.sum(make_float2(s1.x + s1.y, s2.x + s2.y));
            const float m1 = -s.x * inv, m2 = p.pre == kLayer ? -s.y * inv : 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 w[H], o[H];
                params(p.w2, c[i], in[i], 1.f, w);
                ro[i].unpack(o);
#pragma unroll
                for (int e = 0; e < H; ++e)
                    d[i][e] = fma2(fma2(o[e], w[e], fma2(h[i][e], both(m1), both(m2))), both(r2), d[i][e]);
            }
        }
        TR* dx = at<TR>(p.dx, p, row);
        T* dz = p.z.p ? at<T>(p.dz, p, row) : nullptr;
        float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (in[i]) Part<TR, N>::store(dx + c[i], d[i]);
            float2 w[H], b[H], z[H], u[H];
            params(p.w1, c[i], in[i], 1.f, w);
            params(p.b1, c[i], in[i], 0.f, b);
            rz[i].unpack(z);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                d[i][e] = mul2(d[i][e], both(p.alpha));
                if (p.z.p) {
                    float2 a, da;
                    act_slope2(p.act, z[e], &a, &da);
                    z[e] = mul2(mul2(d[i][e], fma2(v[i][e], w[e], b[e])), da);
                    d[i][e] = mul2(d[i][e], a);
                }
                u[e] = mul2(d[i][e], v[i][e]);
            }
            if (in[i] && dz) Part<T, N>::store(dz + c[i], z);
            if (in[i] && (p.sums & 1)) add(i0, i, u);
            if (in[i] && (p.sums & 2)) add(i1, i, d[i]);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                if (!in[i]) continue;       // (m2 reaches what lies beyond the row)
                s1 = fma2(u[e], w[e], s1);
                d[i][e] = mul2(d[i][e], w[e]);
                s2 = add2(s2, d[i][e]);
            }
        }
        float m1 = 0.f, m2 = 0.f;
        if (p.post != kNone) {
            const float2 s = team.sum(make_float2(s1.x + s1.y, s2.x + s2.y));
            m1 = -s.x * inv;
            m2 = p.post == kLayer ? -s.y * inv : 0.f;
        }
        T* dy = at<T>(p.dy, p, row);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!in[i]) continue;
#pragma unroll
            for (int e = 0; e < H; ++e) d[i][e] = mul2(add2(d[i][e], fma2(v[i][e], both(m1), both(m2))), both(r1));
            Part<T, N>::store(dy + c[i], d[i]);
        }
    }
    if (p.nsums == 0) return;
    __syncthreads();
    // the teams' sums, added in order, to the CTA's share
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.nsums * p.C;
    constexpr int kCols = NV * N * 32 * W;
    for (int sum = 0; sum < p.nsums; ++sum)
        for (int k = threadIdx.x; k < kCols / 4; k += block_threads<W>()) {
            const int tt = k % (32 * W), iq = k / (32 * W), q = iq % Q, i = iq / Q;
            const int col = (i * 32 * W + tt) * N + 4 * q;
            if (col >= p.C) continue;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int u = 0; u < kTeams; ++u) {
                const float4 o = *place<W, NV, Q>(reinterpret_cast<float*>(s_cols) + static_cast<size_t>(u) * p.nsums * kCols, sum, i, q, tt);
                a = make_float4(a.x + o.x, a.y + o.y, a.z + o.z, a.w + o.w);
            }
            *reinterpret_cast<float4*>(part + static_cast<int64_t>(sum) * p.C + col) = a;
        }
}

// ---- any width and alignment: one CTA a row, scalar loads, each pass over the row from memory

constexpr int kAny = 256;

__device__ __forceinline__ float block_sum(float v, float* s) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < kAny / 32; ++i) v += s[i];
    return v;
}

__device__ __forceinline__ float act1(int act, float z) {
    const float2 r = act2(act, both(z));
    return r.x;
}

template <typename T, typename TR>
struct AnyRow {
    const BnParams& p;
    const T *y, *z;
    const TR* x;
    float m1 = 0.f, r1 = 1.f, m2 = 0.f, r2 = 1.f;
    __device__ __forceinline__ AnyRow(const BnParams& q, uint32_t row) : p(q) {
        y = at<const T>(p.y, p, row);
        z = p.z.p ? at<const T>(p.z, p, row) : nullptr;
        x = at<const TR>(p.x, p, row);
    }
    __device__ __forceinline__ float yh(int c) const { return (to_f(y[c]) - m1) * r1; }
    __device__ __forceinline__ float n(int c) const { return fmaf(yh(c), p.w1 ? p.w1[c] : 1.f, p.b1 ? p.b1[c] : 0.f); }
    __device__ __forceinline__ float h(int c) const {
        const float v = n(c) * p.alpha;
        return to_f(x[c]) + (z ? v * act1(p.act, to_f(z[c])) : v);
    }
    template <typename F>
    __device__ __forceinline__ void stats(int kind, F&& v, float* m, float* r, float* s) {
        if (kind == kNone) return;
        float mean = 0.f, q = 0.f;
        if (kind == kLayer) {
            for (int c = threadIdx.x; c < p.C; c += kAny) mean += v(c);
            mean = block_sum(mean, s) / p.C;
        }
        for (int c = threadIdx.x; c < p.C; c += kAny) {
            const float d = v(c) - mean;
            q = fmaf(d, d, q);
        }
        *r = rsqrtf(block_sum(q, s) / p.C + p.eps);
        *m = mean;
    }
    __device__ __forceinline__ void all(float* s) {
        stats(p.post, [&](int c) { return to_f(y[c]); }, &m1, &r1, s);
        stats(p.pre, [&](int c) { return h(c); }, &m2, &r2, s);
    }
};

template <typename T, typename TR>
__global__ void __launch_bounds__(kAny) bn_fwd_any_kernel(const __grid_constant__ BnParams p) {
    __shared__ float s[kAny / 32];
    for (uint32_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        AnyRow<T, TR> a(p, row);
        a.all(s);
        TR* h = at<TR>(p.h, p, row);
        T* out = p.pre != kNone ? at<T>(p.out, p, row) : nullptr;
        // this thread alone reads and writes element c from here on: h may be x, out may be y
        for (int c = threadIdx.x; c < p.C; c += kAny) {
            const float v = a.h(c);
            h[c] = from_f<TR>(v);
            if (out) out[c] = from_f<T>(fmaf((v - a.m2) * a.r2, p.w2 ? p.w2[c] : 1.f, p.b2 ? p.b2[c] : 0.f));
        }
        __syncthreads();
    }
}

template <typename T, typename TR>
__global__ void __launch_bounds__(kAny) bn_bwd_any_kernel(const __grid_constant__ BnParams p) {
    __shared__ float s[kAny / 32];
    sm100::grid_dep_launch_dependents();
    float* part[4] = {};
    int n = 0;
    for (int k = 0; k < 4; ++k)
        if (p.sums >> k & 1) part[k] = p.part + (static_cast<int64_t>(blockIdx.x) * p.nsums + n++) * p.C;
    for (int k = 0; k < 4; ++k)
        if (part[k])
            for (int c = threadIdx.x; c < p.C; c += kAny) part[k][c] = 0.f;
    for (uint32_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        AnyRow<T, TR> a(p, row);
        a.all(s);
        const TR* dh = p.dh.p ? at<const TR>(p.dh, p, row) : nullptr;
        const T* dout = p.pre != kNone ? at<const T>(p.dout, p, row) : nullptr;
        T *dy = at<T>(p.dy, p, row), *dz = a.z ? at<T>(p.dz, p, row) : nullptr;
        TR* dx = at<TR>(p.dx, p, row);
        float u1 = 0.f, u2 = 0.f, v1 = 0.f, v2 = 0.f;
        const auto go = [&](int c) { return to_f(dout[c]) * (p.w2 ? p.w2[c] : 1.f); };
        if (dout) {
            for (int c = threadIdx.x; c < p.C; c += kAny) {
                const float g = go(c);
                u1 = fmaf(g, (a.h(c) - a.m2) * a.r2, u1);
                u2 += g;
            }
            u1 = block_sum(u1, s) / p.C;
            u2 = p.pre == kLayer ? block_sum(u2, s) / p.C : 0.f;
        }
        // d, the gradient of h
        const auto back = [&](int c, float hh) {
            const float d = dh ? to_f(dh[c]) : 0.f;
            return dout ? fmaf(a.r2, go(c) - hh * u1 - u2, d) : d;
        };
        for (int pass = p.post == kNone ? 1 : 0; pass < 2; ++pass) {
            for (int c = threadIdx.x; c < p.C; c += kAny) {
                const float hh = (a.h(c) - a.m2) * a.r2, yh = a.yh(c), d = back(c, hh);
                float e = d * p.alpha, slope = 0.f;
                const float dn = e;
                if (a.z) {
                    float2 f, g;
                    act_slope2(p.act, both(to_f(a.z[c])), &f, &g);
                    e *= f.x;
                    slope = g.x;
                }
                const float g = e * (p.w1 ? p.w1[c] : 1.f);
                if (pass == 0) {
                    v1 = fmaf(g, yh, v1);
                    v2 += g;
                    continue;
                }
                if (part[0]) part[0][c] = fmaf(e, yh, part[0][c]);
                if (part[1]) part[1][c] += e;
                if (part[2]) part[2][c] = fmaf(to_f(dout[c]), hh, part[2][c]);
                if (part[3]) part[3][c] += to_f(dout[c]);
                // this thread alone reads and writes element c from here on
                const float nz = a.n(c) * dn * slope;
                dx[c] = from_f<TR>(d);
                if (dz) dz[c] = from_f<T>(nz);
                dy[c] = from_f<T>(a.r1 * (g - yh * v1 - v2));
            }
            if (pass == 0) {
                v1 = block_sum(v1, s) / p.C;
                v2 = p.post == kLayer ? block_sum(v2, s) / p.C : 0.f;
            }
        }
        __syncthreads();
    }
}

// ---- dispatch

template <int w, int v>
struct Shape {
    static constexpr int W = w, NV = v;
};
// Warps and vectors a lane for a row of `vecs` vectors: two vectors a lane from 32 lanes on.
template <typename F>
auto with_shape(int vecs, F&& f) {
    if (vecs <= 32) return f(Shape<1, 1>{});
    if (vecs <= 64) return f(Shape<1, 2>{});
    if (vecs <= 128) return f(Shape<2, 2>{});
    if (vecs <= 256) return f(Shape<4, 2>{});
    if (vecs <= 512) return f(Shape<8, 2>{});
    return f(Shape<16, 2>{});
}
constexpr int kMostVecs = 1024;

bool ok16(const BnTensor& t, int es) {
    return !t.p || ((reinterpret_cast<uintptr_t>(t.p) | static_cast<uintptr_t>(t.batch * es) |
                     static_cast<uintptr_t>(t.row * es)) & 15u) == 0;
}

// 16-byte vectors of a row, or 0 where the vector form does not apply
template <typename T, typename TR>
int vector_count(const BnParams& p) {
    constexpr int N = 16 / sizeof(T);
    if (p.C % N != 0 || p.C / N > kMostVecs) return 0;
    for (const BnTensor* t : {&p.y, &p.z, &p.out, &p.dout, &p.dy, &p.dz})
        if (!ok16(*t, sizeof(T))) return 0;
    for (const BnTensor* t : {&p.x, &p.h, &p.dh, &p.dx})
        if (!ok16(*t, sizeof(TR))) return 0;
    return p.C / N;
}

template <typename K>
int resident(K* kernel, int threads, size_t smem) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n < 1) n = 1;
    return n;
}

// CTAs of the backward: bounded by the workspace's shares
constexpr int kMostPerSm = 4;
int64_t most_shares(int64_t rows) {
    const int64_t most = static_cast<int64_t>(device_sm_count()) * kMostPerSm;
    return rows < most ? (rows > 0 ? rows : 1) : most;
}

template <typename T, typename TR>
cudaError_t launch_fwd(const BnParams& p, cudaStream_t s) {
    const int vecs = vector_count<T, TR>(p);
    const int64_t sms = device_sm_count();
    if (vecs == 0) {
        const int64_t grid = p.rows < 16 * sms ? p.rows : 16 * sms;
        bn_fwd_any_kernel<T, TR><<<static_cast<unsigned>(grid), kAny, 0, s>>>(p);
        return cudaGetLastError();
    }
    with_shape(vecs, [&](auto sh) {
        using S = decltype(sh);
        constexpr int threads = block_threads<S::W>(), teams = threads / (32 * S::W);
        auto* const kernel = bn_fwd_kernel<T, TR, S::W, S::NV>;
        static const int per_sm = resident(kernel, threads, 0);
        const int64_t want = (p.rows + teams - 1) / teams, most = per_sm * sms;
        kernel<<<static_cast<unsigned>(want < most ? want : most), threads, 0, s>>>(p);
        return 0;
    });
    return cudaGetLastError();
}

template <typename T, typename TR>
cudaError_t launch_bwd(BnParams p, float* const (&outs)[4], cudaStream_t s) {
    const int vecs = vector_count<T, TR>(p);
    int shares = 1;
    float* wanted[4] = {};
    for (int k = 0, n = 0; k < 4; ++k)
        if (p.sums >> k & 1) wanted[n++] = outs[k];
    cudaError_t e = cudaSuccess;
    if (vecs > 0) with_shape(vecs, [&](auto sh) {
        using S = decltype(sh);
        constexpr int threads = block_threads<S::W>(), teams = threads / (32 * S::W);
        constexpr int one = teams * S::NV * (16 / static_cast<int>(sizeof(T))) * 32 * S::W * 4;     // bytes of one sum: up to 32 KB
        static_assert(one <= 32768, "a CTA's sums fit");
        auto* const kernel = bn_bwd_kernel<T, TR, S::W, S::NV>;
        static std::atomic<uint64_t> done{0};
        if ((e = allow_smem(kernel, 4 * one, done)) != cudaSuccess) return 0;
        static const int per_sm[5] = {resident(kernel, threads, 0), resident(kernel, threads, one), resident(kernel, threads, 2 * one),
                                      resident(kernel, threads, 3 * one), resident(kernel, threads, 4 * one)};
        const int64_t want = (p.rows + teams - 1) / teams;
        int64_t most = static_cast<int64_t>(device_sm_count()) * (per_sm[p.nsums] < kMostPerSm ? per_sm[p.nsums] : kMostPerSm);
        shares = static_cast<int>(want < most ? want : most);
        kernel<<<static_cast<unsigned>(shares), threads, p.nsums * one, s>>>(p);
        return 0;
    });
    if (e != cudaSuccess) return e;
    if (vecs == 0) {
        shares = static_cast<int>(most_shares(p.rows));
        bn_bwd_any_kernel<T, TR><<<static_cast<unsigned>(shares), kAny, 0, s>>>(p);
    }
    e = cudaGetLastError();
    if (e != cudaSuccess || p.nsums == 0) return e;
    return launch_sum_shares(p.part, shares, p.C, wanted, p.nsums, s);
}

m3_status err(m3_status st, const char* fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return set_error(st, msg);
}

bool both_of(uint32_t f, uint32_t pair) { return (f & pair) == pair; }

m3_status check(const m3_block_norm_dims* d) {
    if (!d) return err(M3_ERR_INVALID_ARG, "dims is NULL");
    if (d->in_dtype != M3_F32 && d->in_dtype != M3_BF16)
        return err(M3_ERR_INVALID_ARG, "in_dtype %d is not M3_F32 or M3_BF16", d->in_dtype);
    if (d->res_dtype != M3_F32 && d->res_dtype != d->in_dtype)
        return err(M3_ERR_INVALID_ARG, "res_dtype %d is not M3_F32 or in_dtype", d->res_dtype);
    if (d->batch < 0 || d->rows < 0) return err(M3_ERR_INVALID_ARG, "batch and rows must be >= 0");
    if (d->channels < 1) return err(M3_ERR_INVALID_ARG, "channels must be >= 1");
    if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return err(M3_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!std::isfinite(d->alpha)) return err(M3_ERR_INVALID_ARG, "alpha must be finite");
    constexpr uint32_t post = M3_BN_POST_RMS | M3_BN_POST_LAYER, pre = M3_BN_PRE_RMS | M3_BN_PRE_LAYER,
                       act = M3_BN_SIGMOID | M3_BN_SILU;
    if (d->flags & ~(post | pre | act)) return err(M3_ERR_INVALID_ARG, "unknown bits in flags (0x%x)", (unsigned)d->flags);
    if (both_of(d->flags, post) || both_of(d->flags, pre) || both_of(d->flags, act))
        return err(M3_ERR_INVALID_ARG, "flags (0x%x) name both of a pair", (unsigned)d->flags);
    if (d->channels > (int64_t(1) << 24) || (d->batch > 0 && d->rows > 0x7fffffffLL / d->batch))
        return err(M3_ERR_UNSUPPORTED, "more than 2^31 rows or 2^24 channels");
    return M3_OK;
}

m3_status check_ptr(const void* q, uintptr_t align, const char* name, bool need) {
    if (!q) return need ? err(M3_ERR_INVALID_ARG, "%s is NULL", name) : M3_OK;
    if (reinterpret_cast<uintptr_t>(q) % align) return err(M3_ERR_INVALID_ARG, "%s is not element-aligned", name);
    return M3_OK;
}
const void* data(const m3_view* v) { return v ? v->data : nullptr; }

// A dimension of one entry has stride 0, whatever the caller's says.
BnTensor tensor(const m3_block_norm_dims* d, const m3_view* v) {
    if (!v || !v->data) return BnTensor{};
    return BnTensor{v->data, d->batch > 1 ? v->batch : 0, d->rows > 1 ? v->token : 0};
}

// Rows of an output that share elements through equal strides.
m3_status check_out(const BnTensor& t, const m3_block_norm_dims* d, const char* name) {
    const int64_t r = t.row < 0 ? -t.row : t.row, b = t.batch < 0 ? -t.batch : t.batch;
    if ((d->rows > 1 && r < d->channels) || (d->batch > 1 && b < d->channels))
        return err(M3_ERR_INVALID_ARG, "%s: rows overlap", name);
    return M3_OK;
}

struct Named {
    const BnTensor* t;
    const void* p;
    const char* name;
};
// An output begins at no other tensor's address, but for `same`, which it may lie on by the same strides.
template <int I>
m3_status check_apart(const Named& out, const void* same, const Named (&others)[I]) {
    for (const Named& o : others) {
        if (!out.p || out.p != o.p) continue;
        if (o.p != same || !o.t || !out.t) return err(M3_ERR_INVALID_ARG, "%s is %s", out.name, o.name);
        if (o.t->batch != out.t->batch || o.t->row != out.t->row)
            return err(M3_ERR_INVALID_ARG, "%s is %s by other strides", out.name, o.name);
    }
    return M3_OK;
}

m3_status check_inputs(const m3_block_norm_dims* d, const m3_block_norm_inputs* in, bool any) {
    if (!in) return err(M3_ERR_INVALID_ARG, "inputs is NULL");
    const uintptr_t es = d->in_dtype == M3_BF16 ? 2 : 4, er = d->res_dtype == M3_BF16 ? 2 : 4;
    m3_status st;
    if ((st = check_ptr(in->y.data, es, "y", any)) != M3_OK || (st = check_ptr(in->residual.data, er, "residual", any)) != M3_OK ||
        (st = check_ptr(in->z.data, es, "z", false)) != M3_OK ||
        (st = check_ptr(in->post_weight, 4, "post_weight", false)) != M3_OK ||
        (st = check_ptr(in->post_bias, 4, "post_bias", false)) != M3_OK ||
        (st = check_ptr(in->pre_weight, 4, "pre_weight", false)) != M3_OK ||
        (st = check_ptr(in->pre_bias, 4, "pre_bias", false)) != M3_OK)
        return st;
    if (!(d->flags & (M3_BN_PRE_RMS | M3_BN_PRE_LAYER)) && (in->pre_weight || in->pre_bias))
        return err(M3_ERR_INVALID_ARG, "pre_weight or pre_bias without a pre norm");
    if (!in->z.data && (d->flags & (M3_BN_SIGMOID | M3_BN_SILU))) return err(M3_ERR_INVALID_ARG, "an activation without z");
    return M3_OK;
}

BnParams make_params(const m3_block_norm_dims* d, const m3_block_norm_inputs* in) {
    BnParams p{};
    p.rows = static_cast<uint32_t>(d->batch * d->rows);
    p.inner = static_cast<uint32_t>(d->rows);
    p.C = static_cast<int>(d->channels);
    p.post = d->flags & M3_BN_POST_LAYER ? kLayer : d->flags & M3_BN_POST_RMS ? kRms : kNone;
    p.pre = d->flags & M3_BN_PRE_LAYER ? kLayer : d->flags & M3_BN_PRE_RMS ? kRms : kNone;
    p.act = d->flags & M3_BN_SILU ? kSilu : d->flags & M3_BN_SIGMOID ? kSigmoid : kIdentity;
    p.y = tensor(d, &in->y);
    p.x = tensor(d, &in->residual);
    p.z = tensor(d, &in->z);
    p.w1 = in->post_weight;
    p.b1 = in->post_bias;
    p.w2 = in->pre_weight;
    p.b2 = in->pre_bias;
    p.alpha = d->alpha;
    p.eps = d->eps;
    return p;
}

template <typename F>
cudaError_t with_types(const m3_block_norm_dims* d, F&& f) {
    using B = __nv_bfloat16;
    if (d->in_dtype == M3_F32) return f(float{}, float{});
    return d->res_dtype == M3_F32 ? f(B{}, float{}) : f(B{}, B{});
}

}  // namespace
}  // namespace m3

using namespace m3;

extern "C" {

m3_status m3_block_norm_fwd(const m3_block_norm_dims* dims, const m3_block_norm_inputs* in, const m3_view* h,
                            const m3_view* out, void* stream) {
    set_error(M3_OK, "");
    m3_status st = check(dims);
    if (st != M3_OK) return st;
    const bool any = dims->batch > 0 && dims->rows > 0, pre = dims->flags & (M3_BN_PRE_RMS | M3_BN_PRE_LAYER);
    const uintptr_t es = dims->in_dtype == M3_BF16 ? 2 : 4, er = dims->res_dtype == M3_BF16 ? 2 : 4;
    if ((st = check_inputs(dims, in, any)) != M3_OK || (st = check_ptr(data(h), er, "h", any)) != M3_OK ||
        (st = check_ptr(data(out), es, "out", any && pre)) != M3_OK)
        return st;
    if (!any) return M3_OK;
    BnParams p = make_params(dims, in);
    p.h = tensor(dims, h);
    if (pre) p.out = tensor(dims, out);
    const Named y{&p.y, p.y.p, "y"}, x{&p.x, p.x.p, "residual"}, z{&p.z, p.z.p, "z"};
    const Named w1{nullptr, p.w1, "post_weight"}, b1{nullptr, p.b1, "post_bias"}, w2{nullptr, p.w2, "pre_weight"},
        b2{nullptr, p.b2, "pre_bias"}, ho{&p.h, p.h.p, "h"}, oo{&p.out, p.out.p, "out"};
    if ((st = check_out(p.h, dims, "h")) != M3_OK || (pre && (st = check_out(p.out, dims, "out")) != M3_OK) ||
        (st = check_apart(ho, p.x.p, {y, x, z, w1, b1, w2, b2})) != M3_OK ||
        (st = check_apart(oo, p.y.p, {y, x, z, w1, b1, w2, b2})) != M3_OK || (st = check_apart(oo, nullptr, {ho})) != M3_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = with_types(dims, [&](auto t, auto r) { return launch_fwd<decltype(t), decltype(r)>(p, s); });
    return e == cudaSuccess ? M3_OK : err(M3_ERR_CUDA, "block norm launch: %s", cudaGetErrorString(e));
}

size_t m3_block_norm_bwd_workspace_bytes(const m3_block_norm_dims* dims) {
    if (check(dims) != M3_OK || dims->batch == 0 || dims->rows == 0) return 0;
    const size_t n = static_cast<size_t>(most_shares(dims->batch * dims->rows)) * 4 * static_cast<size_t>(dims->channels) * 4;
    return (n + 255) / 256 * 256;
}

m3_status m3_block_norm_bwd(const m3_block_norm_dims* dims, const m3_block_norm_inputs* in, const m3_view* dh,
                            const m3_view* dout, const m3_block_norm_grads* grads, void* workspace, size_t ws_bytes,
                            void* stream) {
    set_error(M3_OK, "");
    m3_status st = check(dims);
    if (st != M3_OK) return st;
    const bool any = dims->batch > 0 && dims->rows > 0, pre = dims->flags & (M3_BN_PRE_RMS | M3_BN_PRE_LAYER);
    const uintptr_t es = dims->in_dtype == M3_BF16 ? 2 : 4, er = dims->res_dtype == M3_BF16 ? 2 : 4;
    if ((st = check_inputs(dims, in, any)) != M3_OK) return st;
    if (!grads) return err(M3_ERR_INVALID_ARG, "grads is NULL");
    float* const outs[4] = {grads->dpost_weight, grads->dpost_bias, grads->dpre_weight, grads->dpre_bias};
    const char* const names[4] = {"dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias"};
    if ((st = check_ptr(data(dh), er, "dh", false)) != M3_OK || (st = check_ptr(data(dout), es, "dout", any && pre)) != M3_OK ||
        (st = check_ptr(grads->dy.data, es, "dy", any)) != M3_OK ||
        (st = check_ptr(grads->dresidual.data, er, "dresidual", any)) != M3_OK ||
        (st = check_ptr(grads->dz.data, es, "dz", any && in->z.data)) != M3_OK)
        return st;
    for (int k = 0; k < 4; ++k)
        if ((st = check_ptr(outs[k], 4, names[k], false)) != M3_OK) return st;
    if (!pre && (outs[2] || outs[3])) return err(M3_ERR_INVALID_ARG, "dpre_weight or dpre_bias without a pre norm");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!any) {
        cudaError_t e = cudaSuccess;
        for (int k = 0; k < 4 && e == cudaSuccess; ++k)
            if (outs[k]) e = cudaMemsetAsync(outs[k], 0, dims->channels * 4, s);
        return e == cudaSuccess ? M3_OK : err(M3_ERR_CUDA, "empty gradient: %s", cudaGetErrorString(e));
    }
    BnParams p = make_params(dims, in);
    p.dh = tensor(dims, dh);
    if (pre) p.dout = tensor(dims, dout);
    p.dy = tensor(dims, &grads->dy);
    p.dx = tensor(dims, &grads->dresidual);
    if (p.z.p) p.dz = tensor(dims, &grads->dz);
    const Named ins[] = {{&p.y, p.y.p, "y"}, {&p.x, p.x.p, "residual"}, {&p.z, p.z.p, "z"}, {&p.dh, p.dh.p, "dh"},
                         {&p.dout, p.dout.p, "dout"}, {nullptr, p.w1, "post_weight"}, {nullptr, p.b1, "post_bias"},
                         {nullptr, p.w2, "pre_weight"}, {nullptr, p.b2, "pre_bias"}};
    const Named gs[] = {{&p.dy, p.dy.p, "dy"}, {&p.dx, p.dx.p, "dresidual"}, {&p.dz, p.dz.p, "dz"},
                        {nullptr, outs[0], names[0]}, {nullptr, outs[1], names[1]}, {nullptr, outs[2], names[2]},
                        {nullptr, outs[3], names[3]}};
    const void* same[] = {p.dout.p, p.dh.p, nullptr, nullptr, nullptr, nullptr, nullptr};
    for (int i = 0; i < 7; ++i) {
        if (i < 3 && gs[i].p && (st = check_out(*gs[i].t, dims, gs[i].name)) != M3_OK) return st;
        if ((st = check_apart(gs[i], same[i], ins)) != M3_OK) return st;
        for (int j = 0; j < i; ++j)
            if (gs[i].p && gs[i].p == gs[j].p) return err(M3_ERR_INVALID_ARG, "%s is %s", gs[i].name, gs[j].name);
    }
    const size_t need = m3_block_norm_bwd_workspace_bytes(dims);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || ws_bytes < need)
        return err(M3_ERR_INVALID_ARG, "workspace: NULL, misaligned or below %zu bytes", need);
    for (int k = 0; k < 4; ++k)
        if (outs[k]) {
            p.sums |= 1 << k;
            ++p.nsums;
        }
    p.part = static_cast<float*>(workspace);
    const cudaError_t e = with_types(dims, [&](auto t, auto r) { return launch_bwd<decltype(t), decltype(r)>(p, outs, s); });
    return e == cudaSuccess ? M3_OK : err(M3_ERR_CUDA, "block norm backward launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
