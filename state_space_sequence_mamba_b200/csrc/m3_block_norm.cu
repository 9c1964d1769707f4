// The norms before and after a block with its gate and residual, and their gradients:
//     n = post(y),  h = x + alpha n act(z),  out = pre(h)
//
// Bound by HBM: the forward reads y, x, z and writes h, out, the backward reads those inputs, dh and dout
// and writes dy, dx, dz, each once. 8192 rows of 4096 bf16 channels, both norms RMS with weights, gated: forward 60 us (0.85 of
// what a copy reaches), gradients 115 us (0.71); with means and biases the gradients take 220. A row lies in the
// registers of a team of W warps (NV 16-byte vectors a lane), so h goes from its residual into the second norm's
// statistics without a trip through memory. What such kernels wait for are a row's meetings (shuffles, a barrier, shuffles)
// and the parameters' loads: so the sums of a row meet once, with the next row's first one, and the parameters
// lie in shared memory (gradients with four meetings, parameters from the L1 and column sums in shared memory: 190 us).
// Teams walk over rows, the next row's loads in flight. Rows too wide, or not aligned to vectors, take one CTA each
// with scalar loads.
//
// Backward, with yh = (y - mean) ry, hh = (h - mean) rh, n = yh w1 + b1 and go = dout w2:
//     d  = dh + rh (go - hh mean(go hh) - mean(go) [layer]),     dx = d
//     dz = alpha d n act'(z),  e = alpha d act(z),  g = e w1
//     dy = ry (g - yh mean(g yh) - mean(g) [layer])
//     dw2 = sum dout hh,  db2 = sum dout,  dw1 = sum e yh,  db1 = sum e
// A CTA's column sums go to the workspace and a second launch adds them in a fixed order.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <type_traits>

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
enum Norm { kNone = 0, kRms = 1, kLayerNorm = 2 };
enum Act { kIdentity = 0, kSigmoid = 1, kSilu = 2, kNoGate = 3 };
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

// A thread's part of a row: the N channels of one 16-byte word of the block's type. A tensor of TR has U words of them.
template <typename T>
constexpr int channels() { return 16 / static_cast<int>(sizeof(T)); }
template <typename TR, int N>
constexpr int words() { return N * static_cast<int>(sizeof(TR)) / 16; }
template <typename TR, int N, int U>
__device__ __forceinline__ void unpack(const uint4 (&w)[U], float2 (&f)[N / 2]) {
#pragma unroll
    for (int u = 0; u < U; ++u) Vec<TR>::unpack(w[u], f + u * Vec<TR>::N);
}
template <typename TR, int N>
__device__ __forceinline__ void store(TR* p, const float2 (&f)[N / 2]) {
    constexpr int U = words<TR, N>();
#pragma unroll
    for (int u = 0; u < U; ++u) Vec<TR>::store(p + u * 2 * Vec<TR>::N, f + u * Vec<TR>::N);
}
// 16 bytes from memory to this thread's place in shared memory, without waiting for them
__device__ __forceinline__ void copy_async(uint4* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sm100::smem_u32(dst)), "l"(src) : "memory");
}
template <int keep>
__device__ __forceinline__ void copies_left() { asm volatile("cp.async.wait_group %0;" ::"n"(keep) : "memory"); }
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// The gate and its slope. kNoGate: one, without z.
template <int kAct>
__device__ __forceinline__ float2 act2(const float2& z) {
    if (kAct == kIdentity) return z;
    const float2 s = sigmoid2(z);
    return kAct == kSigmoid ? s : mul2(z, s);
}
template <int kAct>
__device__ __forceinline__ void act_slope2(const float2& z, float2* a, float2* da) {
    if (kAct == kIdentity) {
        *a = z;
        *da = both(1.f);
        return;
    }
    const float2 s = sigmoid2(z), t = fma2(s, both(-1.f), both(1.f));
    if (kAct == kSigmoid) {
        *a = s;
        *da = mul2(s, t);
    } else {
        *a = mul2(z, s);
        *da = fma2(*a, t, s);       // s (1 + z (1 - s))
    }
}
template <int k>
struct ActIs {
    static constexpr int value = k;
};
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    if (act == kSilu) f(ActIs<kSilu>{});
    else if (act == kSigmoid) f(ActIs<kSigmoid>{});
    else if (act == kIdentity) f(ActIs<kIdentity>{});
    else f(ActIs<kNoGate>{});
}

// A team: W warps that hold one row. K sums at once: a warp halves what each lane holds as it adds (K - 1 shuffles and
// the rest of the tree, in place of 5 K), the warps' sums meet in shared memory behind one barrier, in two places in turn.
template <int W, int kTeams>
struct Team {
    float (*s)[kTeams][W][16];
    int team, warp, lane, turn = 0;
    __device__ __forceinline__ explicit Team(float (*places)[kTeams][W][16]) : s(places) {
        team = kTeams == 1 ? 0 : threadIdx.x / (32 * W);
        warp = (threadIdx.x / 32) % W;
        lane = threadIdx.x & 31;
    }
    template <int K>        // a power of two
    __device__ __forceinline__ void sum(float (&a)[K]) {
        constexpr int per = 32 / K;     // lane per j + i ends with the sum of value j
#pragma unroll
        for (int n = K / 2; n >= 1; n /= 2) {
            const bool up = lane & (per * n);
#pragma unroll
            for (int k = 0; k < n; ++k) {
                const float give = up ? a[k] : a[k + n], keep = up ? a[k + n] : a[k];
                a[k] = keep + __shfl_xor_sync(0xffffffffu, give, per * n);
            }
        }
        float t = a[0];
#pragma unroll
        for (int o = per / 2; o >= 1; o /= 2) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (W == 1) {
#pragma unroll
            for (int k = 0; k < K; ++k) a[k] = __shfl_sync(0xffffffffu, t, per * k);
            return;
        }
        if (lane % per == 0) s[turn][team][warp][lane / per] = t;
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(32 * W) : "memory");
        // lane K w + j takes value j of warps w, w + per, ...
        t = lane / K < W ? s[turn][team][lane / K][lane % K] : 0.f;
#pragma unroll
        for (int w = per; w < W; w += per) t += s[turn][team][w + lane / K][lane % K];
        turn ^= 1;
#pragma unroll
        for (int o = K; o < K * W && o < 32; o *= 2) t += __shfl_xor_sync(0xffffffffu, t, o);
#pragma unroll
        for (int k = 0; k < K; ++k) a[k] = __shfl_sync(0xffffffffu, t, k);
    }
};

// One tensor's rows in the order that a team walks through them.
template <typename T>
struct RowPtr {
    T* q;
    int64_t step;
    __device__ __forceinline__ RowPtr(const BnTensor& t, const BnParams& p, uint32_t row, uint32_t by)
        : q(t.p && row < p.rows ? at<T>(t, p, row) : nullptr), step(static_cast<int64_t>(by) * t.row) {}
    // to the row `row`, `by` behind the last one
    __device__ __forceinline__ void next(const BnTensor& t, const BnParams& p, uint32_t row) {
        if (p.inner == p.rows) q += step;
        else if (row < p.rows && t.p) q = at<T>(t, p, row);
    }
};

// The channels' parameters, in shared memory as the threads read them: word q of vector i of thread t lies beside the
// other threads' (from the L1 they would be a wait each, and the rows push them out of it). Parts beyond the row hold zeros.
struct Params {
    const float4* w[4];         // w1, b1, w2, b2 of this thread, or null
};
template <int W, int NV, int N>
__device__ __forceinline__ Params load_params(const BnParams& p, float4* room) {
    constexpr int Q = N / 4, kPlanes = NV * Q;
    const float* const from[4] = {p.w1, p.b1, p.w2, p.b2};      // (the backward has no use for b2)
    Params r{};
    const int t = threadIdx.x % (32 * W);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (!from[k]) continue;
        r.w[k] = room + t;
        if (threadIdx.x < 32 * W)
#pragma unroll
            for (int i = 0; i < kPlanes; ++i) {
                const int c = ((i / Q) * 32 * W + t) * N + 4 * (i % Q);
                room[i * 32 * W + t] = c < p.C ? make_float4(__ldg(from[k] + c), __ldg(from[k] + c + 1), __ldg(from[k] + c + 2), __ldg(from[k] + c + 3))
                                               : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        room += kPlanes * 32 * W;
    }
    return r;
}
// v times a channel's weight plus its bias, where there are any
template <int W, int N>
__device__ __forceinline__ void scaled(const float4* w, const float4* b, int i, float2 (&v)[N / 2]) {
    constexpr int Q = N / 4;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        if (w) {
            const float4 f = w[(i * Q + q) * 32 * W];
            v[2 * q] = mul2(v[2 * q], make_float2(f.x, f.y));
            v[2 * q + 1] = mul2(v[2 * q + 1], make_float2(f.z, f.w));
        }
        if (b) {
            const float4 f = b[(i * Q + q) * 32 * W];
            v[2 * q] = add2(v[2 * q], make_float2(f.x, f.y));
            v[2 * q + 1] = add2(v[2 * q + 1], make_float2(f.z, f.w));
        }
    }
}

template <int W>
constexpr int block_threads() { return 32 * (W > 8 ? W : 8); }

// kLayer: one of the norms takes its mean off; without it, the sum of y^2 of the next row comes with h^2 of this one,
// and a row has one meeting.
template <typename T, typename TR, int W, int NV, bool kLayer>
__global__ void __launch_bounds__(block_threads<W>(), 768 / block_threads<W>()) bn_fwd_kernel(const __grid_constant__ BnParams p) {
    constexpr int kTeams = block_threads<W>() / (32 * W), N = channels<T>(), H = N / 2, U = words<TR, N>();
    __shared__ float s_sum[2][kTeams][W][16];
    extern __shared__ float4 s_dyn[];       // the parameters
    Team<W, kTeams> team(s_sum);
    const int c0 = static_cast<int>(threadIdx.x % (32 * W)) * N;
    constexpr int kStep = 32 * W * N;       // channels from part to part
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) in[i] = c0 + i * kStep < p.C;
    const float inv = 1.f / p.C;
    const uint32_t step = gridDim.x * kTeams;
    uint32_t row = blockIdx.x * kTeams + team.team;
    RowPtr<const T> y(p.y, p, row, step), z(p.z, p, row, step);
    RowPtr<const TR> x(p.x, p, row, step);
    RowPtr<T> out(p.out, p, row, step);
    RowPtr<TR> h(p.h, p, row, step);
    uint4 ry[NV][1] = {}, rz[NV][1] = {}, rx[NV][U] = {};
    const auto fetch = [&](bool live) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!live || !in[i]) continue;
            ry[i][0] = __ldcs(reinterpret_cast<const uint4*>(y.q + c0 + i * kStep));
#pragma unroll
            for (int u = 0; u < U; ++u) rx[i][u] = __ldcs(reinterpret_cast<const uint4*>(x.q + c0 + i * kStep) + u);
            if (p.z.p) rz[i][0] = __ldcs(reinterpret_cast<const uint4*>(z.q + c0 + i * kStep));
        }
    };
    // the mean of a row's values (zero beyond the row), and the sum of what deviates from it squared
    const auto mean = [&](const float2 (&v)[NV][H]) {
        float2 s = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < H; ++e) s = add2(s, v[i][e]);
        float a[1] = {s.x + s.y};
        team.sum(a);
        return a[0] * inv;
    };
    const auto squares = [&](const float2 (&v)[NV][H]) {
        float2 s = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < H; ++e) s = fma2(v[i][e], v[i][e], s);
        return s.x + s.y;
    };
    const auto centre = [&](float2 (&v)[NV][H]) {
        const float m = mean(v);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < H; ++e) v[i][e] = add2(v[i][e], both(in[i] ? -m : 0.f));
    };
    const auto spread = [&](float sum) { return rsqrtf(fmaf(sum, inv, p.eps)); };
    fetch(row < p.rows);
    const Params w = load_params<W, NV, N>(p, s_dyn);
    __syncthreads();
    float r1 = 1.f;
    if (!kLayer && p.post != kNone) {
        float2 v[NV][H];
#pragma unroll
        for (int i = 0; i < NV; ++i) unpack<T, N>(ry[i], v[i]);
        float a[1] = {squares(v)};
        team.sum(a);
        r1 = spread(a[0]);
    }
    for (; row < p.rows; row += step) {
        float2 v[NV][H];
        uint4 cx[NV][U], cz[NV][1];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack<T, N>(ry[i], v[i]);
            cz[i][0] = rz[i][0];
#pragma unroll
            for (int u = 0; u < U; ++u) cx[i][u] = rx[i][u];
        }
        y.next(p.y, p, row + step);
        x.next(p.x, p, row + step);
        z.next(p.z, p, row + step);
        fetch(row + step < p.rows);
        if (kLayer && p.post != kNone) {
            if (p.post == kLayerNorm) centre(v);
            float a[1] = {squares(v)};
            team.sum(a);
            r1 = spread(a[0]);
        }
        with_act(p.act, [&](auto act) {
            constexpr int kAct = decltype(act)::value;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 u[H], g[H];
#pragma unroll
                for (int e = 0; e < H; ++e) v[i][e] = mul2(v[i][e], both(r1));
                scaled<W, N>(w.w[0], w.w[1], i, v[i]);
                unpack<TR, N>(cx[i], u);
                if (kAct != kNoGate) unpack<T, N>(cz[i], g);
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    const float2 n = kAct != kNoGate ? mul2(v[i][e], act2<kAct>(g[e])) : v[i][e];
                    v[i][e] = fma2(n, both(p.alpha), u[e]);
                }
                if (in[i]) store<TR, N>(h.q + c0 + i * kStep, v[i]);
            }
        });
        h.next(p.h, p, row + step);
        float r2 = 1.f;
        if (kLayer) {
            if (p.pre == kNone) continue;
            if (p.pre == kLayerNorm) centre(v);
            float a[1] = {squares(v)};
            team.sum(a);
            r2 = spread(a[0]);
        } else {
            if (p.pre == kNone && p.post == kNone) continue;
            float2 n[NV][H];
#pragma unroll
            for (int i = 0; i < NV; ++i) unpack<T, N>(ry[i], n[i]);
            float a[2] = {squares(v), squares(n)};
            team.sum(a);
            r2 = spread(a[0]);
            if (p.post != kNone) r1 = spread(a[1]);
            if (p.pre == kNone) continue;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < H; ++e) v[i][e] = mul2(v[i][e], both(r2));
            scaled<W, N>(w.w[2], w.w[3], i, v[i]);
            if (in[i]) store<T, N>(out.q + c0 + i * kStep, v[i]);
        }
        out.next(p.out, p, row + step);
    }
}

// Backward. Every sum over a row is linear in what the other sums give, so that one meeting is enough (two with a mean):
// with yh known, hc = h (less its mean), go = dout w2, e = alpha act(z) w1, t = e yh, and q = rh^3 (go.hc) / C,
//     d = dh + rh go - q hc [- rh mean(go)],
//     g.yh = t.dh + rh t.go - q t.hc [- rh mean(go) sum t],     sum g likewise with e for t
// and the next row's y^2 comes with them. The second walk over the row then finds the three gradients. kStaged:
// the rows' tensors go through shared memory, each thread's parts in its own places, the next row's while one is
// worked on; rows too wide for that are read from memory in each walk. dw1 and dw2 are summed in registers, db1 and db2,
// where wanted, in shared memory.
template <typename T, typename TR, int W, int NV, bool kLayer, bool kStaged>
__global__ void __launch_bounds__(block_threads<W>(), 512 / block_threads<W>()) bn_bwd_kernel(const __grid_constant__ BnParams p) {
    constexpr int kAll = block_threads<W>(), kTeams = kAll / (32 * W);
    constexpr int N = channels<T>(), H = N / 2, Q = N / 4, U = words<TR, N>();
    constexpr int kRow = 3 + 2 * U;         // words of a part in all five tensors: y, z, dout, x, dh
    __shared__ float s_sum[2][kTeams][W][16];
    extern __shared__ float4 s_dyn[];       // the stages [2][NV][kRow][threads]; db1, db2 [NV][Q][threads] each; parameters
    sm100::grid_dep_launch_dependents();
    Team<W, kTeams> team(s_sum);
    uint4* const stages = reinterpret_cast<uint4*>(s_dyn) + threadIdx.x;
    float4* const biases = s_dyn + (kStaged ? 2 * NV * kRow * kAll : 0) + threadIdx.x;
    const bool any_bias = p.sums & 10;
    const int t = threadIdx.x % (32 * W), c0 = t * N;
    constexpr int kStep = 32 * W * N;       // channels from part to part
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) in[i] = c0 + i * kStep < p.C;
    if (kStaged)            // (what is not fetched stays zero)
        for (int i = 0; i < 2 * NV * kRow; ++i) stages[i * kAll] = make_uint4(0u, 0u, 0u, 0u);
    if (any_bias)
        for (int i = 0; i < 2 * NV * Q; ++i) biases[i * kAll] = make_float4(0.f, 0.f, 0.f, 0.f);
    float2 sw[2][NV][H];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < H; ++e) sw[0][i][e] = sw[1][i][e] = both(0.f);
    const auto add_bias = [&](int which, int i, const float2 (&v)[H]) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            float4& a = biases[((which * NV + i) * Q + q) * kAll];
            a = make_float4(a.x + v[2 * q].x, a.y + v[2 * q].y, a.z + v[2 * q + 1].x, a.w + v[2 * q + 1].y);
        }
    };
    const uint32_t step = gridDim.x * kTeams;
    uint32_t row = blockIdx.x * kTeams + team.team;
    RowPtr<const T> y(p.y, p, row, step), z(p.z, p, row, step), o(p.dout, p, row, step);
    RowPtr<const TR> x(p.x, p, row, step), dh(p.dh, p, row, step);
    RowPtr<T> dy(p.dy, p, row, step), dz(p.dz, p, row, step);
    RowPtr<TR> dx(p.dx, p, row, step);
    // a row into a stage, y first (its sums are wanted earlier); the pointers move on to the next one
    const auto fetch = [&](uint32_t r, int s) {
        if (!kStaged) return;
        const auto place = [&](int i, int k) { return stages + ((s * NV + i) * kRow + k) * kAll; };
        const bool live = r < p.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && in[i]) copy_async(place(i, 0), y.q + c0 + i * kStep);
        copies_end();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!live || !in[i]) continue;
            if (p.z.p) copy_async(place(i, 1), z.q + c0 + i * kStep);
            if (p.dout.p) copy_async(place(i, 2), o.q + c0 + i * kStep);
#pragma unroll
            for (int u = 0; u < U; ++u) copy_async(place(i, 3 + u), reinterpret_cast<const uint4*>(x.q + c0 + i * kStep) + u);
            if (p.dh.p)
#pragma unroll
                for (int u = 0; u < U; ++u) copy_async(place(i, 3 + U + u), reinterpret_cast<const uint4*>(dh.q + c0 + i * kStep) + u);
        }
        copies_end();
    };
    const auto advance = [&](uint32_t r) {
        y.next(p.y, p, r);
        z.next(p.z, p, r);
        o.next(p.dout, p, r);
        x.next(p.x, p, r);
        dh.next(p.dh, p, r);
    };
    // a part of one tensor: k and U words as staged, or `from` in memory
    int stage = 0;
    const auto part_t = [&](int s, int k, int i, const T* from, float2 (&f)[H]) {
        uint4 v[1] = {};
        if (kStaged) v[0] = stages[((s * NV + i) * kRow + k) * kAll];
        else if (from && in[i]) v[0] = *reinterpret_cast<const uint4*>(from + c0 + i * kStep);
        unpack<T, N>(v, f);
    };
    const auto part_r = [&](int s, int k, int i, const TR* from, float2 (&f)[H]) {
        uint4 v[U] = {};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (kStaged) v[u] = stages[((s * NV + i) * kRow + k + u) * kAll];
            else if (from && in[i]) v[u] = reinterpret_cast<const uint4*>(from + c0 + i * kStep)[u];
        }
        unpack<TR, N>(v, f);
    };
    // sums over the row of y in a stage (or at `from`): of what deviates from m, squared or as it is
    const auto y_sum = [&](int s, const T* from, float m, bool squared) {
        float2 q = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float2 v[H];
            part_t(s, 0, i, from, v);
            const float2 mi = both(kLayer && in[i] ? -m : 0.f);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                const float2 u = kLayer ? add2(v[e], mi) : v[e];
                q = squared ? fma2(u, u, q) : add2(q, u);
            }
        }
        return q.x + q.y;
    };
    const float inv = 1.f / p.C;
    fetch(row, 0);
    const Params w = load_params<W, NV, N>(p, biases - threadIdx.x + (any_bias ? 2 * NV * Q * kAll : 0));
    __syncthreads();
    if (kStaged) copies_left<1>();
    float r1 = 1.f, my = 0.f;
    if (p.post != kNone && (kStaged || row < p.rows)) {
        float a[1];
        if (kLayer && p.post == kLayerNorm) {
            a[0] = y_sum(0, y.q, 0.f, false);
            team.sum(a);
            my = a[0] * inv;
        }
        a[0] = y_sum(0, y.q, my, true);
        team.sum(a);
        r1 = rsqrtf(fmaf(a[0], inv, p.eps));
    }
    const T *py = y.q, *pz = z.q, *po = o.q;
    const TR *px = x.q, *pd = dh.q;
    for (; row < p.rows; row += step) {
        py = y.q, pz = z.q, po = o.q, px = x.q, pd = dh.q;
        advance(row + step);
        fetch(row + step, stage ^ 1);
        if (kStaged) copies_left<2>();      // all of this row
        const bool more = kStaged || row + step < p.rows;
        float2 h[NV][H];
        // yh of a part
        const auto yhat = [&](int i, float2 (&v)[H]) {
            part_t(stage, 0, i, py, v);
            const float2 mi = both(kLayer && in[i] ? -my : 0.f);
#pragma unroll
            for (int e = 0; e < H; ++e) v[e] = mul2(kLayer ? add2(v[e], mi) : v[e], both(r1));
        };
        float mh = 0.f, my1 = 0.f;
        // h of a part and its yh, from e = alpha act(z)
        const auto find_h = [&](int i, float2 (&v)[H], const float2 (&e)[H]) {
            float2 u[H], n[H];
            yhat(i, v);
            part_r(stage, 3, i, px, u);
#pragma unroll
            for (int k = 0; k < H; ++k) n[k] = v[k];
            scaled<W, N>(w.w[0], w.w[1], i, n);
#pragma unroll
            for (int k = 0; k < H; ++k) h[i][k] = fma2(n[k], e[k], u[k]);
        };
        if (kLayer) {       // the means first
            float2 s = both(0.f);
            with_act(p.act, [&](auto act) {
                constexpr int kAct = decltype(act)::value;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float2 v[H], e[H], g[H];
                    if (kAct != kNoGate) part_t(stage, 1, i, pz, g);
#pragma unroll
                    for (int k = 0; k < H; ++k) e[k] = kAct != kNoGate ? mul2(act2<kAct>(g[k]), both(p.alpha)) : both(p.alpha);
                    find_h(i, v, e);
#pragma unroll
                    for (int k = 0; k < H; ++k) s = add2(s, h[i][k]);
                }
            });
            if (kStaged) copies_left<1>();
            float a[2] = {s.x + s.y, p.post == kLayerNorm && more ? y_sum(stage ^ 1, y.q, 0.f, false) : 0.f};
            team.sum(a);
            if (p.pre == kLayerNorm) mh = a[0] * inv;
            my1 = a[1] * inv;
        }
        float2 s0 = both(0.f), s1 = s0, s2 = s0, s3 = s0, s4 = s0, s5 = s0, s6 = s0, s7 = s0, s8 = s0, s9 = s0, s10 = s0;
        with_act(p.act, [&](auto act) {
            constexpr int kAct = decltype(act)::value;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 v[H], e[H], g[H], d[H];
                if (kAct != kNoGate) part_t(stage, 1, i, pz, g);
#pragma unroll
                for (int k = 0; k < H; ++k) e[k] = kAct != kNoGate ? mul2(act2<kAct>(g[k]), both(p.alpha)) : both(p.alpha);
                find_h(i, v, e);
                part_r(stage, 3 + U, i, pd, d);
                part_t(stage, 2, i, po, g);
                scaled<W, N>(w.w[2], nullptr, i, g);
                scaled<W, N>(w.w[0], nullptr, i, e);
                const float2 mi = both(kLayer && in[i] ? -mh : 0.f);
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    if (kLayer) h[i][k] = add2(h[i][k], mi);
                    const float2 tk = mul2(v[k], e[k]);
                    s0 = fma2(h[i][k], h[i][k], s0);
                    s1 = fma2(g[k], h[i][k], s1);
                    s2 = fma2(tk, d[k], s2);
                    s3 = fma2(tk, g[k], s3);
                    s4 = fma2(tk, h[i][k], s4);
                    if (!kLayer || !in[i]) continue;
                    s5 = add2(s5, g[k]);
                    s6 = add2(s6, tk);
                    s7 = fma2(e[k], d[k], s7);
                    s8 = fma2(e[k], g[k], s8);
                    s9 = fma2(e[k], h[i][k], s9);
                    s10 = add2(s10, e[k]);
                }
            }
        });
        if (kStaged) copies_left<1>();      // y of the next row
        const float ysq = p.post != kNone && more ? y_sum(stage ^ 1, y.q, my1, true) : 0.f;
        float r2 = 0.f, k2 = 0.f, m2 = 0.f, m1 = 0.f, n1 = 0.f, next;
        const auto join = [](const float2& v) { return v.x + v.y; };
        if (!kLayer) {
            float a[8] = {join(s0), join(s1), join(s2), join(s3), join(s4), ysq, 0.f, 0.f};
            team.sum(a);
            if (p.pre != kNone) {
                r2 = rsqrtf(fmaf(a[0], inv, p.eps));
                k2 = -r2 * (r2 * (r2 * (a[1] * inv)));     // (r2^3 alone may leave fp32)
            }
            if (p.post != kNone) m1 = -(a[2] + (p.pre != kNone ? fmaf(r2, a[3], k2 * a[4]) : 0.f)) * inv * r1;
            next = a[5];
        } else {
            float a[16] = {join(s0), join(s1), join(s2), join(s3), join(s4), ysq, join(s5), join(s6), join(s7), join(s8),
                           join(s9), join(s10), 0.f, 0.f, 0.f, 0.f};
            team.sum(a);
            if (p.pre != kNone) {
                r2 = rsqrtf(fmaf(a[0], inv, p.eps));
                k2 = -r2 * (r2 * (r2 * (a[1] * inv)));
                if (p.pre == kLayerNorm) m2 = -r2 * a[6] * inv;
            }
            const bool pre = p.pre != kNone;
            if (p.post != kNone) m1 = -(a[2] + (pre ? fmaf(r2, a[3], k2 * a[4]) + m2 * a[7] : 0.f)) * inv * r1;
            if (p.post == kLayerNorm) n1 = -(a[8] + (pre ? fmaf(r2, a[9], k2 * a[10]) + m2 * a[11] : 0.f)) * inv * r1;
            next = a[5];
        }
        with_act(p.act, [&](auto act) {
            constexpr int kAct = decltype(act)::value;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!in[i]) continue;
                float2 v[H], d[H], n[H], g[H];
                yhat(i, v);
                part_r(stage, 3 + U, i, pd, d);
                if (p.pre != kNone) {
                    part_t(stage, 2, i, po, g);
#pragma unroll
                    for (int k = 0; k < H; ++k) sw[1][i][k] = fma2(g[k], mul2(h[i][k], both(r2)), sw[1][i][k]);
                    if (p.sums & 8) add_bias(1, i, g);
                    scaled<W, N>(w.w[2], nullptr, i, g);
#pragma unroll
                    for (int k = 0; k < H; ++k) {
                        d[k] = fma2(g[k], both(r2), fma2(h[i][k], both(k2), d[k]));
                        if (kLayer) d[k] = add2(d[k], both(m2));
                    }
                }
                store<TR, N>(dx.q + c0 + i * kStep, d);
#pragma unroll
                for (int k = 0; k < H; ++k) d[k] = mul2(d[k], both(p.alpha));
                if constexpr (kAct != kNoGate) {
#pragma unroll
                    for (int k = 0; k < H; ++k) n[k] = v[k];
                    scaled<W, N>(w.w[0], w.w[1], i, n);
                    part_t(stage, 1, i, pz, g);
#pragma unroll
                    for (int k = 0; k < H; ++k) {
                        float2 a, da;
                        act_slope2<kAct>(g[k], &a, &da);
                        g[k] = mul2(mul2(d[k], n[k]), da);
                        d[k] = mul2(d[k], a);
                    }
                    store<T, N>(dz.q + c0 + i * kStep, g);
                }
#pragma unroll
                for (int k = 0; k < H; ++k) sw[0][i][k] = fma2(d[k], v[k], sw[0][i][k]);
                if (p.sums & 2) add_bias(0, i, d);
                scaled<W, N>(w.w[0], nullptr, i, d);
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    d[k] = fma2(d[k], both(r1), mul2(v[k], both(m1)));
                    if (kLayer) d[k] = add2(d[k], both(n1));
                }
                store<T, N>(dy.q + c0 + i * kStep, d);
            }
        });
        if (p.post != kNone) r1 = rsqrtf(fmaf(next, inv, p.eps));
        my = my1;
        dx.next(p.dx, p, row + step);
        dz.next(p.dz, p, row + step);
        dy.next(p.dy, p, row + step);
        stage ^= 1;
    }
    if (p.nsums == 0) return;
    // the teams' sums, added in order, to the CTA's share (a sum at a time, through the dynamic shared memory)
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.nsums * p.C;
    copies_left<0>();
    float4 keep[2][NV * Q];
    if (any_bias)
#pragma unroll
        for (int i = 0; i < 2 * NV * Q; ++i) keep[i / (NV * Q)][i % (NV * Q)] = biases[i * kAll];
    float4* const sums = s_dyn;             // [NV][Q][threads]
    for (int which = 0, n = 0; which < 4; ++which) {
        if (!(p.sums >> which & 1)) continue;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                float4 v;
                if (which == 1) v = keep[0][i * Q + q];
                else if (which == 3) v = keep[1][i * Q + q];
                else if (which == 0) v = make_float4(sw[0][i][2 * q].x, sw[0][i][2 * q].y, sw[0][i][2 * q + 1].x, sw[0][i][2 * q + 1].y);
                else v = make_float4(sw[1][i][2 * q].x, sw[1][i][2 * q].y, sw[1][i][2 * q + 1].x, sw[1][i][2 * q + 1].y);
                sums[(i * Q + q) * kAll + threadIdx.x] = v;
            }
        __syncthreads();
        if (team.team == 0)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    if (!in[i]) continue;
                    float4 a = sums[(i * Q + q) * kAll + t];
                    for (int u = 1; u < kTeams; ++u) {
                        const float4 f = sums[(i * Q + q) * kAll + u * 32 * W + t];
                        a = make_float4(a.x + f.x, a.y + f.y, a.z + f.z, a.w + f.w);
                    }
                    *reinterpret_cast<float4*>(part + static_cast<int64_t>(n) * p.C + c0 + i * kStep + 4 * q) = a;
                }
        ++n;
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

__device__ __forceinline__ float2 act1(int act, float z) {
    float2 a = both(1.f), da = both(0.f);
    with_act(act, [&](auto k) {
        if constexpr (decltype(k)::value != kNoGate) act_slope2<decltype(k)::value>(both(z), &a, &da);
    });
    return make_float2(a.x, da.x);
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
        return to_f(x[c]) + (z ? v * act1(p.act, to_f(z[c])).x : v);
    }
    template <typename F>
    __device__ __forceinline__ void stats(int kind, F&& v, float* m, float* r, float* s) {
        if (kind == kNone) return;
        float mean = 0.f, q = 0.f;
        if (kind == kLayerNorm) {
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
            u2 = p.pre == kLayerNorm ? block_sum(u2, s) / p.C : 0.f;
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
                    const float2 f = act1(p.act, to_f(a.z[c]));
                    e *= f.x;
                    slope = f.y;
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
                v2 = p.post == kLayerNorm ? block_sum(v2, s) / p.C : 0.f;
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
// Warps and parts a lane for a row of `parts` parts: two a lane from 32 lanes on, which is what registers (and,
// backward, the stages) hold for two rows an SM at 512 parts; wider rows have an SM each, up to kMostChannels, the most
// whose parameters fit beside them.
template <typename T, typename F>
auto with_shape(int parts, F&& f) {
    if (parts <= 32) return f(Shape<1, 1>{});
    if (parts <= 64) return f(Shape<1, 2>{});
    if (parts <= 128) return f(Shape<2, 2>{});
    if (parts <= 256) return f(Shape<4, 2>{});
    if (parts <= 512) return f(Shape<8, 2>{});
    if constexpr (sizeof(T) == 4) {
        if (parts > 1024) return f(Shape<16, 4>{});
    }
    return f(Shape<16, 2>{});
}
constexpr int kMostChannels = 8192;

bool ok16(const BnTensor& t, int es) {
    return !t.p || ((reinterpret_cast<uintptr_t>(t.p) | static_cast<uintptr_t>(t.batch * es) |
                     static_cast<uintptr_t>(t.row * es)) & 15u) == 0;
}

// 16-byte parts of a row, or 0 where that form does not apply
template <typename T, typename TR>
int part_count(const BnParams& p) {
    constexpr int N = channels<T>();
    if (p.C % N != 0 || p.C > kMostChannels) return 0;
    for (const BnTensor* t : {&p.y, &p.z, &p.out, &p.dout, &p.dy, &p.dz})
        if (!ok16(*t, sizeof(T))) return 0;
    for (const BnTensor* t : {&p.x, &p.h, &p.dh, &p.dx})
        if (!ok16(*t, sizeof(TR))) return 0;
    return p.C / N;
}

// a kernel and its bytes of shared memory beside its sums
template <auto k, int n>
struct Kernel {
    static constexpr auto f = k;
    static constexpr int bytes = n;
};

constexpr int kRoom = 225 * 1024;       // dynamic shared memory of a CTA, beside its teams' places
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
    const int parts = part_count<T, TR>(p);
    const int64_t sms = device_sm_count();
    if (parts == 0) {
        const int64_t grid = p.rows < 16 * sms ? p.rows : 16 * sms;
        bn_fwd_any_kernel<T, TR><<<static_cast<unsigned>(grid), kAny, 0, s>>>(p);
        return cudaGetLastError();
    }
    cudaError_t e = cudaSuccess;
    const bool layer = p.post == kLayerNorm || p.pre == kLayerNorm;
    const int params = (p.w1 != nullptr) + (p.b1 != nullptr) + (p.w2 != nullptr) + (p.b2 != nullptr);
    with_shape<T>(parts, [&](auto sh) {
        using S = decltype(sh);
        constexpr int threads = block_threads<S::W>(), teams = threads / (32 * S::W);
        constexpr int one = S::NV * 32 * S::W * channels<T>() * 4;     // bytes of one parameter: up to 32 KB
        const auto go = [&](auto k) {
            using K = decltype(k);
            static std::atomic<uint64_t> done{0};
            if ((e = allow_smem(K::f, 4 * one < kRoom ? K::bytes + 4 * one : kRoom, done)) != cudaSuccess) return;
            static const int per_sm[5] = {resident(K::f, threads, 0), resident(K::f, threads, one), resident(K::f, threads, 2 * one),
                                          resident(K::f, threads, 3 * one), resident(K::f, threads, 4 * one)};
            const int64_t want = (p.rows + teams - 1) / teams, most = per_sm[params] * sms;
            K::f<<<static_cast<unsigned>(want < most ? want : most), threads, params * one, s>>>(p);
        };
        if (layer) go(Kernel<bn_fwd_kernel<T, TR, S::W, S::NV, true>, 0>{});
        else go(Kernel<bn_fwd_kernel<T, TR, S::W, S::NV, false>, 0>{});
        return 0;
    });
    return e == cudaSuccess ? cudaGetLastError() : e;
}

template <typename T, typename TR>
cudaError_t launch_bwd(BnParams p, float* const (&outs)[4], cudaStream_t s) {
    const int parts = part_count<T, TR>(p);
    int shares = 1;
    float* wanted[4] = {};
    for (int k = 0, n = 0; k < 4; ++k)
        if (p.sums >> k & 1) wanted[n++] = outs[k];
    cudaError_t e = cudaSuccess;
    const bool layer = p.post == kLayerNorm || p.pre == kLayerNorm;
    p.b2 = nullptr;         // has no part in any gradient
    const int params = (p.w1 != nullptr) + (p.b1 != nullptr) + (p.w2 != nullptr);
    if (parts > 0) with_shape<T>(parts, [&](auto sh) {
        using S = decltype(sh);
        constexpr int threads = block_threads<S::W>(), teams = threads / (32 * S::W), N = channels<T>();
        constexpr int one = S::NV * 32 * S::W * N * 4, staged = 2 * S::NV * threads * 16 * (3 + 2 * words<TR, N>());
        const auto go = [&](auto k) {
            using K = decltype(k);
            // parameters, db1 and db2, and room for one sum at the end
            int smem = K::bytes + params * one + (p.sums & 10 ? 2 * teams * one : 0);
            if (smem < teams * one) smem = teams * one;
            static std::atomic<uint64_t> done{0};
            if ((e = allow_smem(K::f, kRoom, done)) != cudaSuccess) return;
            static std::atomic<int> per_sm[5][2];       // looked up once (all devices are alike)
            std::atomic<int>& known = per_sm[params][p.sums & 10 ? 1 : 0];
            int fit = known.load(std::memory_order_relaxed);
            if (fit == 0) known.store(fit = resident(K::f, threads, smem), std::memory_order_relaxed);
            const int64_t want = (p.rows + teams - 1) / teams;
            const int64_t all = device_sm_count() * static_cast<int64_t>(fit < kMostPerSm ? fit : kMostPerSm);
            shares = static_cast<int>(want < all ? want : all);
            K::f<<<static_cast<unsigned>(shares), threads, smem, s>>>(p);
        };
        if constexpr (staged <= kRoom) {
            if (staged + params * one + (p.sums & 10 ? 2 * teams * one : 0) <= kRoom) {
                if (layer) go(Kernel<bn_bwd_kernel<T, TR, S::W, S::NV, true, true>, staged>{});
                else go(Kernel<bn_bwd_kernel<T, TR, S::W, S::NV, false, true>, staged>{});
                return 0;
            }
        }
        if constexpr (staged + 4 * one + 2 * teams * one > kRoom) {
            if (layer) go(Kernel<bn_bwd_kernel<T, TR, S::W, S::NV, true, false>, 0>{});
            else go(Kernel<bn_bwd_kernel<T, TR, S::W, S::NV, false, false>, 0>{});
        }
        return 0;
    });
    if (e != cudaSuccess) return e;
    if (parts == 0) {
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
    // (rows are counted in 32 bits, up to two walks' steps beyond the last)
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
    p.post = d->flags & M3_BN_POST_LAYER ? kLayerNorm : d->flags & M3_BN_POST_RMS ? kRms : kNone;
    p.pre = d->flags & M3_BN_PRE_LAYER ? kLayerNorm : d->flags & M3_BN_PRE_RMS ? kRms : kNone;
    p.act = !in->z.data ? kNoGate : d->flags & M3_BN_SILU ? kSilu : d->flags & M3_BN_SIGMOID ? kSigmoid : kIdentity;
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
