// One token of linear attention for every sequence: S <- a S + k v^T, o = scale S^T q. Prompts of one
// token come here too, with or without a state before and after.
//
// Bound by HBM: the fp32 state (K V 4 bytes per sequence and head) is read once and written once,
// 5 flops per 8 bytes. A CTA owns a sequence's head (or, where there are fewer of those than CTA
// slots, a part of its columns); its 256 threads stand side by side over tx float4 columns and over
// 256 / tx rows, so that a CTA reads and writes its state front to back, and each thread issues the
// loads of up to 8 rows before it uses the first. The products with q are summed over the thread's
// rows in registers, then over the row groups through shared memory, in a fixed order. 128 sequences
// of 64 heads of 128 x 64: 81 us, 6.65 TB/s (what a plain copy reaches on this card).
#include "m3_common.cuh"
#include "m3_internal.h"
#include "m3_linattn.h"

namespace m3 {
namespace {

constexpr int kThreads = 256, kRowsAhead = 8;

template <typename T>
__global__ void __launch_bounds__(kThreads)
lin_step_kernel(const LinStep p, int tiles, int tx) {
    __shared__ float s_q[256], s_k[256];
    __shared__ float4 s_o[kThreads];
    const int tid = threadIdx.x, ry = tid / tx, cx = tid - ry * tx, nry = kThreads / tx;
    const unsigned unit = blockIdx.x / tiles, tile = blockIdx.x - unit * tiles;
    const unsigned i = unit / p.H;
    const int h = static_cast<int>(unit - i * p.H);
    const int64_t st = p.slots ? p.slots[i] : i;
    T* y = static_cast<T*>(p.o) + i * p.o_batch + h * p.o_head;
    const int col = 4 * (static_cast<int>(tile) * tx + cx);
    const bool on = ry < nry && col < p.V;          // V % 4 == 0 (see the launch)
    if (st < 0 || st >= p.nstates) {                // no state: the row is zero
        if (on && ry == 0)
            for (int e = 0; e < 4; ++e) y[col + e] = from_f<T>(0.f);
        return;
    }
    const T* q = static_cast<const T*>(p.q.p) + i * p.q.batch + (h / p.q.ratio) * p.q.head;
    const T* k = static_cast<const T*>(p.k.p) + i * p.k.batch + (h / p.k.ratio) * p.k.head;
    const T* v = static_cast<const T*>(p.v.p) + i * p.v.batch + (h / p.v.ratio) * p.v.head;
    const int64_t base = (st * p.H + h) * p.K * static_cast<int64_t>(p.V) + col;
    const float4* src = reinterpret_cast<const float4*>(p.state_in + base);
    float4* dst = reinterpret_cast<float4*>(p.state_out + base);
    const int row4 = p.V / 4;
    const bool has = p.state_in != nullptr, keep = p.state_out != nullptr;     // a prompt of one token may lack them
    float4 vv = make_float4(0.f, 0.f, 0.f, 0.f), o = vv;
    float4 ahead[kRowsAhead];
    // the state's first rows are on their way before anything else is waited for
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
        const int r = ry + u * nry;
        ahead[u] = (on && has && r < p.K) ? __ldcs(src + r * row4) : vv;
    }
    const float a = expf(p.log_decay[h]);
    for (int d = tid; d < p.K; d += kThreads) {
        s_q[d] = to_f(q[d]);
        s_k[d] = to_f(k[d]);
    }
    if (on) vv = make_float4(to_f(v[col]), to_f(v[col + 1]), to_f(v[col + 2]), to_f(v[col + 3]));
    __syncthreads();
    for (int r0 = ry; r0 < p.K; r0 += kRowsAhead * nry) {
        if (r0 != ry) {
#pragma unroll
            for (int u = 0; u < kRowsAhead; ++u) {
                const int r = r0 + u * nry;
                if (on && has && r < p.K) ahead[u] = __ldcs(src + r * row4);
            }
        }
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u) {
            const int r = r0 + u * nry;
            if (on && r < p.K) {
                const float kr = s_k[r], qr = s_q[r];
                float4 s = ahead[u];
                s.x = fmaf(a, s.x, kr * vv.x); s.y = fmaf(a, s.y, kr * vv.y);
                s.z = fmaf(a, s.z, kr * vv.z); s.w = fmaf(a, s.w, kr * vv.w);
                if (keep) __stcs(dst + r * row4, s);
                o.x = fmaf(qr, s.x, o.x); o.y = fmaf(qr, s.y, o.y);
                o.z = fmaf(qr, s.z, o.z); o.w = fmaf(qr, s.w, o.w);
            }
        }
    }
    s_o[tid] = o;
    // the row groups' sums, the upper half onto the lower until one is left
#pragma unroll 1
    for (int n = nry; n > 1; n = (n + 1) / 2) {
        const int half = (n + 1) / 2;
        __syncthreads();
        if (ry < n - half) {
            const float4 b = s_o[tid + half * tx];
            o.x += b.x; o.y += b.y; o.z += b.z; o.w += b.w;
            s_o[tid] = o;
        }
    }
    if (ry == 0 && on) {
        y[col] = from_f<T>(p.scale * o.x); y[col + 1] = from_f<T>(p.scale * o.y);
        y[col + 2] = from_f<T>(p.scale * o.z); y[col + 3] = from_f<T>(p.scale * o.w);
    }
}

// V not a multiple of 4: one thread per column, rows in turn.
template <typename T>
__global__ void __launch_bounds__(kThreads) lin_step_any_kernel(const LinStep p) {
    __shared__ float s_q[256], s_k[256];
    const int tid = threadIdx.x;
    const int64_t unit = blockIdx.x, i = unit / p.H;
    const int h = static_cast<int>(unit - i * p.H);
    const int64_t st = p.slots ? p.slots[i] : i;
    T* y = static_cast<T*>(p.o) + i * p.o_batch + h * p.o_head;
    if (st < 0 || st >= p.nstates) {        // no state: the row is zero
        if (tid < p.V) y[tid] = from_f<T>(0.f);
        return;
    }
    const T* q = static_cast<const T*>(p.q.p) + i * p.q.batch + (h / p.q.ratio) * p.q.head;
    const T* k = static_cast<const T*>(p.k.p) + i * p.k.batch + (h / p.k.ratio) * p.k.head;
    const T* v = static_cast<const T*>(p.v.p) + i * p.v.batch + (h / p.v.ratio) * p.v.head;
    for (int d = tid; d < p.K; d += kThreads) {
        s_q[d] = to_f(q[d]);
        s_k[d] = to_f(k[d]);
    }
    __syncthreads();
    if (tid >= p.V) return;
    const float a = expf(p.log_decay[h]), vv = to_f(v[tid]);
    const int64_t base = (st * p.H + h) * p.K * static_cast<int64_t>(p.V) + tid;
    float o = 0.f;
    for (int r = 0; r < p.K; ++r) {
        const int64_t at = base + static_cast<int64_t>(r) * p.V;
        const float s = fmaf(a, p.state_in ? p.state_in[at] : 0.f, s_k[r] * vv);
        if (p.state_out) p.state_out[at] = s;
        o = fmaf(s_q[r], s, o);
    }
    y[tid] = from_f<T>(p.scale * o);
}

// Prompts of 2 to 8 tokens (V % 4 == 0): the state is read once into registers, R float4 a thread, the
// tokens follow one another on it, and it is written once. q, k and v of all tokens lie in shared memory;
// the row groups' shares of four tokens' outputs meet there and are added in order.
constexpr int kShort = 8, kAtOnce = 4;
static_assert(kShort == kLinShort);
template <typename T, int R>
__global__ void __launch_bounds__(kThreads)
lin_short_kernel(const LinStep p, int tiles, int tx) {
    __shared__ float s_q[kShort * 256], s_k[kShort * 256];
    __shared__ __align__(16) float s_v[kShort][64];
    __shared__ __align__(16) float s_o[kAtOnce][4 * kThreads];
    const int tid = threadIdx.x, ry = tid / tx, cx = tid - ry * tx, nry = kThreads / tx;
    const unsigned unit = blockIdx.x / tiles, tile = blockIdx.x - unit * tiles;
    const unsigned i = unit / p.H;
    const int h = static_cast<int>(unit - i * p.H);
    const int col0 = 4 * static_cast<int>(tile) * tx, col = col0 + 4 * cx, width = min(4 * tx, p.V - col0);
    const bool on = ry < nry && col < p.V, has = p.state_in != nullptr;
    const int64_t base = (static_cast<int64_t>(i) * p.H + h) * p.K * static_cast<int64_t>(p.V) + col;
    const int row4 = p.V / 4;
    float4 st[R];
#pragma unroll
    for (int u = 0; u < R; ++u) {
        const int r = ry + u * nry;
        st[u] = (on && has && r < p.K) ? __ldcs(reinterpret_cast<const float4*>(p.state_in + base) + r * row4)
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float a = expf(p.log_decay[h]);
    const T* q = static_cast<const T*>(p.q.p) + i * p.q.batch + (h / p.q.ratio) * p.q.head;
    const T* k = static_cast<const T*>(p.k.p) + i * p.k.batch + (h / p.k.ratio) * p.k.head;
    const T* v = static_cast<const T*>(p.v.p) + i * p.v.batch + (h / p.v.ratio) * p.v.head + col0;
    for (int t = 0; t < p.L; ++t) {
        if (tid < p.K) {
            s_q[t * 256 + tid] = to_f(q[t * p.q.token + tid]);
            s_k[t * 256 + tid] = to_f(k[t * p.k.token + tid]);
        }
        if (tid < width) s_v[t][tid] = to_f(v[t * p.v.token + tid]);
    }
    __syncthreads();
    T* y = static_cast<T*>(p.o) + i * p.o_batch + h * p.o_head + col0;
    for (int t0 = 0; t0 < p.L; t0 += kAtOnce) {
#pragma unroll 1
        for (int t = t0; t < t0 + kAtOnce && t < p.L; ++t) {
            if (!on) continue;
            const float4 vv = *reinterpret_cast<const float4*>(&s_v[t][4 * cx]);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int u = 0; u < R; ++u) {
                const int r = ry + u * nry;
                if (r >= p.K) break;
                const float kr = s_k[t * 256 + r], qr = s_q[t * 256 + r];
                float4& s = st[u];
                s.x = fmaf(a, s.x, kr * vv.x); s.y = fmaf(a, s.y, kr * vv.y);
                s.z = fmaf(a, s.z, kr * vv.z); s.w = fmaf(a, s.w, kr * vv.w);
                o.x = fmaf(qr, s.x, o.x); o.y = fmaf(qr, s.y, o.y);
                o.z = fmaf(qr, s.z, o.z); o.w = fmaf(qr, s.w, o.w);
            }
            *reinterpret_cast<float4*>(&s_o[t - t0][4 * (ry * tx + cx)]) = o;
        }
        __syncthreads();
        const int t = tid / (4 * tx), c = tid - t * 4 * tx;     // 4 tx <= 64 columns of up to four tokens
        if (t < kAtOnce && t0 + t < p.L && c < width) {
            float sum = 0.f;
            for (int g = 0; g < nry; ++g) sum += s_o[t][g * 4 * tx + c];
            y[(t0 + t) * p.o_token + c] = from_f<T>(p.scale * sum);
        }
        __syncthreads();
    }
    if (!p.state_out) return;
#pragma unroll
    for (int u = 0; u < R; ++u) {
        const int r = ry + u * nry;
        if (on && r < p.K) __stcs(reinterpret_cast<float4*>(p.state_out + base) + r * row4, st[u]);
    }
}

template <typename T>
cudaError_t launch_short_t(const LinStep& p, cudaStream_t s) {
    // at most 16 float4 of columns a CTA (so 16 float4 of rows a thread at K = 256), fewer while CTA slots are empty
    const int64_t units = p.nseq * p.H;
    const int c4 = p.V / 4;
    int tiles = (c4 + 15) / 16;
    while (units * tiles < 2 * device_sm_count() && c4 >= 8 * tiles) tiles *= 2;
    const int tx = (c4 + tiles - 1) / tiles, rows = (p.K + kThreads / tx - 1) / (kThreads / tx);
    const unsigned grid = static_cast<unsigned>(units * tiles);
    if (rows <= 4) lin_short_kernel<T, 4><<<grid, kThreads, 0, s>>>(p, tiles, tx);
    else if (rows <= 8) lin_short_kernel<T, 8><<<grid, kThreads, 0, s>>>(p, tiles, tx);
    else lin_short_kernel<T, 16><<<grid, kThreads, 0, s>>>(p, tiles, tx);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const LinStep& p, cudaStream_t s) {
    if (p.L > 1) return launch_short_t<T>(p, s);
    const int64_t units = p.nseq * p.H;
    if (p.V % 4 != 0) {
        lin_step_any_kernel<T><<<static_cast<unsigned>(units), kThreads, 0, s>>>(p);
        return cudaGetLastError();
    }
    // columns of a head in parts while heads leave CTA slots empty, of 4 float4 at least
    const int c4 = p.V / 4;
    int tiles = 1;
    while (units * tiles < 2 * device_sm_count() && c4 >= 8 * tiles) tiles *= 2;
    const int tx = (c4 + tiles - 1) / tiles;
    lin_step_kernel<T><<<static_cast<unsigned>(units * tiles), kThreads, 0, s>>>(p, tiles, tx);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_step(const LinStep& p, bool bf16, cudaStream_t s) {
    return bf16 ? launch_t<__nv_bfloat16>(p, s) : launch_t<float>(p, s);
}

}  // namespace m3
