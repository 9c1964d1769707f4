// Linear attention's pass on the CUDA cores in fp32: every type, size, stride and alignment the
// tensor-core form does not take.
//
// One CTA per (sequence, segment, head, 64-column tile of v); chunks of C tokens staged in shared
// memory as fp32. Per chunk of n tokens (i, j: positions in processing order's own direction)
//     P = (q k^T) masked by p_scale a^{|i - j|},  y = P v + o_scale a^{e(i)} q H,
//     H <- a^n H + sum_j x_scale a^{w(j)} k_j v_j^T,
// all three as register-tiled products of 256 threads (4 x 4 outputs a thread and step, operands
// read as float4). With C = 64 a token and head cost 2 (64 Dk + 64 64 + 2 Dk 64) flops, so a
// chunk is bound by the FMA pipe and shared-memory reads, not by DRAM. Measured on b1 L4096 H16
// K128 V64 fp32: see the figures beside the launch.
#include "m3_common.cuh"
#include "m3_internal.h"
#include "m3_linattn.h"

namespace m3 {
namespace {

constexpr int kThreads = 256, kVT = kLinTile, kVS = kVT + 4;

struct SimtSmem {
    int Dp, qs;      // Dk padded to 8, its row stride
    int q, k, v, p, h, pw, bytes;
};
__host__ __device__ inline SimtSmem simt_smem(int Dk, int C) {
    SimtSmem s;
    s.Dp = (Dk + 7) / 8 * 8;
    s.qs = s.Dp + 4;             // 4 mod 8 floats: rows 16 lanes read start in different banks
    s.q = 0;
    s.k = s.q + C * s.qs;
    s.v = s.k + C * s.qs;
    s.p = s.v + C * kVS;
    s.h = s.p + C * (C + 4);
    s.pw = s.h + s.Dp * kVS;
    s.bytes = (s.pw + C + 4) * 4;
    return s;
}

__device__ __forceinline__ void fma4(float4& a, float s, const float4& b) {
    a.x = fmaf(s, b.x, a.x); a.y = fmaf(s, b.y, a.y);
    a.z = fmaf(s, b.z, a.z); a.w = fmaf(s, b.w, a.w);
}

// four consecutive elements as floats
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
}

// four elements of a row from column c on, zeros beyond its `dim` (vec: the row can be read in fours)
template <typename T>
__device__ __forceinline__ float4 fetch4(const T* row, int c, int dim, bool vec) {
    if (vec && c + 4 <= dim) return load4(row + c);
    float v[4];
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const float x = c + i < dim ? to_f(row[c + i]) : 0.f;
        v[0] = i == 0 ? x : v[0]; v[1] = i == 1 ? x : v[1];
        v[2] = i == 2 ? x : v[2]; v[3] = i == 3 ? x : v[3];
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}

// the first `left` of four elements (vec: the address takes all four at once)
__device__ __forceinline__ void put4(float* p, const float (&o)[4]) { *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]); }
__device__ __forceinline__ void put4(__nv_bfloat16* p, const float (&o)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(o[0], o[1]), b = __floats2bfloat162_rn(o[2], o[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&o)[4], int left, bool vec) {
    if (vec && left >= 4) {
        put4(p, o);
        return;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (u < left) p[u] = from_f<T>(o[u]);
}

template <typename T, int C, bool kStateOnly>
__global__ void __launch_bounds__(kThreads)
lin_simt_kernel(const __grid_constant__ LinParams p) {
    constexpr int RI = C / 16;      // rows a thread owns in the S and y products
    extern __shared__ __align__(16) float sm[];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const unsigned per_x = static_cast<unsigned>(p.H) * p.rtiles;
    const unsigned x = blockIdx.x / per_x;
    const int rem = static_cast<int>(blockIdx.x - x * per_x);
    const int h = rem / p.rtiles, rt = rem % p.rtiles;
    int ji = 0, tile = rt;
    while (ji + 1 < p.njobs && tile >= p.job[ji].tiles) tile -= p.job[ji++].tiles;
    const LinJob& j = p.job[ji];
    const LinWhere w = lin_locate(p, x);
    if (!w.valid) return;
    const int64_t seg0 = static_cast<int64_t>(w.seg) * p.seg_len;
    const int64_t seg_end = seg0 + p.seg_len < w.len ? seg0 + p.seg_len : w.len;
    const int order = j.reverse ? w.nseg - 1 - w.seg : w.seg;
    if (kStateOnly && order == w.nseg - 1) return;    // nobody reads the last one's

    const SimtSmem L = simt_smem(j.Dk, C);
    float *sq = sm + L.q, *sk = sm + L.k, *sv = sm + L.v, *sp = sm + L.p, *sh = sm + L.h, *pw = sm + L.pw;
    const float g2 = p.log_decay[h] * 1.4426950408889634f;
    for (int i = tid; i <= C; i += kThreads) pw[i] = lin_pow(g2, static_cast<float>(i));
    const bool blank = kStateOnly || (order == 0 && !j.init);      // no state before this segment
    for (int e = tid; e < L.Dp * kVT; e += kThreads) {
        const int r = e / kVT, c = e % kVT;
        sh[r * kVS + c] = blank || r >= j.Dk ? 0.f : lin_start_state(p, j, w, x, h, rt, tile, g2, r, c);
    }
    const T* q = static_cast<const T*>(j.q.p) + w.batch * j.q.batch + (h / j.q.ratio) * j.q.head + w.row0 * j.q.token;
    const T* k = static_cast<const T*>(j.k.p) + w.batch * j.k.batch + (h / j.k.ratio) * j.k.head + w.row0 * j.k.token;
    const T* v = static_cast<const T*>(j.v.p) + w.batch * j.v.batch + (h / j.v.ratio) * j.v.head + w.row0 * j.v.token +
                 tile * kVT;
    const int vdim = j.Dv - tile * kVT < kVT ? j.Dv - tile * kVT : kVT;
    auto fours = [](const T* base, int64_t token) {
        return ((reinterpret_cast<uintptr_t>(base) | static_cast<uintptr_t>(token * sizeof(T))) & (4 * sizeof(T) - 1)) == 0;
    };
    const bool vq = fours(q, j.q.token), vk = fours(k, j.k.token), vv4 = fours(v, j.v.token);
    const int64_t y0 = w.batch * j.y_batch + w.row0 * j.y_token + h * j.y_head + tile * kVT;
    const int es = j.y_f32 ? 4 : static_cast<int>(sizeof(T));
    const bool yv = ((reinterpret_cast<uintptr_t>(j.y) | static_cast<uintptr_t>(y0 * es) | static_cast<uintptr_t>(j.y_token * es)) &
                     (4 * es - 1)) == 0;
    const int64_t ntok = seg_end - seg0;
    const int nchunks = static_cast<int>((ntok + C - 1) / C);
    const int hrows = (L.Dp + 63) / 64;     // 64-row blocks of the state
    for (int cc = 0; cc < nchunks; ++cc) {
        const int c = j.reverse ? nchunks - 1 - cc : cc;
        const int64_t t0 = seg0 + static_cast<int64_t>(c) * C;
        const int n = seg_end - t0 < C ? static_cast<int>(seg_end - t0) : C;
        // in reverse the given state meets the sequence's last token undecayed
        const int off = (j.reverse && order == 0 && cc == 0) ? 1 : 0;
        __syncthreads();
        // q, k and v rows as fp32, zeros behind the last token and column: 16 threads side by side, four
        // elements each, every load of a sweep issued before the first is stored
#pragma unroll 1
        for (int c = 4 * tx; c < L.Dp || c < kVT; c += 64) {
            float4 fq[RI], fk[RI], fv[RI];
#pragma unroll
            for (int a = 0; a < RI; ++a) {
                const int r = ty + 16 * a;
                fq[a] = fk[a] = fv[a] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < n) {
                    if (!kStateOnly && c < j.Dk) fq[a] = fetch4(q + (t0 + r) * j.q.token, c, j.Dk, vq);
                    if (c < j.Dk) fk[a] = fetch4(k + (t0 + r) * j.k.token, c, j.Dk, vk);
                    if (c < vdim) fv[a] = fetch4(v + (t0 + r) * j.v.token, c, vdim, vv4);
                }
            }
#pragma unroll
            for (int a = 0; a < RI; ++a) {
                const int r = ty + 16 * a;
                if (c < L.Dp) {
                    if (!kStateOnly) *reinterpret_cast<float4*>(sq + r * L.qs + c) = fq[a];
                    *reinterpret_cast<float4*>(sk + r * L.qs + c) = fk[a];
                }
                if (c < kVT) *reinterpret_cast<float4*>(sv + r * kVS + c) = fv[a];
            }
        }
        __syncthreads();
        if (!kStateOnly) {
            float s[RI][RI];
#pragma unroll
            for (int a = 0; a < RI; ++a)
#pragma unroll
                for (int b = 0; b < RI; ++b) s[a][b] = 0.f;
#pragma unroll 1
            for (int d = 0; d < L.Dp; d += 4) {
                float4 qa[RI], kb[RI];
#pragma unroll
                for (int a = 0; a < RI; ++a) qa[a] = *reinterpret_cast<const float4*>(sq + (ty + 16 * a) * L.qs + d);
#pragma unroll
                for (int b = 0; b < RI; ++b) kb[b] = *reinterpret_cast<const float4*>(sk + (tx + 16 * b) * L.qs + d);
#pragma unroll
                for (int a = 0; a < RI; ++a)
#pragma unroll
                    for (int b = 0; b < RI; ++b) {
                        s[a][b] = fmaf(qa[a].x, kb[b].x, s[a][b]);
                        s[a][b] = fmaf(qa[a].y, kb[b].y, s[a][b]);
                        s[a][b] = fmaf(qa[a].z, kb[b].z, s[a][b]);
                        s[a][b] = fmaf(qa[a].w, kb[b].w, s[a][b]);
                    }
            }
#pragma unroll
            for (int a = 0; a < RI; ++a)
#pragma unroll
                for (int b = 0; b < RI; ++b) {
                    const int i = ty + 16 * a, jj = tx + 16 * b;
                    const int d = j.reverse ? jj - i : i - jj;
                    sp[i * (C + 4) + jj] = (d >= 0 && jj < n) ? s[a][b] * (j.p_scale * pw[d]) : 0.f;
                }
            __syncthreads();
            // columns of P that hold tokens; no state yet (a fresh sequence's first chunk): nothing to read
            const int nr = (n + 3) & ~3, hd4 = (cc == 0 && blank) ? 0 : L.Dp;
            float4 yi[RI], yh[RI];
#pragma unroll
            for (int a = 0; a < RI; ++a) yi[a] = yh[a] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int jj = 0; jj < nr; jj += 4) {
                float4 vv[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) vv[u] = *reinterpret_cast<const float4*>(sv + (jj + u) * kVS + 4 * tx);
#pragma unroll
                for (int a = 0; a < RI; ++a) {
                    const float4 pp = *reinterpret_cast<const float4*>(sp + (ty + 16 * a) * (C + 4) + jj);
                    fma4(yi[a], pp.x, vv[0]); fma4(yi[a], pp.y, vv[1]);
                    fma4(yi[a], pp.z, vv[2]); fma4(yi[a], pp.w, vv[3]);
                }
            }
#pragma unroll 1
            for (int d = 0; d < hd4; d += 4) {
                float4 hh[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) hh[u] = *reinterpret_cast<const float4*>(sh + (d + u) * kVS + 4 * tx);
#pragma unroll
                for (int a = 0; a < RI; ++a) {
                    const float4 qq = *reinterpret_cast<const float4*>(sq + (ty + 16 * a) * L.qs + d);
                    fma4(yh[a], qq.x, hh[0]); fma4(yh[a], qq.y, hh[1]);
                    fma4(yh[a], qq.z, hh[2]); fma4(yh[a], qq.w, hh[3]);
                }
            }
#pragma unroll
            for (int a = 0; a < RI; ++a) {
                const int i = ty + 16 * a;
                if (i >= n) continue;
                const float f = j.o_scale * pw[(j.reverse ? n - i : i + 1) - off];
                const float o[4] = {fmaf(f, yh[a].x, yi[a].x), fmaf(f, yh[a].y, yi[a].y),
                                    fmaf(f, yh[a].z, yi[a].z), fmaf(f, yh[a].w, yi[a].w)};
                const int64_t at = y0 + (t0 + i) * j.y_token + 4 * tx;
                if (j.y_f32) store4(static_cast<float*>(j.y) + at, o, vdim - 4 * tx, yv);
                else store4(static_cast<T*>(j.y) + at, o, vdim - 4 * tx, yv);
            }
            __syncthreads();     // the state has been read
        }
        // the last chunk's update only for a state that somebody wants
        if (!kStateOnly && cc + 1 == nchunks && !(j.final_state && order == w.nseg - 1)) break;
        const float hd = pw[n - off];
        for (int b = 0; b < hrows; ++b) {
            const int k0 = 64 * b + 4 * ty;
            if (k0 >= L.Dp) continue;
            float4 acc[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float wt = pw[j.reverse ? i : n - 1 - i];
                const float4 kk = *reinterpret_cast<const float4*>(sk + i * L.qs + k0);
                float4 vv = *reinterpret_cast<const float4*>(sv + i * kVS + 4 * tx);
                vv.x *= wt; vv.y *= wt; vv.z *= wt; vv.w *= wt;
                fma4(acc[0], kk.x, vv); fma4(acc[1], kk.y, vv);
                fma4(acc[2], kk.z, vv); fma4(acc[3], kk.w, vv);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float4* at = reinterpret_cast<float4*>(sh + (k0 + u) * kVS + 4 * tx);
                float4 hv = *at;
                hv.x = fmaf(hd, hv.x, j.x_scale * acc[u].x); hv.y = fmaf(hd, hv.y, j.x_scale * acc[u].y);
                hv.z = fmaf(hd, hv.z, j.x_scale * acc[u].z); hv.w = fmaf(hd, hv.w, j.x_scale * acc[u].w);
                *at = hv;
            }
        }
    }
    __syncthreads();
    if (kStateOnly) {
        float* e = p.seg + ((static_cast<int64_t>(x) * p.H + h) * p.rtiles + rt) * p.seg_rows * kVT;
        for (int i = tid; i < j.Dk * kVT; i += kThreads) e[i] = sh[(i / kVT) * kVS + i % kVT];
        return;
    }
    if (j.final_state && order == w.nseg - 1) {
        const int64_t unit = static_cast<int64_t>(w.seq) * p.H + h;
        float* dst = j.final_state + unit * j.Dk * j.Dv + tile * kVT;
        const float f = (j.reverse && w.len > 0) ? pw[1] : 1.f;
        for (int i = tid; i < j.Dk * kVT; i += kThreads) {
            const int r = i / kVT, c = i % kVT;
            if (c < vdim) dst[static_cast<int64_t>(r) * j.Dv + c] = f * sh[r * kVS + c];
        }
    }
}

template <typename T, int C, bool kStateOnly>
cudaError_t launch_one(const LinParams& p, int Dk, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    auto k = lin_simt_kernel<T, C, kStateOnly>;
    const cudaError_t e = allow_smem(k, simt_smem(C == 64 ? 128 : 256, C).bytes, done);
    if (e != cudaSuccess) return e;
    k<<<static_cast<unsigned>(p.blocks_x * p.H * p.rtiles), kThreads, simt_smem(Dk, C).bytes, s>>>(p);
    return cudaGetLastError();
}

template <typename T, int C>
cudaError_t launch_t(const LinParams& p, int Dk, bool cut, cudaStream_t s) {
    if (cut) {
        const cudaError_t e = launch_one<T, C, true>(p, Dk, s);
        if (e != cudaSuccess) return e;
    }
    return launch_one<T, C, false>(p, Dk, s);
}

}  // namespace

int lin_simt_slots() { return device_sm_count(); }

cudaError_t launch_lin_simt(const LinParams& p, bool bf16, bool cut, cudaStream_t s) {
    int Dk = 1;
    for (int i = 0; i < p.njobs; ++i) Dk = p.job[i].Dk > Dk ? p.job[i].Dk : Dk;
    // 64-token chunks need 222 KB at Dk = 256; there chunks of 32
    if (Dk <= 128) return bf16 ? launch_t<__nv_bfloat16, 64>(p, Dk, cut, s) : launch_t<float, 64>(p, Dk, cut, s);
    return bf16 ? launch_t<__nv_bfloat16, 32>(p, Dk, cut, s) : launch_t<float, 32>(p, Dk, cut, s);
}

}  // namespace m3
