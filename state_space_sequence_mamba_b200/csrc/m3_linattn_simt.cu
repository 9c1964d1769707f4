// Linear attention's pass on the CUDA cores in fp32: every type, size, stride and alignment the
// tensor-core form does not take.
//
// One CTA per (sequence, segment, head, 64-column tile of v); chunks of C tokens staged in shared
// memory as fp32. Per chunk of n tokens (i, j: positions in processing order's own direction)
//     P = (q k^T) masked by p_scale a^{|i - j|},  y = P v + o_scale a^{e(i)} q H,
//     H <- a^n H + sum_j x_scale a^{w(j)} k_j v_j^T,
// as register-tiled products of 256 threads (4 x 4 outputs a thread, operands read as float4; q k^T
// and q H share one sweep over q). With C = 64 a token and head cost 2 (64 Dk + 64 64 + 2 Dk 64)
// flops, so a chunk is bound by instruction issue, not by DRAM: the products are packed pairs of FMAs,
// and blocks above the mask's diagonal are left out. In reverse a chunk's tokens are staged last to
// first, which makes it a forward one. Rows are not padded but swizzled, and P takes q's place, so
// that two CTAs of Dk = 128 fit an SM (112 KB each). 4096 tokens of 16 heads, K 128, V 64, fp32: 182 us,
// 21 TFLOP/s, with an instruction issued in 64 % of the cycles and the FMA pipe busy in 37 %; the rest is
// waiting at the barriers between a chunk's products, which two CTAs an SM do not fill.
#include "m3_common.cuh"
#include "m3_internal.h"
#include "m3_linattn.h"
#include "m3_sm100.cuh"

namespace m3 {
namespace {

constexpr int kThreads = 256, kVT = kLinTile;

struct SimtSmem {
    int Dp;          // Dk padded to 16 or a multiple of 32
    int mask;        // of the swizzle of k's rows: within 16 or 32 columns
    int q, k, v, h, pw, bytes;
};
__host__ __device__ inline SimtSmem simt_smem(int Dk, int C) {
    SimtSmem s;
    s.Dp = Dk <= 16 ? 16 : (Dk + 31) / 32 * 32;
    s.mask = s.Dp == 16 ? 12 : 28;
    s.q = 0;                                            // q, then P [C][C]
    s.k = s.q + C * (s.Dp > C ? s.Dp : C);
    s.v = s.k + C * s.Dp;
    s.h = s.v + C * kVT;
    s.pw = s.h + s.Dp * kVT;
    s.bytes = (s.pw + C + 4) * 4;
    return s;
}
// Column c of row r, swizzled in fours: the rows that a warp reads at once (16 neighbours of k, 2 of q
// and P) start in different banks.
__device__ __forceinline__ int swz_k(int r, int c, int mask) { return c ^ ((r << 2) & mask); }
__device__ __forceinline__ int swz_q(int r, int c) { return c ^ ((r & 1) << 2); }

// pairs of products: c += a b in one instruction
__device__ __forceinline__ void fma2(float2& c, const float2& a, const float2& b) { c = __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 lo2(const float4& v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi2(const float4& v) { return make_float2(v.z, v.w); }
__device__ __forceinline__ float2 dup(float v) { return make_float2(v, v); }
// four columns as two pairs += s times four columns
struct Four {
    float2 a, b;
    __device__ __forceinline__ void add(float s, const float4& v) {
        const float2 d = dup(s);
        fma2(a, d, lo2(v));
        fma2(b, d, hi2(v));
    }
};

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
__global__ void __launch_bounds__(kThreads, 2)
lin_simt_kernel(const __grid_constant__ LinParams p) {
    constexpr int RI = C / 16;      // rows a thread owns in the S and y products
    extern __shared__ __align__(16) float sm[];
    __shared__ volatile int odd_chunk;      // 1 + the last chunk whose v is not all finite
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
    const int64_t seg_end = lin_seg_end(p, w, seg0);
    const int order = j.reverse ? w.nseg - 1 - w.seg : w.seg;
    if (kStateOnly && order == w.nseg - 1) return;    // nobody reads the last one's

    const SimtSmem L = simt_smem(j.Dk, C);
    float *sq = sm + L.q, *sk = sm + L.k, *sv = sm + L.v, *sp = sq, *sh = sm + L.h, *pw = sm + L.pw;
    const float g2 = p.log_decay[h] * 1.4426950408889634f;
    if (tid == 0) odd_chunk = 0;
    for (int i = tid; i <= C; i += kThreads) pw[i] = lin_pow(g2, static_cast<float>(i));
    const bool blank = kStateOnly || (order == 0 && !j.init);      // no state before this segment
    if (kStateOnly) sm100::grid_dep_launch_dependents();
    else if (order > 0) sm100::grid_dep_wait();         // the segments' end states are there
    if (blank) {
        for (int e = tid; e < L.Dp * (kVT / 4); e += kThreads) reinterpret_cast<float4*>(sh)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
        // the given state and the segments before, decayed: eight float4 a thread and sweep
        const int before = static_cast<int>(j.reverse ? (order == 0 ? 0 : w.len - (seg0 + p.seg_len)) : seg0);
        const float fi = lin_pow(g2, static_cast<float>(j.reverse && before > 0 ? before - 1 : before));
        const int64_t unit = static_cast<int64_t>(w.seq) * p.H + h;
#pragma unroll 1
        for (int e0 = tid; e0 < L.Dp * (kVT / 4); e0 += 8 * kThreads) {
            float4 acc[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j.init && fi != 0.f) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = e0 + i * kThreads, r = e / (kVT / 4), c = tile * kVT + e % (kVT / 4) * 4;
                    if (r >= j.Dk) continue;
                    const float* src = j.init + unit * j.Dk * j.Dv + r * j.init_k + c * j.init_v;
                    if (c < j.Dv) acc[i].x = fi * src[0];
                    if (c + 1 < j.Dv) acc[i].y = fi * src[j.init_v];
                    if (c + 2 < j.Dv) acc[i].z = fi * src[2 * j.init_v];
                    if (c + 3 < j.Dv) acc[i].w = fi * src[3 * j.init_v];
                }
            }
#pragma unroll 1
            for (int o = 0; o < order; ++o) {
                const int sg = j.reverse ? w.nseg - 1 - o : o;
                const int64_t gap = j.reverse ? static_cast<int64_t>(sg) * p.seg_len - (seg0 + p.seg_len)
                                              : seg0 - static_cast<int64_t>(sg + 1) * p.seg_len;
                const float f = lin_pow(g2, static_cast<float>(gap));
                if (f == 0.f) continue;
                const float4* src = reinterpret_cast<const float4*>(
                    p.seg + ((static_cast<int64_t>(x - w.seg + sg) * p.H + h) * p.rtiles + rt) * p.seg_rows * kVT);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = e0 + i * kThreads;
                    if (e < j.Dk * (kVT / 4)) fma4(acc[i], f, __ldcg(src + e));
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = e0 + i * kThreads;
                if (e < L.Dp * (kVT / 4)) reinterpret_cast<float4*>(sh)[e] = acc[i];
            }
        }
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
    for (int cc = 0; cc < nchunks; ++cc) {
        const int c = j.reverse ? nchunks - 1 - cc : cc;
        const int64_t t0 = seg0 + static_cast<int64_t>(c) * C;
        const int n = seg_end - t0 < C ? static_cast<int>(seg_end - t0) : C;
        // in reverse the given state meets the sequence's last token undecayed
        const int off = (j.reverse && order == 0 && cc == 0) ? 1 : 0;
        __syncthreads();
        // q, k and v rows as fp32, zeros behind the last token and column: 16 threads side by side, four
        // elements each, every load of a sweep issued before the first is stored
        float odd = 0.f;            // stays zero while v is finite
#pragma unroll 1
        for (int c = 4 * tx; c < L.Dp || c < kVT; c += 64) {
            float4 fq[RI], fk[RI], fv[RI];
#pragma unroll
            for (int a = 0; a < RI; ++a) {
                const int r = ty + 16 * a;
                const int64_t t = t0 + (j.reverse ? n - 1 - r : r);
                fq[a] = fk[a] = fv[a] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < n) {
                    if (!kStateOnly && c < j.Dk) fq[a] = fetch4(q + t * j.q.token, c, j.Dk, vq);
                    if (c < j.Dk) fk[a] = fetch4(k + t * j.k.token, c, j.Dk, vk);
                    if (c < vdim) fv[a] = fetch4(v + t * j.v.token, c, vdim, vv4);
                }
            }
#pragma unroll
            for (int a = 0; a < RI; ++a) {
                const int r = ty + 16 * a;
                if (c < L.Dp) {
                    if (!kStateOnly) *reinterpret_cast<float4*>(sq + r * L.Dp + swz_q(r, c)) = fq[a];
                    *reinterpret_cast<float4*>(sk + r * L.Dp + swz_k(r, c, L.mask)) = fk[a];
                }
                if (c < kVT) {
                    *reinterpret_cast<float4*>(sv + r * kVT + c) = fv[a];
                    if (!kStateOnly) odd = fmaf(0.f, (fv[a].x + fv[a].y) + (fv[a].z + fv[a].w), odd);
                }
            }
        }
        if (!kStateOnly && odd != 0.f) odd_chunk = cc + 1;
        __syncthreads();
        if (!kStateOnly) {
            // s[a][b]: rows ty + 16 a, columns tx + 16 b, the sums of even and odd d apart; b > a is masked
            float2 s[RI][RI];
            Four yh[RI];
#pragma unroll
            for (int a = 0; a < RI; ++a) {
                yh[a].a = yh[a].b = dup(0.f);
#pragma unroll
                for (int b = 0; b < RI; ++b) s[a][b] = dup(0.f);
            }
            const float *qr = sq + ty * L.Dp, *kr = sk + tx * L.Dp, *hr = sh + 4 * tx;
            const bool fresh = blank && cc == 0;        // no state to read yet
            const int xq = swz_q(ty, 0), xk = swz_k(tx, 0, L.mask);
#pragma unroll 1
            for (int d = 0; d < L.Dp; d += 4) {
                float4 qa[RI], kb[RI];
#pragma unroll
                for (int a = 0; a < RI; ++a) qa[a] = *reinterpret_cast<const float4*>(qr + 16 * a * L.Dp + (d ^ xq));
#pragma unroll
                for (int b = 0; b < RI; ++b) kb[b] = *reinterpret_cast<const float4*>(kr + 16 * b * L.Dp + (d ^ xk));
#pragma unroll
                for (int a = 0; a < RI; ++a)
#pragma unroll
                    for (int b = 0; b <= a; ++b) {
                        fma2(s[a][b], lo2(qa[a]), lo2(kb[b]));
                        fma2(s[a][b], hi2(qa[a]), hi2(kb[b]));
                    }
                if (fresh) continue;
                float4 hh[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) hh[u] = *reinterpret_cast<const float4*>(hr + (d + u) * kVT);
#pragma unroll
                for (int a = 0; a < RI; ++a) {
                    yh[a].add(qa[a].x, hh[0]); yh[a].add(qa[a].y, hh[1]);
                    yh[a].add(qa[a].z, hh[2]); yh[a].add(qa[a].w, hh[3]);
                }
            }
            __syncthreads();        // q has been read: P takes its place
#pragma unroll
            for (int a = 0; a < RI; ++a)
#pragma unroll
                for (int b = 0; b <= a; ++b) {
                    // (rows behind the last token are zeros)
                    const int i = ty + 16 * a, jj = tx + 16 * b, d = i - jj;
                    sp[i * C + swz_q(i, jj)] = d >= 0 ? (s[a][b].x + s[a][b].y) * (j.p_scale * pw[d]) : 0.f;
                }
            __syncthreads();
#pragma unroll
            for (int a = 0; a < RI; ++a) {
                const float2 f = dup(j.o_scale * pw[ty + 16 * a + 1 - off]);
                yh[a].a = __fmul2_rn(yh[a].a, f);
                yh[a].b = __fmul2_rn(yh[a].b, f);
            }
            const float *pr = sp + ty * C, *vr = sv + 4 * tx;
            const bool all_finite = odd_chunk != cc + 1;
            if (!all_finite) {
                // zero times what is not finite is NaN: every row over the tokens up to its own alone
#pragma unroll 1
                for (int jj = 0; jj < n; ++jj) {
                    const float4 vv = *reinterpret_cast<const float4*>(vr + jj * kVT);
#pragma unroll
                    for (int a = 0; a < RI; ++a)
                        if (jj <= ty + 16 * a) yh[a].add(pr[16 * a * C + (jj ^ xq)], vv);
                }
            }
            // columns [16 b, 16 b + 16) reach rows from 16 b on
#pragma unroll
            for (int b = 0; b < RI; ++b) {
                if (16 * b >= n || !all_finite) break;
#pragma unroll 2
                for (int jj = 16 * b; jj < 16 * b + 16; jj += 4) {
                    float4 vv[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) vv[u] = *reinterpret_cast<const float4*>(vr + (jj + u) * kVT);
#pragma unroll
                    for (int a = b; a < RI; ++a) {
                        const float4 pp = *reinterpret_cast<const float4*>(pr + 16 * a * C + (jj ^ xq));
                        yh[a].add(pp.x, vv[0]); yh[a].add(pp.y, vv[1]);
                        yh[a].add(pp.z, vv[2]); yh[a].add(pp.w, vv[3]);
                    }
                }
            }
#pragma unroll
            for (int a = 0; a < RI; ++a) {
                const int i = ty + 16 * a;
                if (i >= n) continue;
                const float o[4] = {yh[a].a.x, yh[a].a.y, yh[a].b.x, yh[a].b.y};
                const int64_t at = y0 + (t0 + (j.reverse ? n - 1 - i : i)) * j.y_token + 4 * tx;
                if (j.y_f32) store4(static_cast<float*>(j.y) + at, o, vdim - 4 * tx, yv);
                else store4(static_cast<T*>(j.y) + at, o, vdim - 4 * tx, yv);
            }
        }
        // the last chunk's update only for a state that somebody wants
        if (!kStateOnly && cc + 1 == nchunks && !(j.final_state && order == w.nseg - 1)) break;
        const float hd = pw[n - off];
        if (C == 64 && L.Dp <= 32) {    // (P holds 64 rows of 64: parts x Dp)
            // Rows for a part of the threads only: the others take parts of the chunk's tokens, whose sums
            // meet in P's place and are added in order (one chunk of K 16: 11.8 -> 9.0 us a call).
            const int rows = L.Dp / 4, part = ty / rows, parts = 16 / rows, r0 = 4 * (ty - part * rows);
            float2 acc[2][4];
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[0][c] = acc[1][c] = dup(0.f);
#pragma unroll 4
            for (int i = part; i < n; i += parts) {
                const float wt = j.x_scale * pw[n - 1 - i];
                const float4 ka = *reinterpret_cast<const float4*>(sk + i * L.Dp + swz_k(i, r0, L.mask));
                const float4 vv = *reinterpret_cast<const float4*>(sv + i * kVT + 4 * tx);
                const float2 w[4] = {dup(vv.x * wt), dup(vv.y * wt), dup(vv.z * wt), dup(vv.w * wt)};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    fma2(acc[0][c], lo2(ka), w[c]);
                    fma2(acc[1][c], hi2(ka), w[c]);
                }
            }
            __syncthreads();        // P has been read
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float2* r = acc[u >> 1];
                const bool odd = u & 1;
                *reinterpret_cast<float4*>(sp + (part * L.Dp + r0 + u) * kVT + 4 * tx) =
                    make_float4(odd ? r[0].y : r[0].x, odd ? r[1].y : r[1].x, odd ? r[2].y : r[2].x, odd ? r[3].y : r[3].x);
            }
            __syncthreads();
            for (int e = tid; e < L.Dp * (kVT / 4); e += kThreads) {
                float4* at = reinterpret_cast<float4*>(sh) + e;
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int a = 0; a < parts; ++a) fma4(sum, 1.f, reinterpret_cast<const float4*>(sp)[a * L.Dp * (kVT / 4) + e]);
                fma4(sum, hd, *at);
                *at = sum;
            }
            continue;
        }
#pragma unroll 1
        for (int k0 = 4 * ty; k0 < L.Dp; k0 += 128) {       // two blocks of 64 rows at a time
            const bool two = k0 + 64 < L.Dp;
            // acc[u][c]: rows k0 + 2 u, 2 u + 1 (from u = 2 on those of the other block) of column 4 tx + c
            float2 acc[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[u][c] = dup(0.f);
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float wt = j.x_scale * pw[n - 1 - i];
                const float* kr = sk + i * L.Dp;
                const float4 ka = *reinterpret_cast<const float4*>(kr + swz_k(i, k0, L.mask));
                const float4 vv = *reinterpret_cast<const float4*>(sv + i * kVT + 4 * tx);
                const float2 w[4] = {dup(vv.x * wt), dup(vv.y * wt), dup(vv.z * wt), dup(vv.w * wt)};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    fma2(acc[0][c], lo2(ka), w[c]);
                    fma2(acc[1][c], hi2(ka), w[c]);
                }
                if (two) {
                    const float4 kb = *reinterpret_cast<const float4*>(kr + swz_k(i, k0 + 64, L.mask));
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        fma2(acc[2][c], lo2(kb), w[c]);
                        fma2(acc[3][c], hi2(kb), w[c]);
                    }
                }
            }
            // (every thread owns its rows' columns, and what read the state is behind the last barrier)
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (u >= 4 && !two) break;
                float4* at = reinterpret_cast<float4*>(sh + (k0 + (u & 3) + (u >= 4 ? 64 : 0)) * kVT + 4 * tx);
                float4 hv = *at;
                const float2* r = acc[u >> 1];
                const bool odd = u & 1;
                hv.x = fmaf(hd, hv.x, odd ? r[0].y : r[0].x); hv.y = fmaf(hd, hv.y, odd ? r[1].y : r[1].x);
                hv.z = fmaf(hd, hv.z, odd ? r[2].y : r[2].x); hv.w = fmaf(hd, hv.w, odd ? r[3].y : r[3].x);
                *at = hv;
            }
        }
    }
    if (!kStateOnly && tid == 0) sm100::grid_dep_wait();    // no CTA ends before the launch before it
    __syncthreads();
    if (kStateOnly) {
        float* e = p.seg + ((static_cast<int64_t>(x) * p.H + h) * p.rtiles + rt) * p.seg_rows * kVT;
        for (int i = tid; i < j.Dk * kVT; i += kThreads) e[i] = sh[i];
        return;
    }
    if (j.final_state && order == w.nseg - 1) {
        const int64_t unit = static_cast<int64_t>(w.seq) * p.H + h;
        float* dst = j.final_state + unit * j.Dk * j.Dv + tile * kVT;
        const float f = (j.reverse && w.len > 0) ? pw[1] : 1.f;
        for (int i = tid; i < j.Dk * kVT; i += kThreads) {
            const int r = i / kVT, c = i % kVT;
            if (c < vdim) dst[static_cast<int64_t>(r) * j.Dv + c] = f * sh[i];
        }
    }
}

template <typename T, int C>
cudaError_t launch_t(const LinParams& p, int Dk, bool cut, cudaStream_t s) {
    static std::atomic<uint64_t> done_state{0}, done{0};
    const int most = simt_smem(C == 64 ? 128 : 256, C).bytes, bytes = simt_smem(Dk, C).bytes;
    const unsigned grid = static_cast<unsigned>(p.blocks_x * p.H * p.rtiles);
    cudaError_t e = allow_smem(lin_simt_kernel<T, C, false>, most, done);
    if (e != cudaSuccess) return e;
    if (!cut) {
        lin_simt_kernel<T, C, false><<<grid, kThreads, bytes, s>>>(p);
        return cudaGetLastError();
    }
    if ((e = allow_smem(lin_simt_kernel<T, C, true>, most, done_state)) != cudaSuccess) return e;
    lin_simt_kernel<T, C, true><<<grid, kThreads, bytes, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // may start while the end states' kernel runs; whoever reads them waits for it
    return launch_after_rms(lin_simt_kernel<T, C, false>, grid, kThreads, bytes, s, p);
}

}  // namespace

// What launch_lin_simt runs: chunks of 64 tokens and two CTAs an SM up to Dk = 128, then chunks of 32 and as
// many CTAs an SM as their shared memory leaves room for. (Planned as 64 and two throughout: 2048 tokens of 16
// heads, K 256, V 64, bf16 349 us against 337, 3 x 700 of 24 heads 779 against 617, 100 of 2 heads 76 against 34.)
LinForm lin_simt_form(int Dk, float unit) {
    if (Dk <= 128) return LinForm{2 * device_sm_count(), 64, 1, 0.5f, 0.4f, 0.05f, 1.f};
    const int fit = simt_smem(Dk, 32).bytes <= 113 * 1024 ? 2 : 1;
    return LinForm{fit * device_sm_count(), 32, 1, 0.8f, 0.5f, 0.1f, unit};
}

cudaError_t launch_lin_simt(const LinParams& p, bool bf16, bool cut, cudaStream_t s) {
    int Dk = 1;
    for (int i = 0; i < p.njobs; ++i) Dk = p.job[i].Dk > Dk ? p.job[i].Dk : Dk;
    // 64-token chunks need 208 KB at Dk = 256; there chunks of 32 (136 KB)
    if (Dk <= 128) return bf16 ? launch_t<__nv_bfloat16, 64>(p, Dk, cut, s) : launch_t<float, 64>(p, Dk, cut, s);
    return bf16 ? launch_t<__nv_bfloat16, 32>(p, Dk, cut, s) : launch_t<float, 32>(p, Dk, cut, s);
}

}  // namespace m3
