// Gated linear recurrence of each channel, its single-token form and its gradients.
//
//     power:  log a_t = -power softplus(d) sig(r_t),  w_t = sqrt(1 - a_t^2)
//     lerp:   a_t = sig(r_t + d),                     w_t = 1 - a_t
//     h_t = a_t h_{t-1} + w_t u_t,  u_t = sig(i_t) x_t
// Bound by HBM: the forward reads x, r, i and writes y once, the backward reads those and dy and writes
// three gradients. Two tokens compose as (A, B) after (A', B') = (A A', A B' + B), so time is cut: a
// CTA takes a tile of 64 tokens by 32 words (a word: two bf16 channels or one of fp32), a thread eight
// tokens of one word. It reduces them to one (A, B) in registers, the warps' pairs are combined in order
// through shared memory, and each thread then finishes its eight tokens; the next tile's loads are in
// flight meanwhile. Where columns of channels are fewer than the device holds CTAs, the CTAs of a cluster
// take the tiles of a column in turn and exchange one pair per tile through each other's shared memory.
// Everything is added in a fixed order.
//
// Backward. With g_t = dL/dh_t and G_t = a_t g_t,
//     g_t = dy_t + G_{t+1},   dx = g w sig(i),   di = dx x (1 - sig(i)),
//     power:  l = log a:  l dL/dl = g (a l h_{t-1} - u a^2 l / w),  dr = (1 - sig(r)) l dL/dl,
//             dd = sum l dL/dl sig(d) / softplus(d)      (l / w -> 0 as l -> 0: no singularity is left)
//     lerp:   dr = g (h_{t-1} - u) a w,  dd = sum dr
// in tiles from the last one back. h_{t-1} comes from the forward's states before each tile (marks) and
// the same composition inside a tile, so nothing is read twice and h is not rounded.
#include <cooperative_groups.h>

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

constexpr int kWarps = 8, kTok = 8, kTile = kWarps * kTok, kThreads = 32 * kWarps;
constexpr int kMaxRanks = 8;
static_assert(kTile == M3_GS_BLOCK, "marks lie before every tile");

struct GsTensor {
    void* p;
    int64_t batch, token;       // strides in elements
};
struct GsParams {
    GsTensor x, r, i, y, dy, dx, dr, di;
    const float* decay;
    const int32_t* cu;
    const float* init;
    float* final_state;
    const float* dfinal;
    float* dinit;
    float* marks;               // [nb][tiles][C] or null
    float* part;                // backward: [shares][C]
    int64_t L;
    int64_t nb;                 // batch entries (packed: 1)
    int nseq, C, cols, ranks, tiles, shares;
    float power;
};

// ---- one word: two bf16 channels or one fp32 channel

template <typename T>
struct Word;
template <>
struct Word<__nv_bfloat16> {
    using V = float2;
    static constexpr int E = 2;
    static __device__ __forceinline__ V unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t pack(const V& v) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
        return *reinterpret_cast<const uint32_t*>(&b);
    }
};
template <>
struct Word<float> {
    using V = float;
    static constexpr int E = 1;
    static __device__ __forceinline__ V unpack(uint32_t w) { return __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t pack(V v) { return __float_as_uint(v); }
};

template <typename V>
__device__ __forceinline__ V splat(float v);
template <>
__device__ __forceinline__ float splat<float>(float v) { return v; }
template <>
__device__ __forceinline__ float2 splat<float2>(float v) { return make_float2(v, v); }
template <typename F>
__device__ __forceinline__ float each(float v, F&& f) { return f(v); }
template <typename F>
__device__ __forceinline__ float2 each(const float2& v, F&& f) { return make_float2(f(v.x), f(v.y)); }
template <typename V>
__device__ __forceinline__ V neg(const V& v) { return mul2(v, splat<V>(-1.f)); }

// The hardware's 2^x, 1 / x and 1 / sqrt(x); the bounds keep NaN.
__device__ __forceinline__ float hw_ex2(float v) { asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v)); return v; }
__device__ __forceinline__ float hw_rcp(float v) { asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(v)); return v; }
__device__ __forceinline__ float hw_rsqrt(float v) { asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(v)); return v; }
__device__ __forceinline__ float at_least(float v, float b) { asm("max.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(b)); return v; }

constexpr float kLog2e = 1.4426950408889634f;
// A gate is taken to be at least -43 (NaN stays): then (1 + e^-r)(1 + e^-i) is finite, and a sigmoid ends at 2^-62
// instead of at zero. For a pair of bf16 that is one instruction.
constexpr float kLeast = -43.f;
__device__ __forceinline__ float bounded(float, uint32_t w) { return at_least(__uint_as_float(w), kLeast); }
__device__ __forceinline__ float2 bounded(const float2&, uint32_t w) {
    uint32_t v;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(w), "r"(0xc22cc22cu));       // bf16 -43 twice
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <typename V>
__device__ __forceinline__ V exp_neg(const V& v) { return each(mul2(v, splat<V>(-kLog2e)), hw_ex2); }

// 1 - e^l: the series' up to kSeries, the other beyond
constexpr float kSeries = 0.35f;
__device__ __forceinline__ float beyond(float l, float m, float big) { return l < -kSeries ? big : m; }
__device__ __forceinline__ float2 beyond(const float2& l, const float2& m, const float2& big) {
    return make_float2(beyond(l.x, m.x, big.x), beyond(l.y, m.y, big.y));
}

// What one token does to its channels.
template <typename V>
struct Gates {
    V a, w;         // decay and weight of the input
    V si, ci;       // sig(i) and 1 - sig(i) (with an input gate)
    V cr;           // power: 1 - sig(r)
    V l, lw;        // power: log a and log a / w
};

// r, i: the gates' words. k: power: -power softplus(d), the largest |log a|; lerp: d. kSmall: |k| <= kSeries, the series
// of 1 - e^l alone serves (it holds for |l| <= kSeries: the next term is 0.35^8 / 8! = 6e-9); otherwise e^l from the
// hardware's 2^x where |l| is larger. 1 - a^2 = m (2 - m) with m = 1 - a: no digits are lost for a near 1. log a is
// taken 1e-30 lower, so that w is not zero where sig(r) is.
template <bool kLerp, bool kGate, bool kBack, bool kSmall, typename V>
__device__ __forceinline__ Gates<V> gates(uint32_t rw, uint32_t iw, const V& k) {
    Gates<V> g{};
    const V one = splat<V>(1.f);
    V er, sr;
    if (kLerp) er = exp_neg(each(add2(bounded(k, rw), k), [](float v) { return at_least(v, kLeast); }));
    else er = exp_neg(bounded(k, rw));
    if (kGate) {        // one reciprocal for both sigmoids
        const V ei = exp_neg(bounded(k, iw)), pr = add2(er, one), pi = add2(ei, one);
        const V R = each(mul2(pr, pi), hw_rcp);
        sr = mul2(pi, R);
        g.si = mul2(pr, R);
        if (kBack) g.ci = mul2(ei, g.si);
    } else {
        sr = each(add2(er, one), hw_rcp);
    }
    if (kLerp) {
        g.a = sr;
        g.w = mul2(er, sr);
        return g;
    }
    if (kBack) g.cr = mul2(er, sr);
    const V l = fma2(k, sr, splat<V>(-1e-30f));
    // -m = e^l - 1 = l (1 + l/2 (1 + l/3 (1 + ... l/7)))
    V s = fma2(l, splat<V>(1.f / 5040.f), splat<V>(1.f / 720.f));
    s = fma2(l, s, splat<V>(1.f / 120.f));
    s = fma2(l, s, splat<V>(1.f / 24.f));
    s = fma2(l, s, splat<V>(1.f / 6.f));
    s = fma2(l, s, splat<V>(0.5f));
    s = fma2(l, s, one);
    V m = mul2(l, s);
    if (!kSmall) {
        const V big = each(mul2(l, splat<V>(kLog2e)), [](float x) { return hw_ex2(x) - 1.f; });
        m = beyond(l, m, big);
    }
    g.a = add2(one, m);
    const V q = mul2(neg(m), add2(splat<V>(2.f), m)), rs = each(q, hw_rsqrt);
    g.w = mul2(q, rs);
    if (kBack) {
        g.l = l;
        g.lw = mul2(l, rs);
    }
    return g;
}

// softplus(d) = log(1 + e^d)
__device__ __forceinline__ float softplus(float d) { return d > 20.f ? d : log1pf(expf(d)); }

// ---- a thread's column

template <typename T, bool kVec>
struct Column {
    using W = Word<T>;
    using V = typename W::V;
    int c;              // first channel
    bool ok, two;       // the column exists; its second channel does
    __device__ __forceinline__ Column(const GsParams& p, int col) {
        c = (col * 32 + static_cast<int>(threadIdx.x & 31)) * W::E;
        ok = c < p.C;
        two = W::E == 2 && c + 1 < p.C;
    }
    __device__ __forceinline__ uint32_t load(const T* q, bool live) const {
        if (!live) return 0u;
        if constexpr (kVec) {
            return __ldcs(reinterpret_cast<const uint32_t*>(q));
        } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(q);
            return h[0] | (two ? static_cast<uint32_t>(h[1]) << 16 : 0u);
        }
    }
    __device__ __forceinline__ void store(T* q, const V& v) const {
        const uint32_t w = W::pack(v);
        if constexpr (kVec) {
            __stcs(reinterpret_cast<uint32_t*>(q), w);
        } else {
            uint16_t* h = reinterpret_cast<uint16_t*>(q);
            h[0] = static_cast<uint16_t>(w);
            if (two) h[1] = static_cast<uint16_t>(w >> 16);
        }
    }
    // the decay parameters, aligned to their elements
    __device__ __forceinline__ V param(const float* q) const {
        if (!q) return splat<V>(0.f);
        if constexpr (W::E == 1) return ok ? q[c] : 0.f;
        else return make_float2(ok ? q[c] : 0.f, two ? q[c + 1] : 0.f);
    }
    // fp32 values of this column (states, marks, sums); q points at the row
    __device__ __forceinline__ V get(const float* q) const {
        if constexpr (W::E == 1) return ok ? q[c] : 0.f;
        else if constexpr (kVec) return ok ? *reinterpret_cast<const float2*>(q + c) : make_float2(0.f, 0.f);
        else return make_float2(ok ? q[c] : 0.f, two ? q[c + 1] : 0.f);
    }
    __device__ __forceinline__ void put(float* q, const V& v) const {
        if (!ok) return;
        if constexpr (W::E == 1) {
            q[c] = v;
        } else if constexpr (kVec) {
            *reinterpret_cast<float2*>(q + c) = v;
        } else {
            q[c] = v.x;
            if (two) q[c + 1] = v.y;
        }
    }
};

template <typename T>
__device__ __forceinline__ T* at(const GsTensor& t, int64_t b, int c) { return static_cast<T*>(t.p) + b * t.batch + c; }

// Which of a tile's rows begin and end a sequence, and whose rows they are. Three of them: the next
// tile's is written while the slowest warp still reads the last one's.
struct Rows {
    uint32_t start[2], end[2];
    int seq[kTile];
};

// Rows of the packed tensor that hold tokens.
__device__ __forceinline__ void packed_span(const GsParams& p, int64_t* first, int64_t* last) {
    int64_t f = p.nseq > 0 ? __ldg(p.cu) : 0, l = p.nseq > 0 ? __ldg(p.cu + p.nseq) : 0;
    *first = f < 0 ? 0 : f > p.L ? p.L : f;
    *last = l < *first ? *first : l > p.L ? p.L : l;
}

// threads 0 to 63: the sequence of one row each, by halves (the last that begins at or before it)
__device__ __forceinline__ void find_rows(const GsParams& p, Rows& rows, int64_t tile, int64_t last) {
    const int64_t row = tile * kTile + threadIdx.x;
    int lo = 0, hi = p.nseq;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (__ldg(p.cu + m) <= row) lo = m;
        else hi = m;
    }
    const int64_t s = __ldg(p.cu + lo), e = __ldg(p.cu + lo + 1);
    const bool in = tile >= 0 && row < last && s <= row && row < e;
    const uint32_t st = __ballot_sync(0xffffffffu, in && s == row), en = __ballot_sync(0xffffffffu, in && e == row + 1);
    const int w = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
        rows.start[w] = st;
        rows.end[w] = en;
    }
    rows.seq[threadIdx.x] = lo;
}

// the eight rows of warp w
__device__ __forceinline__ uint32_t mine(const uint32_t (&m)[2], int w) { return (m[w >> 2] >> (8 * (w & 3))) & 0xffu; }

// a sequence without tokens ends in the state it begins with
template <typename Col>
__device__ __forceinline__ void empty_sequences(const GsParams& p, const Col& k, int rank, const float* from, float* to) {
    using V = typename Col::V;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t s0 = (static_cast<int64_t>(rank) * kWarps + warp) * 32; s0 < p.nseq; s0 += static_cast<int64_t>(p.ranks) * kWarps * 32) {
        const int64_t s = s0 + lane;
        unsigned hit = __ballot_sync(0xffffffffu, s < p.nseq && __ldg(p.cu + s + 1) <= __ldg(p.cu + s));
        while (hit) {
            const int64_t off = (s0 + __ffs(hit) - 1) * p.C;
            hit &= hit - 1;
            k.put(to + off, from ? k.get(from + off) : splat<V>(0.f));
        }
    }
}

template <typename V>
struct Pair {
    V a, b;
};

// Tiles of the input tensors. kStaged (rows of whole 16-byte words): rows of 128 bytes in shared memory, brought by
// asynchronous copies while other tiles are worked on; otherwise each thread's own words in its registers, a tile ahead.
constexpr int kRowBytes = 128, kTileBytes = kTile * kRowBytes;
template <typename T, bool kVec, bool kStaged, int kTensors>
struct Tiles {
    using Col = Column<T, kVec>;
    const T* base[kTensors];        // kStaged: of the batch entry; otherwise of this thread's column
    int64_t token[kTensors];
    uint32_t at[kTensors];          // kStaged: this thread's first 16 bytes of a tile
    uint32_t raw[kStaged ? 1 : kTensors][kStaged ? 1 : kTok];
    uint8_t* room;
    const Col& k;
    int chunk_bytes, warp, lane;
    __device__ __forceinline__ Tiles(const Col& col, int column, int C, uint8_t* smem) : room(smem), k(col) {
        warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        const int c = column * 32 * Word<T>::E + static_cast<int>(threadIdx.x & 7) * (16 / static_cast<int>(sizeof(T)));
        chunk_bytes = c < C ? 16 : 0;
    }
    __device__ __forceinline__ void set(int n, const GsTensor& t, int64_t b, int column) {
        token[n] = t.token;
        if (kStaged) {
            const int c = column * 32 * Word<T>::E;
            base[n] = static_cast<const T*>(t.p) + b * t.batch + c;
            at[n] = (static_cast<uint32_t>(threadIdx.x >> 3) * static_cast<uint32_t>(t.token) +
                     (chunk_bytes ? threadIdx.x & 7u : 0u) * static_cast<uint32_t>(16 / sizeof(T)));
        } else {
            base[n] = static_cast<const T*>(t.p) + b * t.batch + k.c;
        }
    }
    // the rows of a tile, `rows` of which hold tokens, into a slot
    __device__ __forceinline__ void fetch(int64_t tile, int rows, int slot) {
        if constexpr (kStaged) {
            const int r = threadIdx.x >> 3;
#pragma unroll
            for (int n = 0; n < kTensors; ++n) {
                const T* src = base[n] + tile * kTile * token[n];
                uint8_t* dst = room + (slot * kTensors + n) * kTileBytes + threadIdx.x * 16;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const bool live = r + 32 * half < rows;
                    const T* from = live ? src + at[n] + static_cast<uint32_t>(half * 32) * static_cast<uint32_t>(token[n]) : base[n];
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(dst + half * 4096)), "l"(from),
                                 "r"(live ? chunk_bytes : 0) : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else {
#pragma unroll
            for (int n = 0; n < kTensors; ++n) {
                const T* src = base[n] + (tile * kTile + warp * kTok) * token[n];
#pragma unroll
                for (int j = 0; j < kTok; ++j) raw[n][j] = k.load(src + j * token[n], k.ok && warp * kTok + j < rows);
            }
        }
    }
    template <int keep>
    __device__ __forceinline__ void wait() const {
        if (kStaged) asm volatile("cp.async.wait_group %0;" ::"n"(keep) : "memory");
    }
    __device__ __forceinline__ uint32_t word(int slot, int n, int j) const {
        if constexpr (kStaged)
            return *reinterpret_cast<const uint32_t*>(room + (slot * kTensors + n) * kTileBytes + (warp * kTok + j) * kRowBytes + lane * 4);
        else return raw[n][j];
    }
};

// the eight rows of a warp that hold tokens: [lo, hi) of its eight
struct Live {
    int lo, hi;
    __device__ __forceinline__ bool all() const { return lo <= 0 && hi >= kTok; }
    __device__ __forceinline__ bool operator()(int j) const { return j >= lo && j < hi; }
};
__device__ __forceinline__ int clamp_tile(int64_t n) { return n < 0 ? 0 : n > kTile ? kTile : static_cast<int>(n); }

template <bool k>
struct Is {
    static constexpr bool value = k;
};
template <typename F>
__device__ __forceinline__ void branch(bool b, F&& f) {
    if (b) f(Is<true>{});
    else f(Is<false>{});
}

// ---- forward

template <typename T, bool kLerp, bool kGate, bool kPacked, int kMode, bool kCluster>
__global__ void __launch_bounds__(kThreads, kMode == 2 ? 3 : 2) gs_fwd_kernel(const __grid_constant__ GsParams p) {
    constexpr bool kVec = kMode >= 1, kStaged = kMode == 2;
    constexpr int kTensors = kGate ? 3 : 2, kSlots = 3;
    using Col = Column<T, kVec>;
    using V = typename Col::V;
    __shared__ Pair<V> s_warp[2][kWarps][32];
    __shared__ Pair<V> s_rank[kCluster ? 2 : 1][kCluster ? kMaxRanks : 1][32];
    __shared__ int s_reset[2][kMaxRanks];
    __shared__ Rows s_rows[kPacked ? 3 : 1];
    extern __shared__ __align__(16) uint8_t s_tiles[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ranks = kCluster ? p.ranks : 1;
    const int rank = kCluster ? static_cast<int>(blockIdx.x % ranks) : 0;
    const int64_t unit = kCluster ? blockIdx.x / ranks : blockIdx.x;
    const int64_t b = unit / p.cols;
    const int column = static_cast<int>(unit - b * p.cols);
    const Col k(p, column);
    int64_t first = 0, last = p.L;
    if (kPacked) packed_span(p, &first, &last);
    const int64_t tiles = (last + kTile - 1) / kTile;
    const int64_t steps = (tiles + ranks - 1) / ranks;

    Tiles<T, kVec, kStaged, kTensors> in(k, column, p.C, s_tiles);
    in.set(0, p.x, b, column);
    in.set(1, p.r, b, column);
    if constexpr (kGate) in.set(2, p.i, b, column);
    const auto fetch = [&](int64_t tile, int slot) { in.fetch(tile, clamp_tile(last - tile * kTile), slot); };
    if (steps > 0) {
        fetch(rank, 0);
        if (kStaged) fetch(rank + ranks, 1);
    }

    const V d = k.param(p.decay);
    const V kd = kLerp ? d : each(d, [&](float v) { return -p.power * softplus(v); });
    bool small = true;
    each(kd, [&](float v) { small = small && v >= -kSeries; return v; });
    small = kLerp || __all_sync(0xffffffffu, small);
    if (kPacked && p.final_state) empty_sequences(p, k, rank, p.init, p.final_state);
    V carry = splat<V>(0.f);
    if (!kPacked && p.init) carry = k.get(p.init + b * p.C);
    if (kPacked && threadIdx.x < kTile) find_rows(p, s_rows[0], rank, last);
    in.template wait<1>();
    if (kStaged || kPacked) __syncthreads();

    T* py = p.y.p ? static_cast<T*>(p.y.p) + b * p.y.batch + k.c : nullptr;
    int rb = 0, slot = 0;
    for (int64_t step = 0; step < steps; ++step) {
        const int64_t tile = step * ranks + rank, t0 = tile * kTile + warp * kTok;
        const int buf = static_cast<int>(step & 1);
        Rows& rows = s_rows[kPacked ? rb : 0];
        uint32_t st = 0;
        V a[kTok], h[kTok];
        if (kPacked) {
            st = mine(rows.start, warp);
            rb = rb == 2 ? 0 : rb + 1;
        }
        // (the slot of the tile before, which every thread has read)
        const int next = slot == 2 ? 0 : slot + 1;
        if (kStaged) fetch(tile + 2 * ranks, next == 2 ? 0 : next + 1);
        branch(small, [&](auto is_small) {
#pragma unroll
            for (int j = 0; j < kTok; ++j) {
                const V x = Word<T>::unpack(in.word(slot, 0, j));
                const Gates<V> g = gates<kLerp, kGate, false, decltype(is_small)::value>(in.word(slot, 1, j), kGate ? in.word(slot, kTensors - 1, j) : 0u, kd);
                a[j] = g.a;
                h[j] = mul2(g.w, kGate ? mul2(g.si, x) : x);
            }
        });
        if (!kStaged) fetch(tile + ranks, 0);
        if (kPacked && st && p.init) {
#pragma unroll
            for (int j = 0; j < kTok; ++j)
                if (st >> j & 1) h[j] = fma2(a[j], k.get(p.init + static_cast<int64_t>(rows.seq[warp * kTok + j]) * p.C), h[j]);
        }
        // a[j] becomes the product of the decays, h[j] the state from zero, both from the thread's first
        // token (or from the last one up to j that begins a sequence)
#pragma unroll
        for (int j = 1; j < kTok; ++j) {
            const V hp = fma2(a[j], h[j - 1], h[j]);
            const bool cut = kPacked && (st >> j & 1);
            h[j] = cut ? h[j] : hp;
            a[j] = mul2(a[j], a[j - 1]);
        }
        s_warp[buf][warp][lane] = Pair<V>{a[kTok - 1], h[kTok - 1]};
        if (kPacked && threadIdx.x < kTile) find_rows(p, s_rows[rb], tile + ranks, last);
        in.template wait<1>();      // the next tile
        __syncthreads();
        V before;       // the state before this thread's tokens
        if (!kCluster) {
            V s = carry;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w == warp) before = s;
                const Pair<V> q = s_warp[buf][w][lane];
                const V n = fma2(q.a, s, q.b);
                s = kPacked && mine(rows.start, w) ? q.b : n;
            }
            if (p.marks && warp == 0 && tile < tiles) k.put(p.marks + (b * p.tiles + tile) * p.C, carry);
            carry = s;
        } else {
            // the tile's pair, and that of the warps before this one
            V pa = splat<V>(1.f), pb = splat<V>(0.f), ea, eb;
            bool cut = false, ecut = false;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w == warp) { ea = pa; eb = pb; ecut = cut; }
                const Pair<V> q = s_warp[buf][w][lane];
                const V n = fma2(q.a, pb, q.b);
                const bool c = kPacked && mine(rows.start, w);
                pb = c ? q.b : n;
                pa = mul2(pa, q.a);
                cut = cut || c;
            }
            cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
            if (warp < ranks) {         // one warp for each rank (at most eight)
                cl.map_shared_rank(&s_rank[buf][rank][0], warp)[lane] = Pair<V>{pa, pb};
                if (lane == 0) cl.map_shared_rank(&s_reset[buf][rank], warp)[0] = cut;
            }
            cl.sync();
            V s = carry;
            for (int r = 0; r < ranks; ++r) {
                if (r == rank) before = s;
                const Pair<V> q = s_rank[buf][r][lane];
                const V n = fma2(q.a, s, q.b);
                s = kPacked && s_reset[buf][r] ? q.b : n;
            }
            carry = s;
            if (p.marks && warp == 0 && tile < tiles) k.put(p.marks + (b * p.tiles + tile) * p.C, before);
            const V n = fma2(ea, before, eb);
            before = kPacked && ecut ? eb : n;
        }
#pragma unroll
        for (int j = 0; j < kTok; ++j) {
            const V n = fma2(a[j], before, h[j]);
            h[j] = kPacked && (st & ((2u << j) - 1)) ? h[j] : n;
        }
        slot = next;
        if (py) {
            const Live live{static_cast<int>(first > t0 ? (first - t0 < kTok ? first - t0 : kTok) : 0),
                            static_cast<int>(last > t0 ? (last - t0 < kTok ? last - t0 : kTok) : 0)};
            T* to = py + t0 * p.y.token;
            if (live.all() && k.ok) {
#pragma unroll
                for (int j = 0; j < kTok; ++j) k.store(to + j * p.y.token, h[j]);
            } else if (k.ok) {
#pragma unroll
                for (int j = 0; j < kTok; ++j)
                    if (live(j)) k.store(to + j * p.y.token, h[j]);
            }
        }
        if (!p.final_state) continue;
        const uint32_t en = kPacked ? mine(rows.end, warp) : 0u;
        if (kPacked && en) {
#pragma unroll
            for (int j = 0; j < kTok; ++j)
                if (en >> j & 1) k.put(p.final_state + static_cast<int64_t>(rows.seq[warp * kTok + j]) * p.C, h[j]);
        }
        if (!kPacked && t0 <= last - 1 && last - 1 < t0 + kTok) {
#pragma unroll
            for (int j = 0; j < kTok; ++j)
                if (t0 + j == last - 1) k.put(p.final_state + b * p.C, h[j]);
        }
    }
    // (no token at all: the state stays)
    if (!kPacked && steps == 0 && rank == 0 && warp == 0 && p.final_state) k.put(p.final_state + b * p.C, carry);
    in.template wait<0>();
}

// ---- backward

template <typename T, bool kLerp, bool kGate, bool kPacked, int kMode, bool kCluster>
__global__ void __launch_bounds__(kThreads, 2) gs_bwd_kernel(const __grid_constant__ GsParams p) {
    constexpr bool kVec = kMode >= 1, kStaged = kMode == 2;
    constexpr int kTensors = kGate ? 4 : 3;
    using Col = Column<T, kVec>;
    using V = typename Col::V;
    __shared__ Pair<V> s_warp[2][kWarps][32];
    __shared__ V s_back[2][kWarps][32];
    __shared__ Pair<V> s_rank[kCluster ? 2 : 1][kCluster ? kMaxRanks : 1][32];
    __shared__ int s_reset[2][kMaxRanks];
    __shared__ Rows s_rows[kPacked ? 3 : 1];
    extern __shared__ __align__(16) uint8_t s_tiles[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ranks = kCluster ? p.ranks : 1;
    const int rank = kCluster ? static_cast<int>(blockIdx.x % ranks) : 0;
    const int64_t unit = kCluster ? blockIdx.x / ranks : blockIdx.x;
    const int share = static_cast<int>(unit / p.cols);
    const int column = static_cast<int>(unit - static_cast<int64_t>(share) * p.cols);
    const Col k(p, column);
    sm100::grid_dep_wait();     // the marks may still be formed
    sm100::grid_dep_launch_dependents();
    int64_t first = 0, last = p.L;
    if (kPacked) packed_span(p, &first, &last);
    const int64_t tiles = (last + kTile - 1) / kTile;
    const int64_t steps = (tiles + ranks - 1) / ranks;

    const V d = k.param(p.decay);
    const V kd = kLerp ? d : each(d, [&](float v) { return -p.power * softplus(v); });
    bool small = true;
    each(kd, [&](float v) { small = small && v >= -kSeries; return v; });
    small = kLerp || __all_sync(0xffffffffu, small);
    if (kPacked && p.dinit) empty_sequences(p, k, rank, p.dfinal, p.dinit);
    V sum = splat<V>(0.f);
    int tick = 0;               // which of the two exchange buffers is next, across sequences
    const V zero = splat<V>(0.f);
    Tiles<T, kVec, kStaged, kTensors> in(k, column, p.C, s_tiles);

    for (int64_t b = share; b < p.nb; b += p.shares) {
        in.set(0, p.x, b, column);
        in.set(1, p.r, b, column);
        in.set(2, p.dy, b, column);
        if constexpr (kGate) in.set(3, p.i, b, column);
        V mark = zero;
        const auto fetch = [&](int64_t tile, int slot) { in.fetch(tile < 0 ? 0 : tile, tile < 0 ? 0 : clamp_tile(last - tile * kTile), slot); };
        const auto get_mark = [&](int64_t tile) { mark = tile >= 0 ? k.get(p.marks + (b * p.tiles + tile) * p.C) : zero; };
        T *qx = static_cast<T*>(p.dx.p) + b * p.dx.batch + k.c, *qr = static_cast<T*>(p.dr.p) + b * p.dr.batch + k.c;
        T* qi = kGate ? static_cast<T*>(p.di.p) + b * p.di.batch + k.c : nullptr;
        if (steps > 0) {
            fetch(tiles - 1 - rank, 0);
            if (kStaged) fetch(tiles - 1 - rank - ranks, 1);
        }
        get_mark(tiles - 1 - rank);
        int rb = 0, slot = 0;
        if (kPacked && threadIdx.x < kTile) find_rows(p, s_rows[0], tiles - 1 - rank, last);
        in.template wait<1>();
        if (kStaged || kPacked) __syncthreads();
        V carry = zero;         // G behind the tiles done so far (set where a sequence ends)
        for (int64_t step = 0; step < steps; ++step) {
            const int64_t tile = tiles - 1 - step * ranks - rank, t0 = tile * kTile + warp * kTok;
            const int buf = tick;
            tick ^= 1;
            Rows& rows = s_rows[kPacked ? rb : 0];
            // rows that begin and end a sequence: bits of the thread's tokens
            uint32_t st, en;
            const int tail = tile >= 0 && last - 1 - tile * kTile < kTile ? static_cast<int>(last - 1 - tile * kTile) : -1;
            const auto ends = [&](int w) {
                if (kPacked) return mine(rows.end, w);
                return tail >= 0 && tail >> 3 == w ? 1u << (tail & 7) : 0u;
            };
            if (kPacked) {
                st = mine(rows.start, warp);
                rb = rb == 2 ? 0 : rb + 1;
            } else {
                st = t0 == 0 ? 1u : 0u;
            }
            en = ends(warp);
            const Live live{static_cast<int>(first > t0 ? (first - t0 < kTok ? first - t0 : kTok) : 0),
                            static_cast<int>(tile >= 0 && last > t0 ? (last - t0 < kTok ? last - t0 : kTok) : 0)};
            const bool plain = st == 0 && en == 0 && live.all();
            const auto seq = [&](int j) { return kPacked ? static_cast<int64_t>(rows.seq[warp * kTok + j]) : b; };
            const auto gin = [&](int j) { return p.dfinal ? k.get(p.dfinal + seq(j) * p.C) : zero; };
            V a[kTok], h[kTok];
            branch(small, [&](auto is_small) {
#pragma unroll
                for (int j = 0; j < kTok; ++j) {
                    const V x = Word<T>::unpack(in.word(slot, 0, j));
                    const Gates<V> g = gates<kLerp, kGate, false, decltype(is_small)::value>(in.word(slot, 1, j), kGate ? in.word(slot, kTensors - 1, j) : 0u, kd);
                    a[j] = g.a;
                    h[j] = mul2(g.w, kGate ? mul2(g.si, x) : x);
                }
            });
            V pa = a[0], pb = h[0], pg = zero;
            if (plain) {
#pragma unroll
                for (int j = 1; j < kTok; ++j) {
                    pb = fma2(a[j], pb, h[j]);
                    pa = mul2(pa, a[j]);
                }
#pragma unroll
                for (int j = kTok - 1; j >= 0; --j) pg = mul2(a[j], add2(Word<T>::unpack(in.word(slot, 2, j)), pg));
            } else {
                if (kPacked && (st & 1) && p.init) pb = fma2(a[0], k.get(p.init + seq(0) * p.C), h[0]);
#pragma unroll
                for (int j = 1; j < kTok; ++j) {
                    if (kPacked && (st >> j & 1)) {
                        pb = p.init ? fma2(a[j], k.get(p.init + seq(j) * p.C), h[j]) : h[j];
                    } else {
                        pb = fma2(a[j], pb, h[j]);
                    }
                    pa = mul2(pa, a[j]);
                }
#pragma unroll
                for (int j = kTok - 1; j >= 0; --j) {
                    if (en >> j & 1) pg = gin(j);
                    pg = mul2(a[j], add2(Word<T>::unpack(in.word(slot, 2, j)), pg));
                }
            }
            s_warp[buf][warp][lane] = Pair<V>{pa, pb};
            s_back[buf][warp][lane] = pg;
            if (kPacked && threadIdx.x < kTile) find_rows(p, s_rows[rb], tile - ranks, last);
            in.template wait<0>();      // the next tile
            __syncthreads();
            // (into the slot of the tile before, which every thread has done with)
            const int next = slot == 2 ? 0 : slot + 1;
            if (kStaged) fetch(tile - 2 * ranks, next == 2 ? 0 : next + 1);
            V hp = mark;        // the state before this thread's tokens
            get_mark(tile - ranks);
#pragma unroll
            for (int w = 0; w < kWarps - 1; ++w) {
                if (w >= warp) break;
                const Pair<V> q = s_warp[buf][w][lane];
                const V n = fma2(q.a, hp, q.b);
                hp = kPacked && mine(rows.start, w) ? q.b : n;
            }
            V G;                // G behind them
            if (!kCluster) {
                V s = carry;
#pragma unroll
                for (int w = kWarps - 1; w >= 0; --w) {
                    if (w == warp) G = s;
                    const V back = s_back[buf][w][lane], n = fma2(s_warp[buf][w][lane].a, s, back);
                    s = ends(w) ? back : n;
                }
                carry = s;
            } else {
                V ca = splat<V>(1.f), cb = zero, ea, eb;
                bool cut = false, ecut = false;
#pragma unroll
                for (int w = kWarps - 1; w >= 0; --w) {
                    if (w == warp) { ea = ca; eb = cb; ecut = cut; }
                    const V qa = s_warp[buf][w][lane].a, qb = s_back[buf][w][lane];
                    const V n = fma2(qa, cb, qb);
                    const bool c = ends(w) != 0;
                    cb = c ? qb : n;
                    ca = mul2(ca, qa);
                    cut = cut || c;
                }
                cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
                if (warp < ranks) {
                    cl.map_shared_rank(&s_rank[buf][rank][0], warp)[lane] = Pair<V>{ca, cb};
                    if (lane == 0) cl.map_shared_rank(&s_reset[buf][rank], warp)[0] = cut;
                }
                cl.sync();
                V s = carry;
                for (int r = 0; r < ranks; ++r) {
                    if (r == rank) G = s;
                    const Pair<V> q = s_rank[buf][r][lane];
                    const V n = fma2(q.a, s, q.b);
                    s = s_reset[buf][r] ? q.b : n;
                }
                carry = s;
                const V n = fma2(ea, G, eb);
                G = ecut ? eb : n;
            }
            // the states before each token, then the gradients from the last token back
#pragma unroll
            for (int j = 0; j < kTok; ++j) {
                if (kPacked && (st >> j & 1)) hp = p.init ? k.get(p.init + seq(j) * p.C) : zero;
                const V n = fma2(a[j], hp, h[j]);
                h[j] = hp;
                hp = n;
            }
            T *tx = qx + t0 * p.dx.token, *tr = qr + t0 * p.dr.token, *ti = kGate ? qi + t0 * p.di.token : nullptr;
            const auto token = [&](int j, auto is_plain, auto is_small) {
                constexpr bool kPlain = decltype(is_plain)::value;
                if (!kPlain && (en >> j & 1)) G = gin(j);
                const V g = add2(Word<T>::unpack(in.word(slot, 2, j)), G);
                const V x = Word<T>::unpack(in.word(slot, 0, j));
                const Gates<V> gt = gates<kLerp, kGate, true, decltype(is_small)::value>(in.word(slot, 1, j), kGate ? in.word(slot, kTensors - 1, j) : 0u, kd);
                const bool on = kPlain ? k.ok : k.ok && live(j);
                const V du = mul2(g, gt.w);
                const V dx = kGate ? mul2(du, gt.si) : du, u = kGate ? mul2(x, gt.si) : x;
                V dr, dl;
                if (kLerp) {
                    dl = dr = mul2(mul2(g, add2(h[j], neg(u))), mul2(a[j], gt.w));
                } else {
                    dl = mul2(g, mul2(a[j], fma2(gt.l, h[j], neg(mul2(mul2(u, a[j]), gt.lw)))));
                    dr = mul2(dl, gt.cr);
                }
                if (kPlain || on) sum = add2(sum, dl);
                G = mul2(a[j], g);
                if (on) {
                    k.store(tx + j * p.dx.token, dx);
                    k.store(tr + j * p.dr.token, dr);
                    if (kGate) k.store(ti + j * p.di.token, mul2(mul2(dx, x), gt.ci));
                }
                if (!kPlain && (st >> j & 1) && tile >= 0 && p.dinit) k.put(p.dinit + seq(j) * p.C, G);
            };
            if (plain && small) {
#pragma unroll
                for (int j = kTok - 1; j >= 0; --j) token(j, Is<true>{}, Is<true>{});
            } else if (plain) {
#pragma unroll
                for (int j = kTok - 1; j >= 0; --j) token(j, Is<true>{}, Is<kLerp>{});
            } else {
#pragma unroll
                for (int j = kTok - 1; j >= 0; --j) token(j, Is<false>{}, Is<kLerp>{});
            }
            if (!kStaged) fetch(tile - ranks, 0);
            slot = next;
        }
        in.template wait<0>();
        __syncthreads();        // the next sequence's rows, tiles and pairs
        if (!kPacked && steps == 0 && rank == 0 && warp == 0 && p.dinit)
            k.put(p.dinit + b * p.C, p.dfinal ? k.get(p.dfinal + b * p.C) : zero);
    }
    if (!p.part) return;
    s_back[0][warp][lane] = sum;
    __syncthreads();
    if (warp != 0) return;
    V total = zero;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total = add2(total, s_back[0][w][lane]);
    if (!kLerp)         // dlog a / dd = log a sig(d) / softplus(d); both go to zero together
        total = mul2(total, each(d, [](float v) {
            const float s = softplus(v);
            return v < -15.f ? 1.f : 1.f / (s * (1.f + expf(-v)));
        }));
    k.put(p.part + (static_cast<int64_t>(share) * ranks + rank) * p.C, total);
}

// ---- one token

template <typename T, bool kLerp, bool kGate, bool kVec>
__global__ void __launch_bounds__(kThreads) gs_step_kernel(const __grid_constant__ GsParams p, const int32_t* __restrict__ slots,
                                                           int64_t nstates) {
    using W = Word<T>;
    using V = typename W::V;
    using Col = Column<T, kVec>;
    // a warp takes 32 words of one sequence
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t b = unit / p.cols;
    if (b >= p.nb) return;
    const Col k(p, static_cast<int>(unit - b * p.cols));
    const int64_t slot = slots ? __ldg(slots + b) : b;
    const uint32_t rx = k.load(at<const T>(p.x, b, k.c), k.ok), rr = k.load(at<const T>(p.r, b, k.c), k.ok);
    const uint32_t ri = kGate ? k.load(at<const T>(p.i, b, k.c), k.ok) : 0u;
    const V d = k.param(p.decay);
    V h = splat<V>(0.f);
    const bool in = slot >= 0 && slot < nstates;
    if (in) {
        const V kd = kLerp ? d : each(d, [&](float v) { return -p.power * softplus(v); });
        const Gates<V> g = gates<kLerp, kGate, false, false>(rr, ri, kd);
        const V x = W::unpack(rx);
        h = fma2(g.a, k.get(p.init + slot * p.C), mul2(g.w, kGate ? mul2(g.si, x) : x));
        k.put(p.final_state + slot * p.C, h);
    }
    if (k.ok) k.store(at<T>(p.y, b, k.c), h);
}

// ---- launches

template <typename... P, typename... Args>
cudaError_t launch(void (*kernel)(P...), int64_t grid, int ranks, int smem, bool after, cudaStream_t s, const Args&... args) {
    if (ranks == 1 && !after) {
        kernel<<<static_cast<unsigned>(grid), kThreads, smem, s>>>(args...);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    if (ranks > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(ranks);
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (after) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    cfg.attrs = attr;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <bool... b>
struct Flags {
    template <int i>
    static constexpr bool at() {
        constexpr bool v[] = {b...};
        return v[i];
    }
};
template <bool... B, typename F>
auto with_bools(F&& f) { return f(Flags<B...>{}); }
template <bool... B, typename F, typename... R>
auto with_bools(F&& f, bool b, R... r) { return b ? with_bools<B..., true>(f, r...) : with_bools<B..., false>(f, r...); }

// Rows of whole units of `bytes`: pointers, strides and channels; a tile's rows within 32-bit offsets.
bool rows_of(const GsParams& p, int es, int bytes) {
    if (p.C * static_cast<int64_t>(es) % bytes) return false;
    for (const GsTensor* t : {&p.x, &p.r, &p.i, &p.y, &p.dy, &p.dx, &p.dr, &p.di})
        if (t->p && (reinterpret_cast<uintptr_t>(t->p) % bytes || t->batch * es % bytes || t->token * es % bytes ||
                     t->token < 0 || t->token > (int64_t(1) << 25)))
            return false;
    return true;
}
// 2: staged through shared memory; 1: words of two bf16 or one fp32; 0: an element at a time
template <typename T>
int mode_of(const GsParams& p) {
    constexpr int es = sizeof(T);
    return rows_of(p, es, 16) ? 2 : es == 4 || rows_of(p, es, 4) ? 1 : 0;
}

// CTAs of a column: as many as there is room for beside the other columns.
constexpr int kPerSm = 2;
int rank_count(int64_t units, int64_t tiles, int per_sm) {
    int64_t r = per_sm * static_cast<int64_t>(device_sm_count()) / (units > 0 ? units : 1);
    if (r > tiles) r = tiles;
    return r < 1 ? 1 : r > kMaxRanks ? kMaxRanks : static_cast<int>(r);
}

// Backward: shares of the batch that one column's CTAs walk through one after another.
int share_count(const GsParams& p) {
    const int64_t want = (kPerSm * static_cast<int64_t>(device_sm_count()) + p.cols - 1) / p.cols;
    return static_cast<int>(p.nb < want ? p.nb : want);
}

// f with the kernel's mode: element-wise code exists for bf16 alone
template <typename T, typename F>
cudaError_t with_mode(int mode, F&& f) {
    if (mode == 2) return f(std::integral_constant<int, 2>{});
    if constexpr (sizeof(T) == 2) {
        if (mode == 0) return f(std::integral_constant<int, 0>{});
    }
    return f(std::integral_constant<int, 1>{});
}

template <auto K>
cudaError_t staged_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    return bytes > 0 ? allow_smem(K, bytes, done) : cudaSuccess;
}

template <typename T>
cudaError_t launch_fwd(GsParams p, bool lerp, cudaStream_t s) {
    const int mode = mode_of<T>(p);
    p.ranks = rank_count(p.nb * p.cols, p.tiles, mode == 2 ? 3 : 2);
    return with_mode<T>(mode, [&](auto m) {
        return with_bools<>([&](auto f) {
            using F = decltype(f);
            constexpr int kMode = decltype(m)::value;
            constexpr auto kernel = gs_fwd_kernel<T, F::template at<0>(), F::template at<1>(), F::template at<2>(), kMode, F::template at<3>()>;
            constexpr int smem = kMode == 2 ? 3 * (F::template at<1>() ? 3 : 2) * kTileBytes : 0;
            const cudaError_t e = staged_smem<kernel>(smem);
            return e != cudaSuccess ? e : launch(kernel, p.nb * p.cols * p.ranks, p.ranks, smem, false, s, p);
        }, lerp, p.i.p != nullptr, p.cu != nullptr, p.ranks > 1);
    });
}

template <typename T>
cudaError_t launch_bwd(GsParams p, bool lerp, bool after, float* ddecay, cudaStream_t s) {
    p.shares = share_count(p);
    p.ranks = rank_count(static_cast<int64_t>(p.shares) * p.cols, p.tiles, kPerSm);
    if (!ddecay) p.part = nullptr;
    else if (p.shares * p.ranks == 1) p.part = ddecay;
    const cudaError_t e = with_mode<T>(mode_of<T>(p), [&](auto m) {
        return with_bools<>([&](auto f) {
            using F = decltype(f);
            constexpr int kMode = decltype(m)::value;
            constexpr auto kernel = gs_bwd_kernel<T, F::template at<0>(), F::template at<1>(), F::template at<2>(), kMode, F::template at<3>()>;
            constexpr int smem = kMode == 2 ? 3 * (F::template at<1>() ? 4 : 3) * kTileBytes : 0;
            const cudaError_t e = staged_smem<kernel>(smem);
            return e != cudaSuccess ? e : launch(kernel, static_cast<int64_t>(p.shares) * p.cols * p.ranks, p.ranks, smem, after, s, p);
        }, lerp, p.i.p != nullptr, p.cu != nullptr, p.ranks > 1);
    });
    if (e != cudaSuccess || !ddecay || p.shares * p.ranks == 1) return e;
    float* const outs[1] = {ddecay};
    return launch_sum_shares(p.part, p.shares * p.ranks, p.C, outs, 1, s);
}

template <typename T>
cudaError_t launch_step(const GsParams& p, bool lerp, const int32_t* slots, int64_t nstates, cudaStream_t s) {
    const int64_t grid = (p.nb * p.cols + kWarps - 1) / kWarps;
    return with_bools<>([&](auto f) {
        using F = decltype(f);
        return launch(gs_step_kernel<T, F::template at<0>(), F::template at<1>(), F::template at<2>() || sizeof(T) == 4>, grid, 1, 0, false, s,
                      p, slots, nstates);
    }, lerp, p.i.p != nullptr, sizeof(T) == 4 || mode_of<T>(p) > 0);
}

m3_status err(m3_status st, const char* fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return set_error(st, msg);
}

m3_status check(const m3_gated_scan_dims* d) {
    if (!d) return err(M3_ERR_INVALID_ARG, "dims is NULL");
    if (d->in_dtype != M3_F32 && d->in_dtype != M3_BF16)
        return err(M3_ERR_INVALID_ARG, "in_dtype %d is not M3_F32 or M3_BF16", d->in_dtype);
    if (d->nseq < 0 || d->seqlen < 0) return err(M3_ERR_INVALID_ARG, "nseq and seqlen must be >= 0");
    if (d->channels < 1) return err(M3_ERR_INVALID_ARG, "channels must be >= 1");
    if (d->flags & ~M3_GS_LERP) return err(M3_ERR_INVALID_ARG, "unknown bits in flags (0x%x)", (unsigned)d->flags);
    if (!(d->flags & M3_GS_LERP) && !(d->power > 0.f && std::isfinite(d->power)))
        return err(M3_ERR_INVALID_ARG, "power must be finite and > 0");
    if (d->nseq > (int64_t(1) << 24) || d->seqlen > (int64_t(1) << 30) || d->channels > (int64_t(1) << 24))
        return err(M3_ERR_UNSUPPORTED, "more than 2^24 sequences, 2^30 tokens or 2^24 channels");
    const int64_t per = d->in_dtype == M3_BF16 ? 64 : 32, cols = (d->channels + per - 1) / per;
    if (d->nseq > 0 && cols > 0x7fffffffLL / kMaxRanks / d->nseq)
        return err(M3_ERR_UNSUPPORTED, "nseq * channels exceeds 2^33 (fp32) or 2^34 (bf16)");
    return M3_OK;
}

m3_status check_ptr(const void* q, uintptr_t align, const char* name, bool need) {
    if (!q) return need ? err(M3_ERR_INVALID_ARG, "%s is NULL", name) : M3_OK;
    if (reinterpret_cast<uintptr_t>(q) % align)
        return err(M3_ERR_INVALID_ARG, "%s is not %s-aligned", name, align == 16 ? "16-byte" : "element");
    return M3_OK;
}

struct Named {
    const void* p;
    const char* name;
};
// An output begins at no input's or other output's address; the pairs that may share are left out by the caller.
template <int I>
m3_status check_apart(const Named& out, const Named (&others)[I]) {
    for (const Named& o : others)
        if (out.p && out.p == o.p) return err(M3_ERR_INVALID_ARG, "%s is %s", out.name, o.name);
    return M3_OK;
}

m3_status check_inputs(const m3_gated_scan_dims* d, const m3_gated_scan_inputs* in, bool any) {
    if (!in) return err(M3_ERR_INVALID_ARG, "inputs is NULL");
    const uintptr_t es = d->in_dtype == M3_BF16 ? 2 : 4;
    m3_status st;
    if ((st = check_ptr(in->x.data, es, "x", any)) != M3_OK || (st = check_ptr(in->r.data, es, "r", any)) != M3_OK ||
        (st = check_ptr(in->i.data, es, "i", false)) != M3_OK || (st = check_ptr(in->cu_seqlens, 4, "cu_seqlens", false)) != M3_OK ||
        (st = check_ptr(in->decay, 4, "decay", any && !(d->flags & M3_GS_LERP))) != M3_OK)
        return st;
    return M3_OK;
}

// Rows of an output that share elements through equal strides.
m3_status check_out(const m3_view& v, const m3_gated_scan_dims* d, bool packed, const char* name) {
    const int64_t t = v.token < 0 ? -v.token : v.token, b = v.batch < 0 ? -v.batch : v.batch;
    if ((d->seqlen > 1 && t < d->channels) || (!packed && d->nseq > 1 && b < d->channels))
        return err(M3_ERR_INVALID_ARG, "%s: rows overlap", name);
    return M3_OK;
}

// A dimension of one entry has stride 0, whatever the caller's says.
GsTensor tensor(const m3_gated_scan_dims* d, const m3_view& v, bool packed) {
    return GsTensor{v.data, packed || d->nseq <= 1 ? 0 : v.batch, d->seqlen <= 1 ? 0 : v.token};
}

GsParams make_params(const m3_gated_scan_dims* d, const m3_gated_scan_inputs* in) {
    GsParams p{};
    const bool packed = in->cu_seqlens != nullptr;
    p.x = tensor(d, in->x, packed);
    p.r = tensor(d, in->r, packed);
    if (in->i.data) p.i = tensor(d, in->i, packed);
    p.decay = in->decay;
    p.cu = in->cu_seqlens;
    p.L = d->seqlen;
    p.nb = packed ? 1 : d->nseq;
    p.nseq = static_cast<int>(d->nseq);
    p.C = static_cast<int>(d->channels);
    const int per = d->in_dtype == M3_BF16 ? 64 : 32;
    p.cols = (p.C + per - 1) / per;
    p.ranks = 1;
    p.tiles = static_cast<int>((d->seqlen + kTile - 1) / kTile);
    p.power = d->power;
    return p;
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }
size_t marks_bytes(const m3_gated_scan_dims* d, bool packed) {
    return up(static_cast<size_t>(packed ? 1 : d->nseq) * static_cast<size_t>((d->seqlen + kTile - 1) / kTile) *
              static_cast<size_t>(d->channels) * 4);
}

m3_status done(cudaError_t e, const char* what) {
    return e == cudaSuccess ? M3_OK : err(M3_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

// states, marks and sums: fp32, 16-byte aligned
template <int N>
m3_status check_f32(const Named (&ts)[N]) {
    m3_status st = M3_OK;
    for (const Named& t : ts)
        if ((st = check_ptr(t.p, 16, t.name, false)) != M3_OK) return st;
    return st;
}

}  // namespace
}  // namespace m3

using namespace m3;

extern "C" {

m3_status m3_gated_scan_fwd(const m3_gated_scan_dims* dims, const m3_gated_scan_inputs* in, const float* init,
                            float* final_state, const m3_view* y, float* marks, void* stream) {
    set_error(M3_OK, "");
    m3_status st = check(dims);
    if (st != M3_OK) return st;
    const bool packed = in && in->cu_seqlens, rows = dims->nseq > 0 && dims->seqlen > 0;
    if ((st = check_inputs(dims, in, rows)) != M3_OK ||
        (st = check_ptr(y ? y->data : nullptr, dims->in_dtype == M3_BF16 ? 2 : 4, "y", rows)) != M3_OK ||
        (st = check_f32({{init, "init"}, {final_state, "final"}, {marks, "marks"}})) != M3_OK)
        return st;
    if (dims->nseq == 0) return M3_OK;
    const Named ins[] = {{in->x.data, "x"}, {in->r.data, "r"}, {in->i.data, "i"}, {in->decay, "decay"},
                         {in->cu_seqlens, "cu_seqlens"}};
    const Named yo{y ? y->data : nullptr, "y"}, fo{final_state, "final"}, mo{marks, "marks"};
    if ((rows && (st = check_out(*y, dims, packed, "y")) != M3_OK) || (st = check_apart(yo, ins)) != M3_OK ||
        (st = check_apart(yo, {{init, "init"}})) != M3_OK || (st = check_apart(fo, ins)) != M3_OK ||
        (st = check_apart(fo, {yo})) != M3_OK || (st = check_apart(mo, ins)) != M3_OK ||
        (st = check_apart(mo, {yo, fo, {init, "init"}})) != M3_OK)
        return st;
    if (!rows && !final_state) return M3_OK;
    GsParams p = make_params(dims, in);
    if (rows) p.y = tensor(dims, *y, packed);
    p.init = init;
    p.final_state = final_state;
    p.marks = marks;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool lerp = dims->flags & M3_GS_LERP;
    return done(dims->in_dtype == M3_BF16 ? launch_fwd<__nv_bfloat16>(p, lerp, s) : launch_fwd<float>(p, lerp, s), "gated scan");
}

m3_status m3_gated_scan_step(const m3_gated_scan_dims* dims, const m3_gated_scan_inputs* in, const float* state_in,
                             float* state_out, int64_t nstates, const int32_t* slots, const m3_view* y, void* stream) {
    set_error(M3_OK, "");
    m3_status st = check(dims);
    if (st != M3_OK) return st;
    const bool any = dims->nseq > 0;
    if (dims->seqlen != 1) return err(M3_ERR_INVALID_ARG, "a step has seqlen 1");
    if (in && in->cu_seqlens) return err(M3_ERR_INVALID_ARG, "a step takes no cu_seqlens");
    if ((st = check_inputs(dims, in, any)) != M3_OK) return st;
    if (nstates < 0 || (!slots && nstates < dims->nseq))
        return err(M3_ERR_INVALID_ARG, "nstates (%lld) below the number of sequences", (long long)nstates);
    if ((st = check_ptr(y ? y->data : nullptr, dims->in_dtype == M3_BF16 ? 2 : 4, "y", any)) != M3_OK ||
        (st = check_ptr(state_in, 16, "state_in", any && nstates > 0)) != M3_OK ||
        (st = check_ptr(state_out, 16, "state_out", any && nstates > 0)) != M3_OK ||
        (st = check_ptr(slots, 4, "slots", false)) != M3_OK)
        return st;
    if (!any) return M3_OK;
    const Named ins[] = {{in->x.data, "x"}, {in->r.data, "r"}, {in->i.data, "i"}, {in->decay, "decay"}, {slots, "slots"}};
    const Named yo{y->data, "y"}, so{state_out, "state_out"};
    if ((st = check_out(*y, dims, false, "y")) != M3_OK || (st = check_apart(yo, ins)) != M3_OK ||
        (st = check_apart(yo, {{state_in, "state_in"}})) != M3_OK || (st = check_apart(so, ins)) != M3_OK ||
        (st = check_apart(so, {yo})) != M3_OK)
        return st;
    GsParams p = make_params(dims, in);
    p.y = tensor(dims, *y, false);
    p.init = state_in;
    p.final_state = state_out;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool lerp = dims->flags & M3_GS_LERP;
    return done(dims->in_dtype == M3_BF16 ? launch_step<__nv_bfloat16>(p, lerp, slots, nstates, s)
                                          : launch_step<float>(p, lerp, slots, nstates, s), "gated scan step");
}

size_t m3_gated_scan_bwd_workspace_bytes(const m3_gated_scan_dims* dims, int packed, int have_marks) {
    if (check(dims) != M3_OK || dims->nseq == 0 || dims->seqlen == 0) return 0;
    m3_gated_scan_inputs in{};
    const int32_t mark = 0;
    if (packed) in.cu_seqlens = &mark;
    GsParams p = make_params(dims, &in);
    p.shares = share_count(p);
    const size_t part = up(static_cast<size_t>(p.shares) * rank_count(static_cast<int64_t>(p.shares) * p.cols, p.tiles, kPerSm) *
                           static_cast<size_t>(p.C) * 4);
    return part + (have_marks ? 0 : marks_bytes(dims, packed));
}

m3_status m3_gated_scan_bwd(const m3_gated_scan_dims* dims, const m3_gated_scan_inputs* in, const float* init,
                            const float* marks, const m3_view* dy, const float* dfinal, const m3_gated_scan_grads* grads,
                            float* ddecay, float* dinit, void* workspace, size_t ws_bytes, void* stream) {
    set_error(M3_OK, "");
    m3_status st = check(dims);
    if (st != M3_OK) return st;
    const bool packed = in && in->cu_seqlens, rows = dims->nseq > 0 && dims->seqlen > 0;
    const uintptr_t es = dims->in_dtype == M3_BF16 ? 2 : 4;
    if ((st = check_inputs(dims, in, rows)) != M3_OK) return st;
    if (!grads) return err(M3_ERR_INVALID_ARG, "grads is NULL");
    const bool gate = in->i.data != nullptr;
    if ((st = check_ptr(dy ? dy->data : nullptr, es, "dy", rows)) != M3_OK ||
        (st = check_ptr(grads->dx.data, es, "dx", rows)) != M3_OK || (st = check_ptr(grads->dr.data, es, "dr", rows)) != M3_OK ||
        (st = check_ptr(grads->di.data, es, "di", rows && gate)) != M3_OK ||
        (st = check_f32({{init, "init"}, {marks, "marks"}, {dfinal, "dfinal"}, {ddecay, "ddecay"}, {dinit, "dinit"}})) != M3_OK)
        return st;
    if (ddecay && !in->decay) return err(M3_ERR_INVALID_ARG, "ddecay without decay");
    const Named x{in->x.data, "x"}, r{in->r.data, "r"}, i{in->i.data, "i"}, g{dy ? dy->data : nullptr, "dy"};
    const Named dx{grads->dx.data, "dx"}, dr{grads->dr.data, "dr"}, di{gate ? grads->di.data : nullptr, "di"};
    const Named rest[] = {{in->decay, "decay"}, {in->cu_seqlens, "cu_seqlens"}, {init, "init"}, {marks, "marks"}};
    const Named dd{ddecay, "ddecay"}, ds{dinit, "dinit"}, df{dfinal, "dfinal"};
    if (dims->nseq > 0) {
        for (const Named* o : {&dx, &dr, &di, &dd, &ds}) {
            if ((st = check_apart(*o, {x, r, i, g})) != M3_OK || (st = check_apart(*o, rest)) != M3_OK) return st;
            if (o != &ds && (st = check_apart(*o, {df})) != M3_OK) return st;
        }
        if ((st = check_apart(dr, {dx})) != M3_OK || (st = check_apart(di, {dx, dr})) != M3_OK ||
            (st = check_apart(dd, {dx, dr, di})) != M3_OK || (st = check_apart(ds, {dx, dr, di, dd})) != M3_OK)
            return st;
        if (rows && ((st = check_out(grads->dx, dims, packed, "dx")) != M3_OK ||
                     (st = check_out(grads->dr, dims, packed, "dr")) != M3_OK ||
                     (gate && (st = check_out(grads->di, dims, packed, "di")) != M3_OK)))
            return st;
    }
    const size_t need = m3_gated_scan_bwd_workspace_bytes(dims, packed, marks != nullptr);
    if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || ws_bytes < need))
        return err(M3_ERR_INVALID_ARG, "workspace: NULL, misaligned or below %zu bytes", need);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!rows) {
        cudaError_t e = cudaSuccess;
        const size_t n = static_cast<size_t>(dims->nseq) * dims->channels * 4;
        if (ddecay) e = cudaMemsetAsync(ddecay, 0, dims->channels * 4, s);
        if (e == cudaSuccess && dinit && n && dinit != dfinal)
            e = dfinal ? cudaMemcpyAsync(dinit, dfinal, n, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(dinit, 0, n, s);
        return done(e, "empty gradient");
    }
    GsParams p = make_params(dims, in);
    const bool lerp = dims->flags & M3_GS_LERP, bf16 = dims->in_dtype == M3_BF16;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.init = init;
    if (!marks) {       // the states before each tile, without y
        p.marks = reinterpret_cast<float*>(ws);
        ws += marks_bytes(dims, packed);
        const cudaError_t e = bf16 ? launch_fwd<__nv_bfloat16>(p, lerp, s) : launch_fwd<float>(p, lerp, s);
        if (e != cudaSuccess) return done(e, "gated scan states");
    } else {
        p.marks = const_cast<float*>(marks);
    }
    p.part = reinterpret_cast<float*>(ws);
    p.dy = tensor(dims, *dy, packed);
    p.dx = tensor(dims, grads->dx, packed);
    p.dr = tensor(dims, grads->dr, packed);
    if (gate) p.di = tensor(dims, grads->di, packed);
    p.dfinal = dfinal;
    p.dinit = dinit;
    return done(bf16 ? launch_bwd<__nv_bfloat16>(p, lerp, !marks, ddecay, s) : launch_bwd<float>(p, lerp, !marks, ddecay, s),
                "gated scan backward");
}

}  // extern "C"
