// Gated linear recurrence of each channel, its single-token form and its gradients.
//
//     power:  log a_t = -power softplus(d) sig(r_t),  w_t = sqrt(1 - a_t^2)
//     lerp:   a_t = sig(r_t + d),                     w_t = 1 - a_t
//     h_t = a_t h_{t-1} + w_t u_t,  u_t = sig(i_t) x_t
// The floor is HBM's: the forward reads x, r, i and writes y once, the backward reads those and dy and writes
// three gradients. bf16, 4 x 2048 x 4096: forward 72 us (0.57 of what a copy reaches), gradients 135 (0.53); one sequence of
// 65 536 x 4096: forward 687 us (0.48). What bounds a batch is the issue of instructions: some 46 a channel and token
// forward, 90 backward (two exponentials, a reciprocal and a root among them, which keep that unit half busy), at three of
// four a cycle; and 256 columns over 148 SMs leave an eighth of the device idle. One sequence, in clusters, waits at the
// meeting of every tile (issue at 61 % of what it could be, fp32 documents at 46 and 41). Two tokens compose as (A, B) after
// (A', B') = (A A', A B' + B), so time is cut: a CTA takes a tile of 8 tokens a warp by 32 words (a word: two bf16 channels or one of fp32), a thread eight tokens of one word.
// It reduces them to one (A, B) in registers, the warps' pairs are combined in order through shared memory, and
// each thread then finishes its eight tokens; the next tile's loads are in flight meanwhile. Where columns of
// channels are fewer than the device holds CTAs, the CTAs of a cluster take the tiles of a column in turn and exchange
// one pair a tile through each other's shared memory. Everything is added in a fixed order.
//
// Backward. With g_t = dL/dh_t and G_t = a_t g_t,
//     g_t = dy_t + G_{t+1},   dx = g w sig(i),   di = dx x (1 - sig(i)),
//     power:  l = log a:  l dL/dl = g (a l h_{t-1} - u a^2 l / w),  dr = (1 - sig(r)) l dL/dl,
//             dd = sum l dL/dl sig(d) / softplus(d)      (l / w -> 0 as l -> 0: no singularity is left)
//     lerp:   dr = g (h_{t-1} - u) a w,  dd = sum dr
// in tiles from the last one back. The forward's states before every eighth token (marks, half a byte for each element)
// give each thread its h: only G is composed, h is not rounded and nothing is read twice. A thread finds the
// decays first (for G), then g from its last token back, then h and the gradients from its first token on.
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

constexpr int kTok = 8;                             // tokens of a thread
// Warps of a CTA. Forward: 16 in two CTAs an SM (8 in three: 83 us against 73 for 4 x 2048 x 4096 bf16), 12 where the
// cluster's exchange shares the room; backward: what 128 registers a thread leave two CTAs of.
constexpr int kFwdWarps = 16, kFwdClusterWarps = 12, kBwdWarps = 8, kStepWarps = 8;
constexpr int kMaxRanks = 8;
static_assert(kTok == M3_GS_BLOCK, "a mark for every thread of a tile");

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
    float* marks;               // [nb][blocks][C] or null
    float* part;                // backward: [shares][C]
    int64_t L;
    int64_t nb;                 // batch entries (packed: 1)
    int nseq, C, cols, ranks, blocks, shares;
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
// An element at a time, never contracted, so that every form of a kernel rounds alike. (Pairs in one instruction saved
// arithmetic and cost as many moves: training step of 4 x 2048 x 4096 222 us against 209.)
__device__ __forceinline__ float mul2(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ float add2(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 mul2(const float2& a, const float2& b) { return make_float2(__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y)); }
__device__ __forceinline__ float2 add2(const float2& a, const float2& b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }
__device__ __forceinline__ float2 fma2(const float2& a, const float2& b, const float2& c) { return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)); }
// with a constant
template <typename V>
__device__ __forceinline__ V plus(const V& v, float c) { return each(v, [=](float x) { return __fadd_rn(x, c); }); }
template <typename V>
__device__ __forceinline__ V times(const V& v, float c) { return each(v, [=](float x) { return __fmul_rn(x, c); }); }
template <typename V>
__device__ __forceinline__ V less_from(const V& v, float c) { return each(v, [=](float x) { return __fadd_rn(c, -x); }); }   // c - v
// c - a b
__device__ __forceinline__ float less2(float a, float b, float c) { return fmaf(-a, b, c); }
__device__ __forceinline__ float2 less2(const float2& a, const float2& b, const float2& c) {
    return make_float2(fmaf(-a.x, b.x, c.x), fmaf(-a.y, b.y, c.y));
}
// a b - c
__device__ __forceinline__ float minus_fma(float a, float b, float c) { return fmaf(a, b, -c); }
__device__ __forceinline__ float2 minus_fma(const float2& a, const float2& b, const float2& c) {
    return make_float2(fmaf(a.x, b.x, -c.x), fmaf(a.y, b.y, -c.y));
}
__device__ __forceinline__ float minus(float a, float b) { return __fadd_rn(a, -b); }
__device__ __forceinline__ float2 minus(const float2& a, const float2& b) { return make_float2(__fadd_rn(a.x, -b.x), __fadd_rn(a.y, -b.y)); }

// The hardware's 2^x, 1 / x and 1 / sqrt(x); the bounds keep NaN.
__device__ __forceinline__ float hw_ex2(float v) { asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v)); return v; }
__device__ __forceinline__ float hw_rcp(float v) { asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(v)); return v; }
__device__ __forceinline__ float hw_rsqrt(float v) { asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(v)); return v; }
__device__ __forceinline__ float at_least(float v, float b) { asm("max.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(b)); return v; }

// The same value, which the compiler takes for another: what follows from it is worked out again, not kept.
__device__ __forceinline__ float apart(float v) { asm("" : "+f"(v)); return v; }
__device__ __forceinline__ float2 apart(const float2& v) { return make_float2(apart(v.x), apart(v.y)); }

constexpr float kLog2e = 1.4426950408889634f;
// A sigmoid's argument is taken to be at least -43 (NaN stays): then (1 + e^-r)(1 + e^-i) is finite, and a sigmoid ends at 2^-62
// instead of at zero. For a pair of bf16 that is one instruction.
constexpr float kLeast = -43.f;
__device__ __forceinline__ float unpacked(float, uint32_t w) { return Word<float>::unpack(w); }
__device__ __forceinline__ float2 unpacked(const float2&, uint32_t w) { return Word<__nv_bfloat16>::unpack(w); }
__device__ __forceinline__ float bounded(float, uint32_t w) { return at_least(__uint_as_float(w), kLeast); }
__device__ __forceinline__ float2 bounded(const float2&, uint32_t w) {
    uint32_t v;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(w), "r"(0xc22cc22cu));       // bf16 -43 twice
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <typename V>
__device__ __forceinline__ V exp_neg(const V& v) { return each(times(v, -kLog2e), hw_ex2); }

constexpr float kSeries = 0.125f;

// r's part: e^-r, a and n = 1 - a. k: power: power softplus(d), the largest -log a; lerp: d. kSmall: k <= kSeries, the
// series of 1 - e^-t alone serves (the next term is kSeries^5 / 6! = 4e-8 of the first); otherwise e^-t from
// the hardware's 2^x where t is larger: there that is a, and n what is left of one (as one less n, an a of e^-16 would keep
// no digits). Just above kSeries 2^x costs n some digits: w is measured within 9 units of 2^-24 there, 3.4 below and from one half
// on. t = -log a is taken 1e-30 higher, so that w is not zero where sig(r) is.
__device__ __forceinline__ float decay_of(float sr, float k) { return fmaf(k, sr, 1e-30f); }
__device__ __forceinline__ float2 decay_of(const float2& sr, const float2& k) { return make_float2(decay_of(sr.x, k.x), decay_of(sr.y, k.y)); }
__device__ __forceinline__ float series(float t) {      // t (1 - t/2 (1 - t/3 (1 - t/4 (1 - t/5))))
    float s = fmaf(t, 1.f / 120.f, -1.f / 24.f);
    s = fmaf(t, s, 1.f / 6.f);
    s = fmaf(t, s, -0.5f);
    s = fmaf(t, s, 1.f);
    return __fmul_rn(t, s);
}
// a of t, given n where the series has it (kSmall: everywhere)
template <bool kSmall>
__device__ __forceinline__ float a_of(float t, float n) {
    const float a = __fadd_rn(1.f, -n);
    return !kSmall && t > kSeries ? hw_ex2(__fmul_rn(t, -kLog2e)) : a;
}
template <bool kSmall>
__device__ __forceinline__ float2 a_of(const float2& t, const float2& n) { return make_float2(a_of<kSmall>(t.x, n.x), a_of<kSmall>(t.y, n.y)); }
// n of t, given a where that is 2^x
template <bool kSmall>
__device__ __forceinline__ float n_of(float t, float a) { return !kSmall && t > kSeries ? __fadd_rn(1.f, -a) : series(t); }
template <bool kSmall>
__device__ __forceinline__ float2 n_of(const float2& t, const float2& a) { return make_float2(n_of<kSmall>(t.x, a.x), n_of<kSmall>(t.y, a.y)); }
// 1 / p from the hardware's, which leans by a quarter of 2^-24 where p is near one: a convex decay is that at every token, and
// a memory of thousands adds it up. One step of Newton's leaves roundings alone.
template <typename V>
__device__ __forceinline__ V settled(const V& s, const V& p) { return fma2(s, less2(p, s, splat<V>(1.f)), s); }
template <bool kLerp, typename V>
__device__ __forceinline__ V exp_r(uint32_t rw, const V& k) {
    if (!kLerp) return exp_neg(bounded(k, rw));
    // (only the sum is bounded: r alone may lie far below where the bias lifts it)
    return exp_neg(each(add2(unpacked(k, rw), k), [](float v) { return at_least(v, kLeast); }));
}
// The decay and the weighted input of one token.
template <bool kLerp, bool kGate, bool kSmall, typename V>
__device__ __forceinline__ void gates(uint32_t rw, uint32_t iw, const V& x, const V& k, V* a, V* add) {
    const V er = exp_r<kLerp>(rw, k), pi = plus(er, 1.f);
    V sr, u = x;
    if (kGate) {        // one reciprocal for both sigmoids
        const V ei = exp_neg(bounded(k, iw)), pr = plus(ei, 1.f), R = each(mul2(pr, pi), hw_rcp);
        sr = mul2(pr, R);
        u = mul2(u, mul2(pi, R));
    } else {
        sr = each(pi, hw_rcp);
    }
    if (kLerp) {
        *a = settled(sr, pi);
        *add = mul2(mul2(er, sr), u);
        return;
    }
    // 1 - a^2 = n (1 + a): no digits are lost for a near 1
    const V t = decay_of(sr, k);
    *a = a_of<kSmall>(t, each(t, series));
    const V n = n_of<kSmall>(t, *a);
    const V q = fma2(n, *a, n);
    *add = mul2(mul2(q, each(q, hw_rsqrt)), u);
}

// softplus(d) = log(1 + e^d)
__device__ __forceinline__ float softplus(float d) { return d > 20.f ? d : log1pf(expf(d)); }

// The warp's index, the same in every lane for the compiler too: what follows from it (rows, addresses) is then worked out
// once a warp. (Forward 742 -> 724 us for 65536 x 4096; the backward, which has more of it, loses 5 %.)
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0); }

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
    // whether the channels that exist are all below (NaN is not)
    __device__ __forceinline__ bool below(const V& v, float most) const {
        if constexpr (W::E == 1) return !ok || v <= most;
        else return (!ok || v.x <= most) && (!two || v.y <= most);
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
template <int kTile>
struct Rows {
    uint32_t start[kTile / 32], end[kTile / 32];
    int seq[kTile];
};

// Rows of the packed tensor that hold tokens.
__device__ __forceinline__ void packed_span(const GsParams& p, int* first, int* last) {
    const int L = static_cast<int>(p.L), f = p.nseq > 0 ? __ldg(p.cu) : 0, l = p.nseq > 0 ? __ldg(p.cu + p.nseq) : 0;
    *first = min(max(f, 0), L);
    *last = min(max(l, *first), L);
}

// the first kTile threads: the sequence of one row each, by halves (the last that begins at or before it)
template <int kTile>
__device__ __forceinline__ void find_rows(const GsParams& p, Rows<kTile>& rows, int tile, int last) {
    if (threadIdx.x >= kTile) return;
    const int row = tile * kTile + static_cast<int>(threadIdx.x);
    int lo = 0, hi = p.nseq;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (__ldg(p.cu + m) <= row) lo = m;
        else hi = m;
    }
    const int s = __ldg(p.cu + lo), e = __ldg(p.cu + lo + 1);
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
template <int n>
__device__ __forceinline__ uint32_t mine(const uint32_t (&m)[n], int w) { return (m[w >> 2] >> (8 * (w & 3))) & 0xffu; }

// a sequence without tokens ends in the state it begins with
template <int kWarps, typename Col>
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

// Tiles of the input tensors. kMode 2 (rows of whole 16-byte words) and 1 (of whole words): rows of 128 bytes in
// shared memory, brought by asynchronous copies while other tiles are worked on; 0: each thread's own words in its
// registers, a tile ahead.
constexpr int kRowBytes = 128;
template <typename T, int kMode, int kTensors, int kWarps>
struct Tiles {
    static constexpr bool kVec = kMode >= 1, kStaged = kMode >= 1;
    static constexpr int kTile = kWarps * kTok, kTileBytes = kTile * kRowBytes, kPass = kTile / 2;    // rows of one copy a thread
    using Col = Column<T, kVec>;
    const T* next[kTensors];        // this thread's place in the tile to come: its 16 bytes of the first row (mode 2), its first word
    const T* first[kMode == 1 ? kTensors : 1];      // a place that can be read
    int64_t token[kTensors], step;  // step: rows from tile to tile
    uint32_t raw[kStaged ? 1 : kTensors][kStaged ? 1 : kTok];
    uint8_t* room;
    const Col& k;
    int chunk_bytes, warp, lane;
    // step: tiles from one to the next
    __device__ __forceinline__ Tiles(const Col& col, int column, int C, uint8_t* smem, int tiles, int warp_) : step(static_cast<int64_t>(tiles) * kTile), room(smem), k(col) {
        warp = warp_;
        lane = threadIdx.x & 31;
        const int c = column * 32 * Word<T>::E + static_cast<int>(threadIdx.x & 7) * (16 / static_cast<int>(sizeof(T)));
        chunk_bytes = c < C ? 16 : 0;
    }
    // tensor n, from this tile on
    __device__ __forceinline__ void set(int n, const GsTensor& t, int64_t b, int column, int64_t tile) {
        token[n] = t.token;
        const T* base = static_cast<const T*>(t.p) + b * t.batch;
        if (kMode == 1) first[kMode == 1 ? n : 0] = base;
        if (kMode == 2)
            next[n] = base + column * 32 * Word<T>::E + (chunk_bytes ? threadIdx.x & 7u : 0u) * (16 / sizeof(T)) +
                      (tile * kTile + (threadIdx.x >> 3)) * t.token;
        else
            next[n] = base + k.c + (tile * kTile + warp * kTok) * t.token;
    }
    // the rows of the tile to come, `rows` of which hold tokens, into a slot
    __device__ __forceinline__ void fetch(int rows, int slot) {
        if constexpr (kMode == 2) {
            const int r = threadIdx.x >> 3;
            const uint32_t dst = sm100::smem_u32(room + slot * kTensors * kTileBytes + threadIdx.x * 16);
            if (rows == kTile) {
#pragma unroll
                for (int n = 0; n < kTensors; ++n) {
                    copy(dst + n * kTileBytes, next[n], chunk_bytes);
                    copy(dst + n * kTileBytes + kTileBytes / 2, next[n] + kPass * token[n], chunk_bytes);
                }
            } else if (rows > 0) {      // (a row without a token is zero, read from the tile's first)
#pragma unroll
                for (int n = 0; n < kTensors; ++n)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const bool live = r + half * kPass < rows;
                        copy(dst + n * kTileBytes + half * (kTileBytes / 2), next[n] + (live ? half * kPass : -r) * token[n], live ? chunk_bytes : 0);
                    }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else if constexpr (kMode == 1) {
            const uint32_t dst = sm100::smem_u32(room + slot * kTensors * kTileBytes + warp * kTok * kRowBytes + lane * 4);
            const int mine = k.ok ? rows - warp * kTok : 0;
#pragma unroll
            for (int n = 0; n < kTensors; ++n) {
                const T* q = next[n];
#pragma unroll
                for (int j = 0; j < kTok; ++j, q += token[n])       // (past the last token: zero, read from nowhere)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + n * kTileBytes + j * kRowBytes),
                                 "l"(j < mine ? q : first[n]), "r"(j < mine ? 4 : 0) : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else {
#pragma unroll
            for (int n = 0; n < kTensors; ++n)
#pragma unroll
                for (int j = 0; j < kTok; ++j) raw[n][j] = k.load(next[n] + j * token[n], k.ok && warp * kTok + j < rows);
        }
#pragma unroll
        for (int n = 0; n < kTensors; ++n) next[n] += step * token[n];
    }
    static __device__ __forceinline__ void copy(uint32_t dst, const T* src, int bytes) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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
template <int kMost>
__device__ __forceinline__ int clamp_to(int n) { return min(max(n, 0), kMost); }

template <bool k>
struct Is {
    static constexpr bool value = k;
};
template <typename F>
__device__ __forceinline__ void branch(bool b, F&& f) {
    if (b) f(Is<true>{});
    else f(Is<false>{});
}

// ---- the exchange of a cluster

// a tile's pair into rank `to`'s shared memory
template <typename V>
__device__ __forceinline__ void send(Pair<V>* place, const Pair<V>& pair, int* reset, bool cut, int to) {
    cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
    *cl.map_shared_rank(place, to) = pair;
    if ((threadIdx.x & 31) == 0) *cl.map_shared_rank(reset, to) = cut;
}
// Every CTA's pairs are sent. Only the warps that sent release what they wrote: that waits for all of a
// warp's stores, the outputs' too.
__device__ __forceinline__ void meet(bool sent) {
    __syncwarp();
    if (sent) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    else asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- forward

constexpr int fwd_warps(bool cluster) { return cluster ? kFwdClusterWarps : kFwdWarps; }

template <typename T, bool kLerp, bool kGate, bool kPacked, int kMode, bool kCluster>
__global__ void __launch_bounds__(32 * fwd_warps(kCluster), kMode >= 1 ? 2 : 1) gs_fwd_kernel(const __grid_constant__ GsParams p) {
    constexpr bool kVec = kMode >= 1, kStaged = kMode >= 1;
    constexpr int kTensors = kGate ? 3 : 2, kWarps = fwd_warps(kCluster), kTile = kWarps * kTok;
    using Col = Column<T, kVec>;
    using V = typename Col::V;
    __shared__ Pair<V> s_warp[2][kWarps][32];
    __shared__ V s_carry[2][kCluster ? 1 : 32];     // the state behind a tile
    __shared__ Pair<V> s_rank[kCluster ? 2 : 1][kCluster ? kMaxRanks : 1][32];
    __shared__ int s_reset[2][kMaxRanks];
    __shared__ Rows<kTile> s_rows[kPacked ? 3 : 1];
    extern __shared__ __align__(16) uint8_t s_tiles[];
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int ranks = kCluster ? p.ranks : 1;
    const int rank = kCluster ? static_cast<int>(blockIdx.x % ranks) : 0;
    const int64_t unit = kCluster ? blockIdx.x / ranks : blockIdx.x;
    const int64_t b = unit / p.cols;
    const int column = static_cast<int>(unit - b * p.cols);
    const Col k(p, column);
    int first = 0, last = static_cast<int>(p.L);       // (up to 2^30: rows are counted in 32 bits)
    if (kPacked) packed_span(p, &first, &last);
    const int tiles = (last + kTile - 1) / kTile, steps = (tiles + ranks - 1) / ranks;

    Tiles<T, kMode, kTensors, kWarps> in(k, column, p.C, s_tiles, ranks, warp);
    in.set(0, p.x, b, column, rank);
    in.set(1, p.r, b, column, rank);
    if constexpr (kGate) in.set(2, p.i, b, column, rank);
    const auto fetch = [&](int tile, int slot) { in.fetch(clamp_to<kTile>(last - tile * kTile), slot); };
    if (steps > 0) {
        fetch(rank, 0);
        if (kStaged) fetch(rank + ranks, 1);
    }

    const V d = k.param(p.decay);
    const V kd = kLerp ? d : each(d, [&](float v) { return p.power * softplus(v); });
    const bool small = kLerp || __all_sync(0xffffffffu, k.below(kd, kSeries));
    if (kPacked && p.final_state) empty_sequences<kWarps>(p, k, rank, p.init, p.final_state);
    V carry = splat<V>(0.f);
    if (!kPacked && p.init) carry = k.get(p.init + b * p.C);
    if (!kCluster && warp == 0) s_carry[0][lane] = carry;
    if (kPacked) find_rows(p, s_rows[0], rank, last);
    in.template wait<1>();
    if (kStaged || kPacked) __syncthreads();
    if (kCluster) meet(false);      // every CTA of the cluster runs

    T* py = p.y.p ? static_cast<T*>(p.y.p) + b * p.y.batch : nullptr;
    int rb = 0;
    for (int step = 0; step < steps; ++step) {
        const int tile = step * ranks + rank, t0 = tile * kTile + warp * kTok, buf = step & 1;
        Rows<kTile>& rows = s_rows[kPacked ? rb : 0];
        uint32_t st = 0;
        V a[kTok], h[kTok];
        if (kPacked) {
            st = mine(rows.start, warp);
            rb = rb == 2 ? 0 : rb + 1;
        }
        branch(small, [&](auto is_small) {
#pragma unroll
            for (int j = 0; j < kTok; ++j)
                gates<kLerp, kGate, decltype(is_small)::value>(in.word(buf, 1, j), kGate ? in.word(buf, kTensors - 1, j) : 0u,
                                                               Word<T>::unpack(in.word(buf, 0, j)), kd, &a[j], &h[j]);
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
        if (kPacked) find_rows(p, s_rows[rb], tile + ranks, last);
        in.template wait<0>();      // the next tile
        __syncthreads();
        // (into this tile's slot, which every thread has read)
        if (kStaged) fetch(tile + 2 * ranks, buf);
        V before;       // the state before the tile, then before this thread's tokens
        if (!kCluster) {
            before = s_carry[buf][lane];
        } else {
            if (warp < ranks) {         // one warp for each rank sends it the tile's pair
                V pa = splat<V>(1.f), pb = splat<V>(0.f);
                bool cut = false;
#pragma unroll 4
                for (int w = 0; w < kWarps; ++w) {
                    const Pair<V> q = s_warp[buf][w][lane];
                    const V n = fma2(q.a, pb, q.b);
                    const bool c = kPacked && mine(rows.start, w);
                    pb = c ? q.b : n;
                    pa = mul2(pa, q.a);
                    cut = cut || c;
                }
                send(&s_rank[buf][rank][lane], Pair<V>{pa, pb}, &s_reset[buf][rank], cut, warp);
            }
            meet(warp < ranks);
            for (int r = 0; r < ranks; ++r) {
                if (r == rank) before = carry;
                const Pair<V> q = s_rank[buf][r][lane];
                const V n = fma2(q.a, carry, q.b);
                carry = kPacked && s_reset[buf][r] ? q.b : n;
            }
        }
#pragma unroll
        for (int w = 0; w < kWarps - 1; ++w) {
            if (w >= warp) break;
            const Pair<V> q = s_warp[buf][w][lane];
            const V n = fma2(q.a, before, q.b);
            before = kPacked && mine(rows.start, w) ? q.b : n;
        }
        const Live live{clamp_to<kTok>(first - t0), clamp_to<kTok>(last - t0)};
        if (p.marks && live.hi > 0) k.put(p.marks + (b * p.blocks + (tile * kWarps + warp)) * p.C, before);
#pragma unroll
        for (int j = 0; j < kTok; ++j) {
            const V n = fma2(a[j], before, h[j]);
            h[j] = kPacked && (st & ((2u << j) - 1)) ? h[j] : n;
        }
        if (!kCluster && warp == kWarps - 1) s_carry[buf ^ 1][lane] = h[kTok - 1];
        if (py && k.ok) {
            T* to = py + static_cast<int64_t>(t0) * p.y.token;
            if (live.all()) {
#pragma unroll
                for (int j = 0; j < kTok; ++j) k.store(to + j * p.y.token + k.c, h[j]);
            } else {
#pragma unroll
                for (int j = 0; j < kTok; ++j)
                    if (live(j)) k.store(to + j * p.y.token + k.c, h[j]);
            }
        }
        if (p.final_state) {
            const uint32_t en = kPacked ? mine(rows.end, warp) : 0u;
            if (kPacked && en) {
#pragma unroll
                for (int j = 0; j < kTok; ++j)
                    if (en >> j & 1) k.put(p.final_state + static_cast<int64_t>(rows.seq[warp * kTok + j]) * p.C, h[j]);
            }
            if (!kPacked && live.hi > 0 && last <= t0 + kTok) {
#pragma unroll
                for (int j = 0; j < kTok; ++j)
                    if (t0 + j == last - 1) k.put(p.final_state + b * p.C, h[j]);
            }
        }
    }
    in.template wait<0>();
    // (no token at all: the state stays)
    if (!kPacked && steps == 0 && rank == 0 && warp == 0 && p.final_state) k.put(p.final_state + b * p.C, carry);
}

// ---- backward

template <typename T, bool kLerp, bool kGate, bool kPacked, int kMode, bool kCluster>
__global__ void __launch_bounds__(32 * kBwdWarps, 2) gs_bwd_kernel(const __grid_constant__ GsParams p) {
    constexpr bool kVec = kMode >= 1, kStaged = kMode >= 1;
    constexpr int kTensors = kGate ? 4 : 3, kWarps = kBwdWarps, kTile = kWarps * kTok;
    using Col = Column<T, kVec>;
    using V = typename Col::V;
    __shared__ Pair<V> s_warp[2][kWarps][32];
    __shared__ V s_carry[2][32];            // G before a tile
    __shared__ Pair<V> s_rank[kCluster ? 2 : 1][kCluster ? kMaxRanks : 1][32];
    __shared__ int s_reset[2][kMaxRanks];
    __shared__ Rows<kTile> s_rows[kPacked ? 3 : 1];
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
    if (kCluster) meet(false);  // every CTA of the cluster runs
    int first = 0, last = static_cast<int>(p.L);       // (up to 2^30: rows are counted in 32 bits)
    if (kPacked) packed_span(p, &first, &last);
    const int tiles = (last + kTile - 1) / kTile, steps = (tiles + ranks - 1) / ranks;

    const V d = k.param(p.decay);
    const V kd = kLerp ? d : each(d, [&](float v) { return p.power * softplus(v); });
    const bool small = kLerp || __all_sync(0xffffffffu, k.below(kd, kSeries));
    if (kPacked && p.dinit) empty_sequences<kWarps>(p, k, rank, p.dfinal, p.dinit);
    V sum = splat<V>(0.f);
    int tick = 0;               // which of the two exchange buffers is next, across sequences
    const V zero = splat<V>(0.f);
    Tiles<T, kMode, kTensors, kWarps> in(k, column, p.C, s_tiles, -ranks, warp);

    for (int64_t b = share; b < p.nb; b += p.shares) {
        in.set(0, p.x, b, column, tiles - 1 - rank);
        in.set(1, p.r, b, column, tiles - 1 - rank);
        in.set(2, p.dy, b, column, tiles - 1 - rank);
        if constexpr (kGate) in.set(3, p.i, b, column, tiles - 1 - rank);
        V mark = zero;
        const auto fetch = [&](int tile, int slot) { in.fetch(tile < 0 ? 0 : clamp_to<kTile>(last - tile * kTile), slot); };
        const auto get_mark = [&](int tile) {       // the state before this thread's tokens
            const int block = tile * kWarps + warp;
            mark = tile >= 0 && block * kTok < last ? k.get(p.marks + (b * p.blocks + block) * p.C) : zero;
        };
        T *qx = static_cast<T*>(p.dx.p) + b * p.dx.batch + k.c, *qr = static_cast<T*>(p.dr.p) + b * p.dr.batch + k.c;
        T* qi = kGate ? static_cast<T*>(p.di.p) + b * p.di.batch + k.c : nullptr;
        if (steps > 0) {
            fetch(tiles - 1 - rank, 0);
            if (kStaged) fetch(tiles - 1 - rank - ranks, 1);
        }
        get_mark(tiles - 1 - rank);
        int rb = 0, slot = 0;
        if (kPacked) find_rows(p, s_rows[0], tiles - 1 - rank, last);
        if (!kCluster && warp == 0) s_carry[tick][lane] = zero;
        in.template wait<1>();
        __syncthreads();
        V carry = zero;         // G behind the tiles done so far (set where a sequence ends)
        // Every warp of the cluster has the same channels and takes the same way. Small decays are kept as n, which saves an
        // instruction each; others as a (4 x 2048 x 4096 bf16, all of one sort: 135 and 142 us).
        branch(small, [&](auto is_small) {
            constexpr bool kSmall = decltype(is_small)::value, kHaveA = kLerp || !kSmall;
            for (int step = 0; step < steps; ++step) {
                const int tile = tiles - 1 - step * ranks - rank, t0 = tile * kTile + warp * kTok;
                const int buf = tick;
                tick ^= 1;
                Rows<kTile>& rows = s_rows[kPacked ? rb : 0];
                // rows that begin and end a sequence: bits of the thread's tokens
                uint32_t st, en;
                const int tail = tile >= 0 && last - 1 - tile * kTile < kTile ? last - 1 - tile * kTile : -1;
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
                const Live live{clamp_to<kTok>(first - t0), tile >= 0 ? clamp_to<kTok>(last - t0) : 0};
                const bool plain = st == 0 && en == 0 && live.all();
                const auto seq = [&](int j) { return kPacked ? static_cast<int64_t>(rows.seq[warp * kTok + j]) : b; };
                const auto gin = [&](int j) { return p.dfinal ? k.get(p.dfinal + seq(j) * p.C) : zero; };
                // e^-r and the decays (kSmall: n, else a), then their product and G from zero
                V er[kTok], c[kTok];
#pragma unroll
                for (int j = 0; j < kTok; ++j) {
                    er[j] = exp_r<kLerp>(in.word(slot, 1, j), kd);
                    const V p = plus(er[j], 1.f);
                    c[j] = each(p, hw_rcp);
                    if (kLerp) {
                        c[j] = settled(c[j], p);
                    } else {
                        const V t = decay_of(c[j], kd), n = each(t, series);
                        c[j] = kSmall ? n : a_of<kSmall>(t, n);
                    }
                }
                const auto a = [&](int j) { return kHaveA ? c[j] : less_from(c[j], 1.f); };
                const auto decayed = [&](int j, const V& v) { return kHaveA ? mul2(c[j], v) : less2(c[j], v, v); };
                V pa = a(0), pg = zero;
#pragma unroll
                for (int j = 1; j < kTok; ++j) pa = decayed(j, pa);
#pragma unroll
                for (int j = kTok - 1; j >= 0; --j) {
                    if (!plain && (en >> j & 1)) pg = gin(j);
                    pg = decayed(j, add2(Word<T>::unpack(in.word(slot, 2, j)), pg));
                }
                s_warp[buf][warp][lane] = Pair<V>{pa, pg};
                if (kPacked) find_rows(p, s_rows[rb], tile - ranks, last);
                in.template wait<0>();      // the next tile
                __syncthreads();
                // (into the slot of the tile before, which every thread has done with)
                const int next = slot == 2 ? 0 : slot + 1;
                if (kStaged) fetch(tile - 2 * ranks, next == 2 ? 0 : next + 1);
                V hp = mark;
                get_mark(tile - ranks);
                V G;                // G behind the tile, then behind this thread's tokens
                if (!kCluster) {
                    G = s_carry[buf][lane];
                } else {
                    if (warp < ranks) {
                        V ca = splat<V>(1.f), cb = zero;
                        bool cut = false;
#pragma unroll
                        for (int w = kWarps - 1; w >= 0; --w) {
                            const Pair<V> q = s_warp[buf][w][lane];
                            const V m = fma2(q.a, cb, q.b);
                            const bool at_end = ends(w) != 0;
                            cb = at_end ? q.b : m;
                            ca = mul2(ca, q.a);
                            cut = cut || at_end;
                        }
                        send(&s_rank[buf][rank][lane], Pair<V>{ca, cb}, &s_reset[buf][rank], cut, warp);
                    }
                    meet(warp < ranks);
                    for (int r = 0; r < ranks; ++r) {
                        if (r == rank) G = carry;
                        const Pair<V> q = s_rank[buf][r][lane];
                        const V m = fma2(q.a, carry, q.b);
                        carry = s_reset[buf][r] ? q.b : m;
                    }
                }
                if (!kPacked && tail < 0) {
#pragma unroll
                    for (int w = kWarps - 1; w > 0; --w) {
                        if (w <= warp) break;
                        const Pair<V> q = s_warp[buf][w][lane];
                        G = fma2(q.a, G, q.b);
                    }
                } else {
#pragma unroll 1
                    for (int w = kWarps - 1; w > warp; --w) {
                        const Pair<V> q = s_warp[buf][w][lane];
                        const V m = fma2(q.a, G, q.b);
                        G = ends(w) ? q.b : m;
                    }
                }
                // g of each token from the last one back
                V g[kTok];
#pragma unroll
                for (int j = kTok - 1; j >= 0; --j) {
                    if (!plain && (en >> j & 1)) G = gin(j);
                    g[j] = add2(Word<T>::unpack(in.word(slot, 2, j)), G);
                    G = decayed(j, g[j]);
                    if (!plain && (st >> j & 1) && tile >= 0 && p.dinit) k.put(p.dinit + seq(j) * p.C, G);
                }
                if (!kCluster && warp == 0) s_carry[buf ^ 1][lane] = G;
                // h and the gradients from the first token on (words in registers leave no room for both ways of large decays)
                const int64_t row0 = t0;
                T *tx = qx + row0 * p.dx.token, *tr = qr + row0 * p.dr.token, *ti = kGate ? qi + row0 * p.di.token : nullptr;
                branch((kStaged || kSmall) && plain, [&](auto is_plain) {
                    constexpr bool kPlain = decltype(is_plain)::value;
#pragma unroll
                    for (int j = 0; j < kTok; ++j) {
                        if (!kPlain && kPacked && (st >> j & 1)) hp = p.init ? k.get(p.init + seq(j) * p.C) : zero;
                        const V x = Word<T>::unpack(in.word(slot, 0, j)), pi = plus(kGate ? er[j] : apart(er[j]), 1.f);
                        V sr, si, ci, u = x;
                        if (kGate) {
                            const V ei = exp_neg(bounded(kd, in.word(slot, kTensors - 1, j))), pr = plus(ei, 1.f);
                            const V R = each(mul2(pr, pi), hw_rcp);
                            sr = mul2(pr, R);
                            si = mul2(pi, R);
                            ci = mul2(ei, si);
                            u = mul2(x, si);
                        } else {
                            sr = kLerp ? c[j] : each(pi, hw_rcp);
                        }
                        const V aj = a(j), cr = mul2(er[j], sr);
                        V w, dr, dl;
                        if (kLerp) {
                            w = cr;
                            dl = dr = mul2(mul2(g[j], minus(hp, u)), mul2(aj, w));
                        } else {
                            // with t = -log a: l dL/dl = g a t (u a / w - h)
                            const V t = decay_of(sr, kd), n = kSmall ? c[j] : n_of<kSmall>(t, aj);
                            const V q = fma2(n, aj, n), rs = each(q, hw_rsqrt);
                            w = mul2(q, rs);
                            dl = mul2(mul2(mul2(g[j], aj), t), minus_fma(mul2(u, aj), rs, hp));
                            dr = mul2(dl, cr);
                        }
                        hp = fma2(aj, hp, mul2(w, u));
                        const V du = mul2(g[j], w), dx = kGate ? mul2(du, si) : du;
                        if (kPlain || live(j)) {
                            sum = add2(sum, dl);
                            if (k.ok) {
                                k.store(tx + j * p.dx.token, dx);
                                k.store(tr + j * p.dr.token, dr);
                                if (kGate) k.store(ti + j * p.di.token, mul2(mul2(dx, x), ci));
                            }
                        }
                    }
                });
                if (!kStaged) fetch(tile - ranks, 0);
                slot = next;
            }
        });
        in.template wait<0>();
        __syncthreads();        // the next sequence's rows, tiles and pairs
        if (!kPacked && steps == 0 && rank == 0 && warp == 0 && p.dinit)
            k.put(p.dinit + b * p.C, p.dfinal ? k.get(p.dfinal + b * p.C) : zero);
    }
    if (!p.part) return;
    s_warp[0][warp][lane].a = sum;
    __syncthreads();
    if (warp != 0) return;
    V total = zero;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total = add2(total, s_warp[0][w][lane].a);
    if (!kLerp)         // dlog a / dd = log a sig(d) / softplus(d); both go to zero together
        total = mul2(total, each(d, [](float v) {
            const float s = softplus(v);
            return v < -15.f ? 1.f : 1.f / (s * (1.f + expf(-v)));
        }));
    k.put(p.part + (static_cast<int64_t>(share) * ranks + rank) * p.C, total);
}

// ---- one token

template <typename T, bool kLerp, bool kGate, bool kVec>
__global__ void __launch_bounds__(32 * kStepWarps) gs_step_kernel(const __grid_constant__ GsParams p, const int32_t* __restrict__ slots,
                                                           int64_t nstates) {
    using W = Word<T>;
    using V = typename W::V;
    using Col = Column<T, kVec>;
    // a warp takes 32 words of one sequence
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kStepWarps + (threadIdx.x >> 5);
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
        const V kd = kLerp ? d : each(d, [&](float v) { return p.power * softplus(v); });
        V a, add;
        gates<kLerp, kGate, false>(rr, ri, W::unpack(rx), kd, &a, &add);
        h = fma2(a, k.get(p.init + slot * p.C), add);
        k.put(p.final_state + slot * p.C, h);
    }
    if (k.ok) k.store(at<T>(p.y, b, k.c), h);
}

// ---- launches

template <typename... P, typename... Args>
cudaError_t launch(void (*kernel)(P...), int64_t grid, int threads, int ranks, int smem, bool after, cudaStream_t s, const Args&... args) {
    if (ranks == 1 && !after) {
        kernel<<<static_cast<unsigned>(grid), threads, smem, s>>>(args...);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
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
// 2: copied by 16 bytes; 1: by words of two bf16 or one fp32; 0: loaded an element at a time
template <typename T>
int mode_of(const GsParams& p) {
    constexpr int es = sizeof(T);
    return rows_of(p, es, 16) ? 2 : es == 4 || rows_of(p, es, 4) ? 1 : 0;
}

// CTAs of a column: as many as there is room for beside the other columns.
constexpr int kPerSm = 2;       // of the backward
int64_t bwd_tiles(int64_t L) { return (L + kBwdWarps * kTok - 1) / (kBwdWarps * kTok); }
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
    p.ranks = rank_count(p.nb * p.cols, (p.L + kFwdClusterWarps * kTok - 1) / (kFwdClusterWarps * kTok), mode >= 1 ? 2 : 1);
    return with_mode<T>(mode, [&](auto m) {
        return with_bools<>([&](auto f) {
            using F = decltype(f);
            constexpr int kMode = decltype(m)::value;
            constexpr auto kernel = gs_fwd_kernel<T, F::template at<0>(), F::template at<1>(), F::template at<2>(), kMode, F::template at<3>()>;
            constexpr int warps = fwd_warps(F::template at<3>());
            constexpr int smem = kMode >= 1 ? 2 * (F::template at<1>() ? 3 : 2) * warps * kTok * kRowBytes : 0;
            const cudaError_t e = staged_smem<kernel>(smem);
            return e != cudaSuccess ? e : launch(kernel, p.nb * p.cols * p.ranks, 32 * warps, p.ranks, smem, false, s, p);
        }, lerp, p.i.p != nullptr, p.cu != nullptr, p.ranks > 1);
    });
}

template <typename T>
cudaError_t launch_bwd(GsParams p, bool lerp, bool after, float* ddecay, cudaStream_t s) {
    p.shares = share_count(p);
    p.ranks = rank_count(static_cast<int64_t>(p.shares) * p.cols, bwd_tiles(p.L), kPerSm);
    if (!ddecay) p.part = nullptr;
    else if (p.shares * p.ranks == 1) p.part = ddecay;
    const cudaError_t e = with_mode<T>(mode_of<T>(p), [&](auto m) {
        return with_bools<>([&](auto f) {
            using F = decltype(f);
            constexpr int kMode = decltype(m)::value;
            constexpr auto kernel = gs_bwd_kernel<T, F::template at<0>(), F::template at<1>(), F::template at<2>(), kMode, F::template at<3>()>;
            constexpr int smem = kMode >= 1 ? 3 * (F::template at<1>() ? 4 : 3) * kBwdWarps * kTok * kRowBytes : 0;
            const cudaError_t e = staged_smem<kernel>(smem);
            return e != cudaSuccess ? e : launch(kernel, static_cast<int64_t>(p.shares) * p.cols * p.ranks, 32 * kBwdWarps, p.ranks, smem, after, s, p);
        }, lerp, p.i.p != nullptr, p.cu != nullptr, p.ranks > 1);
    });
    if (e != cudaSuccess || !ddecay || p.shares * p.ranks == 1) return e;
    float* const outs[1] = {ddecay};
    return launch_sum_shares(p.part, p.shares * p.ranks, p.C, outs, 1, s);
}

template <typename T>
cudaError_t launch_step(const GsParams& p, bool lerp, const int32_t* slots, int64_t nstates, cudaStream_t s) {
    const int64_t grid = (p.nb * p.cols + kStepWarps - 1) / kStepWarps;
    return with_bools<>([&](auto f) {
        using F = decltype(f);
        return launch(gs_step_kernel<T, F::template at<0>(), F::template at<1>(), F::template at<2>() || sizeof(T) == 4>, grid, 32 * kStepWarps, 1, 0, false, s,
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
    p.blocks = static_cast<int>((d->seqlen + kTok - 1) / kTok);
    p.power = d->power;
    return p;
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }
size_t marks_bytes(const m3_gated_scan_dims* d, bool packed) {
    return up(static_cast<size_t>(packed ? 1 : d->nseq) * static_cast<size_t>((d->seqlen + kTok - 1) / kTok) *
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
    const size_t part = up(static_cast<size_t>(p.shares) * rank_count(static_cast<int64_t>(p.shares) * p.cols, bwd_tiles(p.L), kPerSm) *
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
            if ((st = check_apart(*o, {x, r, i, g, df})) != M3_OK || (st = check_apart(*o, rest)) != M3_OK) return st;
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
        if (e == cudaSuccess && dinit && n)
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
