// Rotary positions of queries and keys: pair j of the first `rot` dimensions of every head is turned by
// the angle position * freq[j], the rest is copied.
//
// Bound by HBM: every element is read and written once (8192 tokens of 128 heads of 128, bf16: 85 us, 6.3 TB/s, 0.96 of
// what a copy reaches; the step of 128 sequences is launch and one chain of loads, 3.3 us). A thread takes 16 + 16 bytes of
// pairs of one token and walks over up to eight heads, so the sines are formed once for them. Angles of far positions lose their
// digits in fp32 (position 65 536 at one radian: 4e-3), so they are counted in turns, as 64-bit fractions:
// freq / 2 pi modulo one, times 2^64, multiplied by the position modulo 2^64, is the angle
// modulo one turn to 2^-54 turns a position, for any integer position and frequencies up to 2^40, without a division. The top
// 32 bits, reduced to an eighth of a turn either way, go through the series of sine and cosine.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "m3_common.cuh"
#include "m3_internal.h"
#include "m3_vec.cuh"

namespace m3 {
namespace {

constexpr int kThreads = 256, kMaxPairs = 512, kMostHeads = 8;

struct RotTensor {
    const void* in;
    void* out;
    int64_t in_batch, in_token, in_head, out_batch, out_token, out_head;
};
struct RotParams {
    RotTensor q, k;
    const double* freq;
    const void* pos;                // int32 or int64, or null
    int64_t pos_batch, pos_token, offset;
    const int32_t* cu;
    int nseq;
    uint32_t tokens, len;           // in all, and of each batch entry
    int hq, heads, per;             // heads of q, of both, of one thread
    int D, rot, turned, items;      // items of a token: those that turn pairs, and all
    int pos64;
    float scale, sign;
};

// sine and cosine of a 32-bit fraction of a turn. Up to pi / 4 the series' next terms are 2e-9 and 1.2e-10.
__device__ __forceinline__ float2 turn(uint32_t u) {
    const uint32_t q = (u + 0x20000000u) >> 30;
    const float t = static_cast<float>(static_cast<int32_t>(u - (q << 30))) * 1.4629180792671596e-9f;     // 2 pi / 2^32
    const float t2 = t * t;
    float s = fmaf(t2, 2.7557319e-6f, -1.9841270e-4f);
    s = fmaf(t2, s, 8.3333333e-3f);
    s = fmaf(t2, s, -1.6666667e-1f);
    s = fmaf(t * t2, s, t);
    float c = fmaf(t2, -2.7557319e-7f, 2.4801587e-5f);
    c = fmaf(t2, c, -1.3888889e-3f);
    c = fmaf(t2, c, 4.1666667e-2f);
    c = fmaf(t2, c, -0.5f);
    c = fmaf(t2, c, 1.f);
    if (q & 1u) {
        const float n = -s;
        s = c;
        c = n;
    }
    return q & 2u ? make_float2(-s, -c) : make_float2(s, c);
}

// PP pairs of one head: 16 + 16 bytes, or (PP = 1) an element each
template <typename T, int PP>
struct Bytes;
template <typename T>
struct Bytes<T, 1> {
    T lo, hi;
    __device__ __forceinline__ void load(const T* a, const T* b, bool, bool two) {
        lo = *a;
        if (two) hi = *b;
    }
    __device__ __forceinline__ void store(T* a, T* b, bool, bool two) const {
        *a = lo;
        if (two) *b = hi;
    }
    __device__ __forceinline__ void rotate(bool, const float (&s)[1], const float (&c)[1]) {
        const float x = to_f(lo), y = to_f(hi);
        lo = from_f<T>(fmaf(x, c[0], -(y * s[0])));
        hi = from_f<T>(fmaf(y, c[0], x * s[0]));
    }
};
template <typename T, int PP>
struct Bytes {
    uint4 lo, hi;
    __device__ __forceinline__ void load(const T* a, const T* b, bool, bool two) {
        lo = __ldcs(reinterpret_cast<const uint4*>(a));
        if (two) hi = __ldcs(reinterpret_cast<const uint4*>(b));
    }
    __device__ __forceinline__ void store(T* a, T* b, bool, bool two) const {
        __stcs(reinterpret_cast<uint4*>(a), lo);
        if (two) __stcs(reinterpret_cast<uint4*>(b), hi);
    }
    __device__ __forceinline__ void rotate(bool inter, const float (&s)[PP], const float (&c)[PP]) {
        float2 v[2][PP / 2];
        Vec<T>::unpack(lo, v[0]);
        Vec<T>::unpack(hi, v[1]);
        if (inter) {        // (x, y) side by side
#pragma unroll
            for (int j = 0; j < PP; ++j) {
                float2& e = v[j / (PP / 2)][j % (PP / 2)];
                e = make_float2(fmaf(e.x, c[j], -(e.y * s[j])), fmaf(e.y, c[j], e.x * s[j]));
            }
        } else {
#pragma unroll
            for (int j = 0; j < PP / 2; ++j) {
                const float2 sj = make_float2(s[2 * j], s[2 * j + 1]), cj = make_float2(c[2 * j], c[2 * j + 1]);
                const float2 x = v[0][j], y = v[1][j];
                v[0][j] = fma2(x, cj, mul2(mul2(y, sj), both(-1.f)));
                v[1][j] = fma2(y, cj, mul2(x, sj));
            }
        }
        alignas(16) T out[2 * PP];
        Vec<T>::store(out, v[0]);
        Vec<T>::store(out + PP, v[1]);
        lo = *reinterpret_cast<const uint4*>(out);
        hi = *reinterpret_cast<const uint4*>(out + PP);
    }
};

template <typename T, int PP, bool kInter>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotParams p) {
    __shared__ uint64_t s_turns[kMaxPairs];
    constexpr int kTwo = PP == 1 ? 1 : PP;      // elements of one of an item's two parts
    for (int j = threadIdx.x; j < p.rot / 2; j += kThreads) {
        // 1 / 2 pi in two parts, the whole turns taken off before the digits that the product lost are added
        const double f = p.freq[j], whole = f * 0.15915494309189535;
        const double lost = fma(f, -9.839338337591243e-18, fma(f, 0.15915494309189535, -whole));
        double t = (whole - rint(whole)) + lost;
        t -= rint(t);
        s_turns[j] = static_cast<uint64_t>(__double2ll_rn(t * 18446744073709551616.0));     // (one half: saturates, 2^-64 off)
    }
    __syncthreads();
    const uint32_t idx = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t tok = idx / p.items;
    const int item = static_cast<int>(idx - tok * p.items);
    if (tok >= p.tokens) return;
    const uint32_t b = p.len == p.tokens ? 0u : tok / p.len, t = tok - b * p.len;
    int64_t pos;
    if (p.cu) {     // the last sequence that begins at or before this row
        int lo = 0, hi = p.nseq;
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (static_cast<int64_t>(__ldg(p.cu + m)) <= t) lo = m;
            else hi = m;
        }
        const int64_t s = __ldg(p.cu + lo), e = __ldg(p.cu + lo + 1);
        if (t < s || t >= e) return;
        pos = t - s;
    } else {
        pos = t;
    }
    if (p.pos) {
        const int64_t at = b * p.pos_batch + t * p.pos_token;
        pos = p.pos64 ? static_cast<const int64_t*>(p.pos)[at] : static_cast<const int32_t*>(p.pos)[at];
    }
    pos += p.offset;
    // the item's two parts; those behind the turned pairs are copied
    const bool turns = item < p.turned;
    int e0, e1;
    bool two = true;
    float s[PP], c[PP];
    if (turns) {
        const int j0 = item * PP;
        e0 = kInter ? 2 * j0 : j0;
        e1 = kInter ? e0 + kTwo : e0 + p.rot / 2;
#pragma unroll
        for (int j = 0; j < PP; ++j) {
            const float2 sc = turn(static_cast<uint32_t>((static_cast<uint64_t>(pos) * s_turns[j0 + j]) >> 32));
            s[j] = sc.x * p.sign;
            c[j] = sc.y * p.scale;
        }
    } else {
        e0 = p.rot + (item - p.turned) * 2 * kTwo;
        e1 = e0 + kTwo;
        two = e1 < p.D;
    }
    const int h0 = blockIdx.y * p.per, h1 = min(h0 + p.per, p.heads);
    const auto part = [&](const RotTensor& x, int lo, int hi) {
        const T* in = static_cast<const T*>(x.in) + b * x.in_batch + t * x.in_token + lo * x.in_head;
        T* out = static_cast<T*>(x.out) + b * x.out_batch + t * x.out_token + lo * x.out_head;
        int h = lo;
        constexpr int U = 4;
        for (; h + U <= hi; h += U) {
            Bytes<T, PP> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u].load(in + u * x.in_head + e0, in + u * x.in_head + e1, kInter, two);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (turns) v[u].rotate(kInter, s, c);
                v[u].store(out + u * x.out_head + e0, out + u * x.out_head + e1, kInter, two);
            }
            in += U * x.in_head;
            out += U * x.out_head;
        }
        for (; h < hi; ++h) {
            Bytes<T, PP> v;
            v.load(in + e0, in + e1, kInter, two);
            if (turns) v.rotate(kInter, s, c);
            v.store(out + e0, out + e1, kInter, two);
            in += x.in_head;
            out += x.out_head;
        }
    };
    if (h0 < p.hq) part(p.q, h0, min(h1, p.hq));
    if (h1 > p.hq) part(p.k, max(h0, p.hq) - p.hq, h1 - p.hq);
}

bool ok16(const RotTensor& t, int es) {
    return !t.in || ((reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out) |
                      static_cast<uintptr_t>(t.in_batch * es) | static_cast<uintptr_t>(t.in_token * es) |
                      static_cast<uintptr_t>(t.in_head * es) | static_cast<uintptr_t>(t.out_batch * es) |
                      static_cast<uintptr_t>(t.out_token * es) | static_cast<uintptr_t>(t.out_head * es)) & 15u) == 0;
}

template <typename T, int PP>
cudaError_t launch(RotParams p, bool inter, bool copy, cudaStream_t s) {
    constexpr int part = PP;            // elements
    p.turned = p.rot / 2 / PP;
    p.items = p.turned + (copy ? (p.D - p.rot + 2 * part - 1) / (2 * part) : 0);
    if (p.items == 0) return cudaSuccess;
    const int64_t n = static_cast<int64_t>(p.tokens) * p.items;
    // Heads of a thread: eight share their sines, fewer where the device would not be full.
    p.per = kMostHeads;
    while (p.per > (p.heads > 65535 ? 2 : 1) && n * ((p.heads + p.per - 1) / p.per) < static_cast<int64_t>(device_sm_count()) * 1024) p.per /= 2;
    const dim3 grid(static_cast<unsigned>((n + kThreads - 1) / kThreads), static_cast<unsigned>((p.heads + p.per - 1) / p.per));
    if (inter) rotary_kernel<T, PP, true><<<grid, kThreads, 0, s>>>(p);
    else rotary_kernel<T, PP, false><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_any(const RotParams& p, bool inter, bool copy, cudaStream_t s) {
    constexpr int PP = 16 / sizeof(T), es = sizeof(T);
    const bool vec = p.rot / 2 % PP == 0 && (!copy || (p.D - p.rot) % PP == 0) && ok16(p.q, es) && ok16(p.k, es);
    return vec ? launch<T, PP>(p, inter, copy, s) : launch<T, 1>(p, inter, copy, s);
}

m3_status err(m3_status st, const char* fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return set_error(st, msg);
}

m3_status check(const m3_rotary_dims* d, bool packed) {
    if (!d) return err(M3_ERR_INVALID_ARG, "dims is NULL");
    if (d->in_dtype != M3_F32 && d->in_dtype != M3_BF16)
        return err(M3_ERR_INVALID_ARG, "in_dtype %d is not M3_F32 or M3_BF16", d->in_dtype);
    if (d->nseq < 0 || d->seqlen < 0) return err(M3_ERR_INVALID_ARG, "nseq and seqlen must be >= 0");
    if (d->qheads < 1 || d->kheads < 0) return err(M3_ERR_INVALID_ARG, "qheads must be >= 1, kheads >= 0");
    if (d->headdim < 1 || d->rotdim < 0 || d->rotdim > d->headdim || d->rotdim % 2)
        return err(M3_ERR_INVALID_ARG, "rotdim (%lld) must be even and at most headdim (%lld)", (long long)d->rotdim,
                   (long long)d->headdim);
    if (d->flags & ~(M3_ROT_INTERLEAVED | M3_ROT_INVERSE | M3_ROT_POS64))
        return err(M3_ERR_INVALID_ARG, "unknown bits in flags (0x%x)", (unsigned)d->flags);
    if (!std::isfinite(d->scale)) return err(M3_ERR_INVALID_ARG, "scale must be finite");
    if (d->headdim > 2 * kMaxPairs || d->qheads > 32768 || d->kheads > 32768)
        return err(M3_ERR_UNSUPPORTED, "headdim above %d or more than 32768 heads", 2 * kMaxPairs);
    // (token, item) pairs are counted in 32 bits
    const int64_t n = packed || d->nseq < 1 ? 1 : d->nseq;
    if (d->nseq > (int64_t(1) << 30) || d->seqlen > (int64_t(1) << 30) || d->seqlen > 0xfffffe00LL / d->headdim / n)
        return err(M3_ERR_UNSUPPORTED, "tokens * headdim exceeds 2^32");
    return M3_OK;
}

m3_status check_ptr(const void* q, uintptr_t align, const char* name, bool need) {
    if (!q) return need ? err(M3_ERR_INVALID_ARG, "%s is NULL", name) : M3_OK;
    if (reinterpret_cast<uintptr_t>(q) % align) return err(M3_ERR_INVALID_ARG, "%s is not element-aligned", name);
    return M3_OK;
}

// A dimension of one entry has stride 0, whatever the caller's says.
RotTensor tensor(const m3_rotary_dims* d, const m3_view* in, const m3_view* out, int64_t heads, bool packed) {
    if (!in || !in->data || heads == 0) return RotTensor{};
    const bool b = !packed && d->nseq > 1, t = d->seqlen > 1, h = heads > 1;
    return RotTensor{in->data, out->data, b ? in->batch : 0, t ? in->token : 0, h ? in->head : 0,
                     b ? out->batch : 0, t ? out->token : 0, h ? out->head : 0};
}

// An output lies on its own input in the same places, or begins elsewhere; its heads and rows do not overlap.
m3_status check_out(const m3_rotary_dims* d, const RotTensor& x, int64_t heads, bool packed, const char* name) {
    if (x.out == x.in && (x.in_batch != x.out_batch || x.in_token != x.out_token || x.in_head != x.out_head))
        return err(M3_ERR_INVALID_ARG, "%s lies on its input by other strides", name);
    const auto small = [&](int64_t s) { return (s < 0 ? -s : s) < d->headdim; };
    if ((heads > 1 && small(x.out_head)) || (d->seqlen > 1 && small(x.out_token)) || (!packed && d->nseq > 1 && small(x.out_batch)))
        return err(M3_ERR_INVALID_ARG, "%s: heads or rows overlap", name);
    return M3_OK;
}

}  // namespace
}  // namespace m3

using namespace m3;

extern "C" m3_status m3_rotary(const m3_rotary_dims* dims, const m3_view* q, const m3_view* k, const double* freq,
                               const void* positions, int64_t pos_batch, int64_t pos_token, const int32_t* cu_seqlens,
                               const m3_view* q_out, const m3_view* k_out, void* stream) {
    set_error(M3_OK, "");
    const bool packed = cu_seqlens != nullptr;
    m3_status st = check(dims, packed);
    if (st != M3_OK) return st;
    const bool any = dims->nseq > 0 && dims->seqlen > 0, keys = dims->kheads > 0;
    const uintptr_t es = dims->in_dtype == M3_BF16 ? 2 : 4;
    if ((st = check_ptr(q ? q->data : nullptr, es, "q", any)) != M3_OK ||
        (st = check_ptr(k ? k->data : nullptr, es, "k", any && keys)) != M3_OK ||
        (st = check_ptr(q_out ? q_out->data : nullptr, es, "q_out", any)) != M3_OK ||
        (st = check_ptr(k_out ? k_out->data : nullptr, es, "k_out", any && keys)) != M3_OK ||
        (st = check_ptr(freq, 8, "freq", any && dims->rotdim > 0)) != M3_OK ||
        (st = check_ptr(positions, dims->flags & M3_ROT_POS64 ? 8 : 4, "positions", false)) != M3_OK ||
        (st = check_ptr(cu_seqlens, 4, "cu_seqlens", false)) != M3_OK)
        return st;
    if (!any) return M3_OK;
    RotParams p{};
    p.q = tensor(dims, q, q_out, dims->qheads, packed);
    p.k = tensor(dims, k, k_out, dims->kheads, packed);
    if ((st = check_out(dims, p.q, dims->qheads, packed, "q_out")) != M3_OK ||
        (keys && (st = check_out(dims, p.k, dims->kheads, packed, "k_out")) != M3_OK))
        return st;
    if (keys && (p.q.out == p.k.in || p.k.out == p.q.in || p.q.out == p.k.out))
        return err(M3_ERR_INVALID_ARG, "q_out or k_out begins where the other's tensors do");
    for (const void* o : {static_cast<const void*>(p.q.out), static_cast<const void*>(p.k.out)})
        if (o && (o == freq || o == positions || o == cu_seqlens))
            return err(M3_ERR_INVALID_ARG, "an output begins where freq, positions or cu_seqlens do");
    p.freq = freq;
    p.pos = positions;
    p.pos_batch = packed || dims->nseq == 1 ? 0 : pos_batch;
    p.pos_token = dims->seqlen == 1 ? 0 : pos_token;
    p.offset = dims->offset;
    p.cu = cu_seqlens;
    p.nseq = static_cast<int>(dims->nseq);
    p.len = static_cast<uint32_t>(dims->seqlen);
    p.tokens = static_cast<uint32_t>(packed ? dims->seqlen : dims->nseq * dims->seqlen);
    p.hq = static_cast<int>(dims->qheads);
    p.heads = static_cast<int>(dims->qheads + dims->kheads);
    p.D = static_cast<int>(dims->headdim);
    p.rot = static_cast<int>(dims->rotdim);
    p.pos64 = dims->flags & M3_ROT_POS64 ? 1 : 0;
    p.scale = dims->scale;
    p.sign = dims->flags & M3_ROT_INVERSE ? -dims->scale : dims->scale;
    const bool inter = dims->flags & M3_ROT_INTERLEAVED;
    const bool copy = p.rot < p.D && (p.q.in != p.q.out || (keys && p.k.in != p.k.out));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dims->in_dtype == M3_BF16 ? launch_any<__nv_bfloat16>(p, inter, copy, s)
                                                    : launch_any<float>(p, inter, copy, s);
    return e == cudaSuccess ? M3_OK : err(M3_ERR_CUDA, "rotary launch: %s", cudaGetErrorString(e));
}
