// Linear attention with a decay for each head: host side of its entry points (validation, the cut
// into segments, workspace layout, dispatch) and the sum of shared heads' gradients.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "m3_common.cuh"
#include "m3_internal.h"
#include "m3_linattn.h"

namespace m3 {

// Segments trade work for parallelism: every cut sequence reads its k and v a second time (for the
// segments' end states) and sums its predecessors' states, but the CTAs fill the device's slots more
// evenly. A batch takes the number of segments with the least estimated time (waves of CTAs, of both
// launches, times a CTA's chunks), more of them only for a tenth less: they read more of k and v
// again. (b1 H64 L65536: 2 segments, one wave of 256 chunks on 128 SMs, 0.96 ms; 9 segments, 4 waves of
// 57 on all 148, 4 % more.)
LinPlan lin_plan(int64_t nseq, int64_t L, bool packed, int64_t per_x, const LinForm& form) {
    LinPlan pl{};
    const int64_t chunks = (L + form.chunk - 1) / form.chunk;
    if (!packed) {
        const int64_t units = nseq * per_x, slots = form.slots;
        int64_t best = 1;
        float least = 0.f;
        for (int64_t n = 1; n <= kLinMaxSegs && (n == 1 || n * form.min_chunks <= chunks); ++n) {
            const int64_t seg = (chunks + n - 1) / n;
            if (n > 1 && (chunks + seg - 1) / seg != n) continue;   // the same cut as a smaller n
            const auto waves = [&](int64_t segs) { return std::ceil(static_cast<float>(units * segs) * form.unit / slots); };
            float cost = waves(n) * (seg + form.setup);
            if (n > 1)
                cost += waves(n - 1) * (form.state_chunk * seg + form.setup) +
                        form.predecessor * (n - 1);
            if (n == 1 || cost < 0.9f * least) {
                best = n;
                least = cost;
            }
        }
        const int64_t seg = chunks > 0 ? (chunks + best - 1) / best : 1;    // chunks of a segment
        pl.seg_len = static_cast<int>(seg * form.chunk);
        pl.nseg = static_cast<int>(best);
        pl.blocks_x = nseq * best;
        pl.cut = best > 1;
        return pl;
    }
    // the rows' share of one slot, whichever sequences they belong to
    int64_t seg = (L * per_x + form.chunk * static_cast<int64_t>(form.slots) - 1) / (form.chunk * static_cast<int64_t>(form.slots));
    const int64_t least = (chunks + kLinMaxSegs - 1) / kLinMaxSegs;
    if (seg < least) seg = least;
    if (seg < form.min_chunks) seg = form.min_chunks;
    pl.seg_len = static_cast<int>(seg * form.chunk);
    pl.nseg = 1;
    // sum of max(1, ceil(len / seg_len)) over nseq sequences of at most L rows together
    pl.blocks_x = L / pl.seg_len + nseq;
    pl.cut = L > pl.seg_len;
    return pl;
}

namespace {

// One CTA walks down the sequences, 1024 at a time: starts[i + 1] = i + 1 + the segments beyond their first of
// the sequences up to i, of those before the reserve runs out.
constexpr int kStartThreads = 1024;
__global__ void __launch_bounds__(kStartThreads) lin_starts_kernel(const LinParams p, int32_t* starts) {
    __shared__ int s_sum[32];
    __shared__ int s_cap;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int reserve = static_cast<int>(p.blocks_x - p.nseq);      // at most kLinMaxSegs
    int asked = 0, cap = 0;         // what the sequences before ask for, and what of it fits
    if (tid == 0) {
        starts[0] = 0;
        s_cap = 0;
    }
    for (int base = 0; base < p.nseq; base += kStartThreads) {
        const int i = base + tid;
        // (more than the reserve is as good as one more than it: the sums stay small)
        int incl = i < p.nseq ? min(lin_span(p, i).more, reserve + 1) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) s_sum[warp] = incl;
        __syncthreads();
        if (warp == 0) {
            int sum = s_sum[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            s_sum[lane] = sum;
        }
        __syncthreads();
        incl += asked + (warp > 0 ? s_sum[warp - 1] : 0);
        if (incl <= reserve) atomicMax(&s_cap, incl);       // ascends: the last that fits
        asked = min(asked + s_sum[31], reserve + 1);
        __syncthreads();
        cap = s_cap;
        if (i < p.nseq) starts[i + 1] = i + 1 + min(incl, cap);
        __syncthreads();
    }
}

m3_status err(m3_status st, const char* fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return set_error(st, msg);
}
m3_status cuda_err(cudaError_t e, const char* where) {
    return err(M3_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

constexpr int64_t kMaxGrid = 0x7fffffffLL, kMaxStepUnits = kMaxGrid / 16;      // (up to 16 parts of a head)

m3_status check_dims(const m3_linattn_dims* d) {
    if (!d) return err(M3_ERR_INVALID_ARG, "dims is NULL");
    if (d->in_dtype != M3_F32 && d->in_dtype != M3_BF16)
        return err(M3_ERR_INVALID_ARG, "in_dtype %d is not M3_F32 or M3_BF16", d->in_dtype);
    if (d->nseq < 0 || d->seqlen < 0) return err(M3_ERR_INVALID_ARG, "nseq and seqlen must be >= 0");
    const int64_t H = d->nheads;
    if (H < 1) return err(M3_ERR_INVALID_ARG, "nheads must be >= 1");
    const int64_t hs[] = {d->qheads, d->kheads, d->vheads};
    const char* names[] = {"qheads", "kheads", "vheads"};
    for (int i = 0; i < 3; ++i)
        if (hs[i] < 1 || H % hs[i] != 0)
            return err(M3_ERR_INVALID_ARG, "%s (%lld) must divide nheads (%lld)", names[i],
                       (long long)hs[i], (long long)H);
    if (d->kdim < 1 || d->vdim < 1) return err(M3_ERR_INVALID_ARG, "kdim and vdim must be >= 1");
    if (!std::isfinite(d->scale)) return err(M3_ERR_INVALID_ARG, "scale must be finite");
    if (d->kdim > 256 || d->vdim > 256)
        return err(M3_ERR_UNSUPPORTED, "kdim %lld or vdim %lld exceeds 256", (long long)d->kdim, (long long)d->vdim);
    // indexes of one sequence fit 32 bits. As fp32 exponents of the decay, token counts above 2^24 are rounded: by
    // 2^-24 of the exponent, so of the power by 2^-24 of its logarithm.
    if (d->seqlen > (int64_t(1) << 30) || H > 65536 || d->nseq > (int64_t(1) << 24))
        return err(M3_ERR_UNSUPPORTED, "seqlen above 2^30, nheads above 65536 or nseq above 2^24");
    return M3_OK;
}

m3_status check_view(const m3_view* v, const char* name, int es, bool need) {
    if (!v || !v->data) return need ? err(M3_ERR_INVALID_ARG, "%s is NULL", name) : M3_OK;
    if (reinterpret_cast<uintptr_t>(v->data) % static_cast<uintptr_t>(es) != 0)
        return err(M3_ERR_INVALID_ARG, "%s is not aligned to its element size", name);
    return M3_OK;
}
m3_status check_state(const float* q, const char* name) {
    return reinterpret_cast<uintptr_t>(q) & 15u ? err(M3_ERR_INVALID_ARG, "%s is not 16-byte aligned", name) : M3_OK;
}
m3_status check_inputs(const m3_linattn_dims* d, const m3_linattn_inputs* in, bool any) {
    if (!in) return err(M3_ERR_INVALID_ARG, "inputs is NULL");
    const int es = d->in_dtype == M3_BF16 ? 2 : 4;
    m3_status st;
    if ((st = check_view(&in->q, "q", es, any)) != M3_OK || (st = check_view(&in->k, "k", es, any)) != M3_OK ||
        (st = check_view(&in->v, "v", es, any)) != M3_OK)
        return st;
    if (!in->log_decay) return err(M3_ERR_INVALID_ARG, "log_decay is NULL");
    if (reinterpret_cast<uintptr_t>(in->log_decay) & 3u) return err(M3_ERR_INVALID_ARG, "log_decay is misaligned");
    if (reinterpret_cast<uintptr_t>(in->cu_seqlens) & 3u) return err(M3_ERR_INVALID_ARG, "cu_seqlens is misaligned");
    return M3_OK;
}

// An output that begins where an input or another output does would be written while it is read (or
// written twice); overlaps further in are the caller's to avoid. The last output is a state, which may be
// the last input: the state that it follows.
struct Named {
    const void* p;
    const char* name;
};
template <int I, int O>
m3_status check_apart(const Named (&ins)[I], const Named (&outs)[O]) {
    for (int i = 0; i < O; ++i) {
        if (!outs[i].p) continue;
        for (int a = 0; a < I; ++a)
            if (outs[i].p == ins[a].p && !(i == O - 1 && a == I - 1))
                return err(M3_ERR_INVALID_ARG, "%s is %s", outs[i].name, ins[a].name);
        for (int a = 0; a < i; ++a)
            if (outs[i].p == outs[a].p) return err(M3_ERR_INVALID_ARG, "%s is %s", outs[i].name, outs[a].name);
    }
    return M3_OK;
}

// A dimension of one entry has stride 0, whatever the caller's says.
LinTensor tensor(const m3_linattn_dims* d, const m3_view& v, int64_t heads, bool packed) {
    return LinTensor{v.data, packed || d->nseq == 1 ? 0 : v.batch, d->seqlen == 1 ? 0 : v.token,
                     heads == 1 ? 0 : v.head, static_cast<int>(d->nheads / heads)};
}

void set_output(LinJob& j, const m3_linattn_dims* d, const m3_view& v, int64_t heads, bool packed) {
    const LinTensor t = tensor(d, v, heads, packed);
    j.y = v.data;
    j.y_batch = t.batch;
    j.y_token = t.token;
    j.y_head = t.head;
}

LinParams make_params(const m3_linattn_dims* d, const m3_linattn_inputs* in) {
    LinParams p{};
    p.log_decay = in->log_decay;
    p.cu = in->cu_seqlens;
    p.nseq = static_cast<int>(d->nseq);
    p.H = static_cast<int>(d->nheads);
    p.L = d->seqlen;
    return p;
}

LinStep make_step(const m3_linattn_dims* d, const m3_linattn_inputs* in, const float* state_in, float* state_out,
                  int64_t nstates, const int32_t* slots, const m3_view* o) {
    LinStep p{};
    p.q = tensor(d, in->q, d->qheads, false);
    p.k = tensor(d, in->k, d->kheads, false);
    p.v = tensor(d, in->v, d->vheads, false);
    p.log_decay = in->log_decay;
    p.state_in = state_in;
    p.state_out = state_out;
    p.nstates = nstates;
    p.slots = slots;
    p.o = o->data;
    p.o_batch = o->batch;
    p.o_token = o->token;
    p.L = static_cast<int>(d->seqlen);
    p.o_head = o->head;
    p.nseq = d->nseq;
    p.H = static_cast<int>(d->nheads);
    p.K = static_cast<int>(d->kdim);
    p.V = static_cast<int>(d->vdim);
    p.scale = d->scale;
    return p;
}

int tiles_of(int64_t dim) { return static_cast<int>((dim + kLinTile - 1) / kLinTile); }

// Tiles of the launches: forward, and the three gradients of the backward in one
int fwd_tiles(const m3_linattn_dims* d) { return tiles_of(d->vdim); }
int bwd_tiles(const m3_linattn_dims* d) { return 2 * tiles_of(d->kdim) + tiles_of(d->vdim); }
int bwd_rows(const m3_linattn_dims* d) { return static_cast<int>(d->kdim > d->vdim ? d->kdim : d->vdim); }

// The fp32 form's plan. A backward's units have states of V and of K rows: a chunk of 32 tokens of Dk costs
// 32 (16 Dk + 16 64 + 2 Dk 64) products. (Counted as if all took as long as the longest: gradients of
// 2048 tokens of 16 heads, K 256, V 64, bf16 1534 us, of 300 tokens of 4 heads 104; so 1132 and 62.)
LinForm simt_form(const m3_linattn_dims* d, bool backward) {
    if (!backward) return lin_simt_form(static_cast<int>(d->kdim), 1.f);
    const auto cost = [](int64_t Dk) { return 144.f * Dk + 1024.f; };
    const float k = cost(d->kdim), v = cost(d->vdim), most = k > v ? k : v;
    const int tk = tiles_of(d->kdim), tv = tiles_of(d->vdim);
    return lin_simt_form(bwd_rows(d), (2 * tk * v + tv * k) / ((2 * tk + tv) * most));
}

size_t seg_bytes(const m3_linattn_dims* d, bool packed, int rtiles, int rows, const LinForm& form) {
    if (d->nseq == 0 || d->seqlen == 0) return 0;
    const LinPlan pl = lin_plan(d->nseq, d->seqlen, packed, d->nheads * rtiles, form);
    return pl.cut ? static_cast<size_t>(pl.blocks_x) * d->nheads * rtiles * rows * kLinTile * 4 : 0;
}
// the larger of what the two forms take (which one runs depends on the tensors' alignment)
size_t table_bytes(const m3_linattn_dims* d, bool packed) {
    if (!packed || d->nseq <= kLinScanned || d->seqlen == 0) return 0;
    return ((static_cast<size_t>(d->nseq) + 1) * 4 + 255) / 256 * 256;
}

size_t seg_bytes(const m3_linattn_dims* d, bool packed, bool backward) {
    const int rtiles = backward ? bwd_tiles(d) : fwd_tiles(d), rows = backward ? bwd_rows(d) : static_cast<int>(d->kdim);
    const size_t a = seg_bytes(d, packed, rtiles, rows, simt_form(d, backward));
    const size_t b = seg_bytes(d, packed, rtiles, rows < 128 ? 128 : rows, lin_tc_form());
    return ((a > b ? a : b) + 255) / 256 * 256;
}

// fp32 per-head gradients of tensors whose heads are shared: [rows][H][dim] each
size_t shared_bytes(const m3_linattn_dims* d, int which, bool packed) {
    const int64_t heads = which == 0 ? d->qheads : which == 1 ? d->kheads : d->vheads;
    const int64_t dim = which == 2 ? d->vdim : d->kdim;
    if (heads == d->nheads) return 0;
    const int64_t rows = packed ? d->seqlen : d->nseq * d->seqlen;
    return (static_cast<size_t>(rows) * d->nheads * dim * 4 + 255) / 256 * 256;
}

// The sum over the H / heads heads that read one head of a tensor, in order, rounded once: up to
// three tensors in one launch (blockIdx.y), eight columns a thread where the dimension allows.
struct Fold {
    const float* part;
    void* out;
    int64_t batch, token, head;
    int heads, ratio, dim, vec;
    int64_t units;          // rows * heads * (dim / vec)
};
struct Folds {
    Fold f[3];
    const int32_t* cu;
    int64_t L;
    int nseq;
};
template <typename T>
__global__ void __launch_bounds__(256) fold_heads_kernel(const __grid_constant__ Folds p) {
    const Fold& f = p.f[blockIdx.y];
    const int per = f.dim / f.vec;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < f.units;
         e += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int c = static_cast<int>(e % per) * f.vec;
        const int64_t rh = e / per;
        const int g = static_cast<int>(rh % f.heads);
        const int64_t row = rh / f.heads;
        if (p.cu) {     // rows of no sequence are left alone: the last sequence that starts by this row
            int lo = 0, hi = p.nseq - 1;
            while (lo < hi) {
                const int m = (lo + hi + 1) >> 1;
                if (p.cu[m] <= row) lo = m;
                else hi = m - 1;
            }
            if (row < p.cu[lo] || row >= p.cu[lo + 1]) continue;
        }
        const int64_t b = p.cu ? 0 : row / p.L, t = p.cu ? row : row % p.L;
        const float* src = f.part + (row * f.heads + g) * static_cast<int64_t>(f.ratio) * f.dim + c;
        T* out = static_cast<T*>(f.out) + b * f.batch + t * f.token + g * f.head + c;
        if (f.vec == 8) {
            float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int i = 0; i < f.ratio; ++i) {
                const float4 lo = __ldcs(reinterpret_cast<const float4*>(src + static_cast<int64_t>(i) * f.dim));
                const float4 hi = __ldcs(reinterpret_cast<const float4*>(src + static_cast<int64_t>(i) * f.dim + 4));
                s[0] += lo.x; s[1] += lo.y; s[2] += lo.z; s[3] += lo.w;
                s[4] += hi.x; s[5] += hi.y; s[6] += hi.z; s[7] += hi.w;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) out[i] = from_f<T>(s[i]);
        } else {
            float s = 0.f;
            for (int i = 0; i < f.ratio; ++i) s += src[static_cast<int64_t>(i) * f.dim];
            *out = from_f<T>(s);
        }
    }
}

cudaError_t fold_heads(const m3_linattn_dims* d, float* const (&part)[3], const m3_view* const (&v)[3],
                       const int32_t* cu, cudaStream_t s) {
    Folds p{};
    p.cu = cu;
    p.L = d->seqlen;
    p.nseq = static_cast<int>(d->nseq);
    const int64_t rows = cu ? d->seqlen : d->nseq * d->seqlen;
    int n = 0;
    int64_t most = 0;
    for (int i = 0; i < 3; ++i) {
        if (!part[i]) continue;
        Fold& f = p.f[n++];
        const int64_t heads = i == 0 ? d->qheads : i == 1 ? d->kheads : d->vheads;
        f.part = part[i];
        f.out = v[i]->data;
        f.batch = v[i]->batch;
        f.token = v[i]->token;
        f.head = v[i]->head;
        f.heads = static_cast<int>(heads);
        f.ratio = static_cast<int>(d->nheads / heads);
        f.dim = static_cast<int>(i == 2 ? d->vdim : d->kdim);
        f.vec = f.dim % 8 == 0 ? 8 : 1;
        f.units = rows * heads * (f.dim / f.vec);
        most = f.units > most ? f.units : most;
    }
    if (n == 0 || most == 0) return cudaSuccess;
    int64_t grid = (most + 255) / 256;
    const int64_t lim = 16LL * device_sm_count();
    if (grid > lim) grid = lim;
    const dim3 g(static_cast<unsigned>(grid), static_cast<unsigned>(n));
    if (d->in_dtype == M3_BF16) fold_heads_kernel<__nv_bfloat16><<<g, 256, 0, s>>>(p);
    else fold_heads_kernel<float><<<g, 256, 0, s>>>(p);
    return cudaGetLastError();
}

// Plans and launches the jobs of p in the form that takes them. table: table_bytes of the workspace.
m3_status run_jobs(LinParams& p, const m3_linattn_dims* d, int state_rows, char* ws, char* table, cudaStream_t s) {
    const bool bf16 = d->in_dtype == M3_BF16, packed = p.cu != nullptr;
    const bool few = (packed ? d->seqlen : d->nseq * d->seqlen) * d->nheads <= kLinFew;
    const bool tc = bf16 && !few && lin_tc_supported(p);
    const LinPlan pl = lin_plan(d->nseq, d->seqlen, packed, d->nheads * p.rtiles,
                                tc ? lin_tc_form() : simt_form(d, p.njobs > 1));
    p.seg_len = pl.seg_len;
    p.nseg = pl.nseg;
    p.blocks_x = pl.blocks_x;
    p.seg = reinterpret_cast<float*>(ws);
    p.seg_rows = tc && state_rows < 128 ? 128 : state_rows;
    if (p.blocks_x > kMaxGrid / (d->nheads * p.rtiles))
        return err(M3_ERR_UNSUPPORTED, "sequences * heads * column tiles exceed the grid limit");
    cudaError_t e = cudaSuccess;
    if (table_bytes(d, packed) > 0) {
        int32_t* starts = reinterpret_cast<int32_t*>(table);
        lin_starts_kernel<<<1, kStartThreads, 0, s>>>(p, starts);
        if ((e = cudaGetLastError()) != cudaSuccess) return cuda_err(e, "linear attention table launch");
        p.starts = starts;
    }
    e = tc ? launch_lin_tc(p, pl.cut, s) : launch_lin_simt(p, bf16, pl.cut, s);
    return e == cudaSuccess ? M3_OK : cuda_err(e, "linear attention launch");
}

// No token at all: the state passes through.
m3_status pass_state(const m3_linattn_dims* d, const float* from, float* to, cudaStream_t s) {
    if (!to || to == from) return M3_OK;
    const size_t n = static_cast<size_t>(d->nseq) * d->nheads * d->kdim * d->vdim * 4;
    if (n == 0) return M3_OK;
    const cudaError_t e = from ? cudaMemcpyAsync(to, from, n, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(to, 0, n, s);
    return e == cudaSuccess ? M3_OK : cuda_err(e, "empty-sequence state copy");
}

// A copy of a state that the call overwrites while it may still read it.
size_t state_bytes(const m3_linattn_dims* d) {
    return (static_cast<size_t>(d->nseq) * d->nheads * d->kdim * d->vdim * 4 + 255) / 256 * 256;
}
m3_status keep_state(const m3_linattn_dims* d, const float* from, char* to, cudaStream_t s) {
    const cudaError_t e = cudaMemcpyAsync(to, from, static_cast<size_t>(d->nseq) * d->nheads * d->kdim * d->vdim * 4,
                                          cudaMemcpyDeviceToDevice, s);
    return e == cudaSuccess ? M3_OK : cuda_err(e, "state copy");
}

m3_status check_workspace(void* ws, size_t have, size_t need) {
    if (need > 0 && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || have < need))
        return err(M3_ERR_INVALID_ARG, "workspace: NULL, misaligned or below %zu bytes", need);
    return M3_OK;
}

}  // namespace
}  // namespace m3

using namespace m3;

extern "C" {

size_t m3_linattn_workspace_bytes(const m3_linattn_dims* dims, int packed) {
    if (check_dims(dims) != M3_OK) return 0;
    const size_t n = seg_bytes(dims, packed != 0, false);
    return (n ? n + state_bytes(dims) : 0) + table_bytes(dims, packed != 0);
}

size_t m3_linattn_bwd_workspace_bytes(const m3_linattn_dims* dims, int packed) {
    if (check_dims(dims) != M3_OK) return 0;
    size_t n = seg_bytes(dims, packed != 0, true);
    for (int i = 0; i < 3; ++i) n += shared_bytes(dims, i, packed != 0);
    return n + state_bytes(dims) + table_bytes(dims, packed != 0);
}

m3_status m3_linattn_fwd(const m3_linattn_dims* dims, const m3_linattn_inputs* in, const float* init,
                         float* final_state, const m3_view* o, void* workspace, size_t ws_bytes,
                         void* stream) {
    set_error(M3_OK, "");
    m3_status st = check_dims(dims);
    if (st != M3_OK) return st;
    const bool any = dims->nseq > 0 && dims->seqlen > 0;
    if ((st = check_inputs(dims, in, any)) != M3_OK || (st = check_state(init, "init")) != M3_OK ||
        (st = check_state(final_state, "final_state")) != M3_OK ||
        (st = check_view(o, "o", dims->in_dtype == M3_BF16 ? 2 : 4, any)) != M3_OK)
        return st;
    const size_t need = m3_linattn_workspace_bytes(dims, in->cu_seqlens != nullptr);
    if ((st = check_workspace(workspace, ws_bytes, need)) != M3_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!any) return pass_state(dims, init, final_state, s);
    const Named ins[] = {{in->q.data, "q"}, {in->k.data, "k"}, {in->v.data, "v"}, {in->log_decay, "log_decay"},
                         {in->cu_seqlens, "cu_seqlens"}, {init, "init"}};
    const Named outs[] = {{o->data, "o"}, {final_state, "final_state"}};
    if ((st = check_apart(ins, outs)) != M3_OK) return st;
    const bool packed = in->cu_seqlens != nullptr;
    if (!packed && dims->seqlen <= kLinShort && (dims->seqlen == 1 || dims->vdim % 4 == 0) &&
        dims->nseq * dims->nheads <= kMaxStepUnits) {
        // Few tokens are steps on a state held in registers: exact products, and less time than a chunk with few
        // rows. bf16, K 128, V 64, 64 sequences of 64 heads: 42, 55, 155 us for 1, 2, 8 tokens against 218 to
        // 221; 4 sequences: 5.5, 6.1, 12.2 against 16.5. One sequence of 4 heads (V 64): 3.0, 3.8, 7.4 against 6.4, a
        // microsecond more at 8 tokens, which is left so that the products are exact whatever the batch.
        const LinStep p = make_step(dims, in, init, final_state, dims->nseq, nullptr, o);
        const cudaError_t e = launch_lin_step(p, dims->in_dtype == M3_BF16, s);
        return e == cudaSuccess ? M3_OK : cuda_err(e, "linear attention launch");
    }
    LinParams p = make_params(dims, in);
    LinJob& j = p.job[0];
    j.q = tensor(dims, in->q, dims->qheads, packed);
    j.k = tensor(dims, in->k, dims->kheads, packed);
    j.v = tensor(dims, in->v, dims->vheads, packed);
    set_output(j, dims, *o, dims->nheads, packed);
    j.Dk = static_cast<int>(dims->kdim);
    j.Dv = static_cast<int>(dims->vdim);
    j.tiles = fwd_tiles(dims);
    j.p_scale = j.o_scale = dims->scale;
    j.x_scale = 1.f;
    j.init = init;
    j.init_k = dims->vdim;
    j.init_v = 1;
    j.final_state = final_state;
    p.njobs = 1;
    p.rtiles = j.tiles;
    const size_t seg = seg_bytes(dims, packed, false);
    char* const ws = static_cast<char*>(workspace);
    if (init && init == final_state && seg > 0) {   // cut: later segments read it while the last writes
        char* copy = ws + seg;
        if ((st = keep_state(dims, init, copy, s)) != M3_OK) return st;
        j.init = reinterpret_cast<const float*>(copy);
    }
    return run_jobs(p, dims, j.Dk, ws, ws + need - table_bytes(dims, packed), s);
}

m3_status m3_linattn_bwd(const m3_linattn_dims* dims, const m3_linattn_inputs* in, const float* init,
                         const m3_view* d_o, const float* dfinal, const m3_linattn_grads* grads,
                         float* dinit, void* workspace, size_t ws_bytes, void* stream) {
    set_error(M3_OK, "");
    m3_status st = check_dims(dims);
    if (st != M3_OK) return st;
    const bool any = dims->nseq > 0 && dims->seqlen > 0;
    const int es = dims->in_dtype == M3_BF16 ? 2 : 4;
    if (!grads) return err(M3_ERR_INVALID_ARG, "grads is NULL");
    if ((st = check_inputs(dims, in, any)) != M3_OK || (st = check_view(d_o, "d_o", es, any)) != M3_OK ||
        (st = check_view(&grads->dq, "dq", es, any)) != M3_OK || (st = check_view(&grads->dk, "dk", es, any)) != M3_OK ||
        (st = check_view(&grads->dv, "dv", es, any)) != M3_OK || (st = check_state(init, "init")) != M3_OK ||
        (st = check_state(dfinal, "dfinal")) != M3_OK || (st = check_state(dinit, "dinit")) != M3_OK)
        return st;
    const bool packed = in->cu_seqlens != nullptr;
    const size_t need = m3_linattn_bwd_workspace_bytes(dims, packed);
    if ((st = check_workspace(workspace, ws_bytes, need)) != M3_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dinit && dinit == init) return err(M3_ERR_INVALID_ARG, "dinit is init");
    if (!any) return pass_state(dims, dfinal, dinit, s);

    LinParams p = make_params(dims, in);
    const int64_t H = dims->nheads;
    const int K = static_cast<int>(dims->kdim), V = static_cast<int>(dims->vdim);
    const LinTensor q = tensor(dims, in->q, dims->qheads, packed), k = tensor(dims, in->k, dims->kheads, packed),
                    v = tensor(dims, in->v, dims->vheads, packed), g = tensor(dims, *d_o, H, packed);
    char* ws = static_cast<char*>(workspace);
    char* seg = ws;
    ws += seg_bytes(dims, packed, true);
    const m3_view* const outs[3] = {&grads->dq, &grads->dk, &grads->dv};
    const Named ins[] = {{in->q.data, "q"}, {in->k.data, "k"}, {in->v.data, "v"}, {d_o->data, "d_o"},
                         {in->log_decay, "log_decay"}, {in->cu_seqlens, "cu_seqlens"}, {init, "init"}, {dfinal, "dfinal"}};
    const Named named[] = {{grads->dq.data, "dq"}, {grads->dk.data, "dk"}, {grads->dv.data, "dv"}, {dinit, "dinit"}};
    if ((st = check_apart(ins, named)) != M3_OK) return st;
    float* part[3];
    for (int i = 0; i < 3; ++i) {
        const size_t n = shared_bytes(dims, i, packed);
        part[i] = n ? reinterpret_cast<float*>(ws) : nullptr;
        ws += n;
    }
    const LinTensor a[3] = {g, v, k}, b[3] = {v, g, q}, c[3] = {k, q, g};   // (do, v, k), (v, do, q), (k, q, do)
    const int Dk[3] = {V, V, K}, Dv[3] = {K, K, V};
    p.rtiles = 0;
    for (int i = 0; i < 3; ++i) {
        LinJob& j = p.job[i];
        j.q = a[i]; j.k = b[i]; j.v = c[i];
        j.Dk = Dk[i]; j.Dv = Dv[i];
        j.tiles = tiles_of(Dv[i]);
        p.rtiles += j.tiles;
        j.reverse = i > 0;
        j.p_scale = dims->scale;
        // forward states carry plain sums, backward ones the scaled gradient beside dfinal
        j.o_scale = i > 0 ? 1.f : dims->scale;
        j.x_scale = i > 0 ? dims->scale : 1.f;
        j.init = i > 0 ? dfinal : init;
        j.init_k = i < 2 ? 1 : V;       // dq's and dk's states are the transposed ones
        j.init_v = i < 2 ? V : 1;
        if (part[i]) {
            j.y = part[i];
            j.y_f32 = 1;
            j.y_head = Dv[i];
            j.y_token = H * Dv[i];
            j.y_batch = packed ? 0 : dims->seqlen * j.y_token;
        } else {
            set_output(j, dims, *outs[i], H, packed);
        }
    }
    p.job[2].final_state = dinit;
    p.njobs = 3;
    if (dfinal && dinit == dfinal) {    // other CTAs read it while one writes it
        if ((st = keep_state(dims, dfinal, ws, s)) != M3_OK) return st;
        p.job[1].init = p.job[2].init = reinterpret_cast<const float*>(ws);
    }
    char* const table = static_cast<char*>(workspace) + need - table_bytes(dims, packed);
    if ((st = run_jobs(p, dims, bwd_rows(dims), seg, table, s)) != M3_OK) return st;
    const cudaError_t e = fold_heads(dims, part, outs, in->cu_seqlens, s);
    if (e != cudaSuccess) return cuda_err(e, "gradient sum launch");
    return M3_OK;
}

m3_status m3_linattn_step(const m3_linattn_dims* dims, const m3_linattn_inputs* in, const float* state_in,
                          float* state_out, int64_t nstates, const int32_t* slots, const m3_view* o,
                          void* stream) {
    set_error(M3_OK, "");
    m3_status st = check_dims(dims);
    if (st != M3_OK) return st;
    if (dims->seqlen != 1) return err(M3_ERR_INVALID_ARG, "a step needs seqlen == 1");
    const bool any = dims->nseq > 0;
    if ((st = check_inputs(dims, in, any)) != M3_OK) return st;
    if (in->cu_seqlens) return err(M3_ERR_INVALID_ARG, "a step takes no cu_seqlens");
    if (nstates < 0 || (!slots && nstates < dims->nseq))
        return err(M3_ERR_INVALID_ARG, "nstates (%lld) is below nseq (%lld)", (long long)nstates, (long long)dims->nseq);
    if (reinterpret_cast<uintptr_t>(slots) & 3u) return err(M3_ERR_INVALID_ARG, "slots is misaligned");
    if (any && nstates > 0 && (!state_in || !state_out)) return err(M3_ERR_INVALID_ARG, "state_in and state_out are required");
    if ((st = check_state(state_in, "state_in")) != M3_OK || (st = check_state(state_out, "state_out")) != M3_OK ||
        (st = check_view(o, "o", dims->in_dtype == M3_BF16 ? 2 : 4, any)) != M3_OK)
        return st;
    if (dims->nseq * dims->nheads > kMaxStepUnits) return err(M3_ERR_UNSUPPORTED, "nseq * nheads exceeds the grid limit");
    if (!any) return M3_OK;
    const Named ins[] = {{in->q.data, "q"}, {in->k.data, "k"}, {in->v.data, "v"}, {in->log_decay, "log_decay"},
                         {slots, "slots"}, {state_in, "state_in"}};
    const Named outs[] = {{o->data, "o"}, {state_out, "state_out"}};
    if ((st = check_apart(ins, outs)) != M3_OK) return st;
    const LinStep p = make_step(dims, in, state_in, state_out, nstates, slots, o);
    const cudaError_t e = launch_lin_step(p, dims->in_dtype == M3_BF16, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? M3_OK : cuda_err(e, "linear attention step launch");
}

m3_status m3_linattn_check(void) {
    set_error(M3_OK, "");
    int flag = 0;
    const cudaError_t e = lin_tc_timeout(&flag);
    if (e != cudaSuccess) return cuda_err(e, "timeout mark");
    return flag ? err(M3_ERR_TIMEOUT, "a bounded wait inside a linear attention kernel gave up") : M3_OK;
}

}  // extern "C"
