// Internal declarations of linear attention with a decay for each head: the pass that the
// forward and each gradient run, and its launchers.
//
// One pass. Per sequence and head, with a = e^{log_decay}:
//     y_t = p_scale sum_{s <= t} a^{t - s} (q_t . k_s) v_s + o_scale a^{t + 1} H_in^T q_t
//     H_out = a^n H_in + x_scale sum_s a^{n - 1 - s} k_s v_s^T
// run over the tokens in order or (reverse) from the last one back. The forward is
// (q, k, v) -> o; dq is (do, v, k); dk and dv are (v, do, q) and (k, q, do) in reverse: the
// gradients of a bilinear recurrence are the same recurrence with the operands exchanged.
// The state's columns (of v and y) are independent, so a pass is cut into 64-column tiles.
// Long sequences are cut into segments: a first launch runs each segment's state from zero
// (state_only), and in the second every segment sums its predecessors' end states, decayed.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

namespace m3 {

constexpr int kLinTile = 64;        // columns of v and y one CTA owns
constexpr int kLinMaxSegs = 64;     // segments of one sequence of a batch

struct LinTensor {
    const void* p;
    int64_t batch, token, head;     // strides in elements
    int ratio;                      // head h reads head h / ratio
};

struct LinJob {
    LinTensor q, k, v;
    void* y;
    int64_t y_batch, y_token, y_head;   // head h writes at h * y_head
    int y_f32;                      // y is fp32 (a per-head gradient still to be summed)
    int Dk, Dv, tiles;              // tiles = ceil(Dv / 64)
    int reverse;
    float p_scale, o_scale, x_scale;
    // state before the first token in processing order: element (k, v) of unit u at
    // init[u * Dk * Dv + k * init_k + v * init_v]; in reverse it enters the last token's
    // adjoint undecayed (the recurrence's R_T with a R_T = init)
    const float* init;
    int64_t init_k, init_v;
    float* final_state;             // [unit][Dk][Dv], in reverse times a once more; or null
};

struct LinParams {
    const float* log_decay;
    const int32_t* cu;              // packed sequences, or null
    const int32_t* starts;          // many packed sequences: [nseq + 1], the first block of each, or null
    int nseq, H;
    int64_t L;                      // tokens of each sequence, or rows in all
    int seg_len;                    // tokens of a segment (a multiple of the form's chunk)
    int nseg;                       // segments of every sequence (batches)
    int64_t blocks_x;               // (sequence, segment) pairs, or (packed) a bound of theirs
    int njobs, rtiles;              // rtiles = all jobs' tiles
    float* seg;                     // segment end states, [blocks_x][H][rtiles][seg_rows][64]
    int seg_rows;
    LinJob job[3];
};

// Cuts of nseq sequences of L tokens (packed: L rows in all) into segments of at least min_chunks
// chunks, for `slots` CTAs on the device.
struct LinPlan {
    int seg_len, nseg;
    int64_t blocks_x;
    bool cut;                       // some sequence may have more than one segment
};
struct LinForm {
    int slots, chunk, min_chunks;
    // costs in chunks of the full pass: a CTA's set-up, a chunk of the state-only pass, the sum of one
    // predecessor's end state
    float setup, state_chunk, predecessor;
    float unit;                     // a unit's time on average, as a part of the longest one's
};
LinPlan lin_plan(int64_t nseq, int64_t L, bool packed, int64_t per_x, const LinForm& form);

// (token, head) pairs of the largest bf16 call that the fp32 form takes though the tensor cores could. A score's
// rounding to bf16 is the same for a whole row of the output, and in few rows such roundings do not average out:
// up to 1.5 times the output's own error and more, where it is 1.4 in large calls. (Gradients of 1, 8, 32 tokens of 4 heads,
// K 64, V 64: 11.6, 12.1, 14.7 us in fp32, 7.4, 7.8, 7.8 on the tensor cores; packed 8 x 8 of 4 heads 13.0 and 9.9.)
constexpr int64_t kLinFew = 512;
// Packed sequences up to which each CTA counts blocks itself, which grows with their square; for more a launch
// before it makes the table of first blocks. (Sequences of 4 tokens, 4 heads, counted against table: 64 26 us
// against 31, 192 70 both, 256 91 against 82, 4096 7544 against 1089, 16 384 123 ms against 4.5.)
constexpr int kLinScanned = 256;

// fp32 on the CUDA cores, any dims and strides. Dk: the largest of the jobs; unit: as in LinForm.
LinForm lin_simt_form(int Dk, float unit);
cudaError_t launch_lin_simt(const LinParams& p, bool bf16, bool cut, cudaStream_t s);
// bf16 on the tensor cores: Dk <= 128, 16-byte aligned tensors.
LinForm lin_tc_form();
bool lin_tc_supported(const LinParams& p);
cudaError_t launch_lin_tc(const LinParams& p, bool cut, cudaStream_t s);
cudaError_t lin_tc_timeout(int* flag);   // reads and clears the timeout mark (blocks)

constexpr int kLinShort = 8;        // tokens of the longest prompt that runs as steps
struct LinStep {
    LinTensor q, k, v;
    const float* log_decay;
    const float* state_in;
    float* state_out;
    int64_t nstates;
    const int32_t* slots;
    void* o;
    int64_t o_batch, o_token, o_head;
    int64_t nseq;
    int H, K, V, L;                 // L tokens of each, from 2 on without slots and for V % 4 == 0
    float scale;
};
cudaError_t launch_lin_step(const LinStep& p, bool bf16, cudaStream_t s);

// Raises a kernel's limit of dynamic shared memory to `bytes` (the kernel's largest), once per device.
template <typename K>
cudaError_t allow_smem(K* kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

#ifdef __CUDACC__
// What a CTA's (sequence, segment) index stands for.
struct LinWhere {
    int seq, seg, nseg;
    int row0;           // the sequence's first row (token index inside its batch entry)
    int batch;          // batch entry of the tensors
    int len;            // tokens of the sequence
    bool valid;
};

// A packed sequence's rows, and the segments beyond its first that it asks for.
struct LinSpan {
    int s, e, more;
};
__device__ __forceinline__ LinSpan lin_span(const LinParams& p, int i) {
    const int L = static_cast<int>(p.L);
    LinSpan r;
    r.s = min(max(p.cu[i], 0), L);
    r.e = min(max(p.cu[i + 1], r.s), L);
    r.more = max((r.e - r.s + p.seg_len - 1) / p.seg_len, 1) - 1;
    return r;
}

// Sequence and segment of block x. Packed: the running count of segments, 32 sequences at a
// time (all lanes of a warp call this together), or by halves in the table. The plan reserves a block for each
// sequence and L / seg_len more, which is all that ascending offsets can ask for. Descending ones may overlap and
// ask for any number: the sequence that would go beyond the reserve, and every long one behind it, is
// one segment, however long. So no segment has an index at or above blocks_x, and every sequence runs.
// This is that count in full:
__device__ __forceinline__ void lin_locate_any(const LinParams& p, unsigned x, LinWhere& w) {
    const int lane = threadIdx.x & 31;
    const int64_t reserve = p.blocks_x - p.nseq;
    int64_t before = 0, asked = 0;      // blocks of the sequences before; segments beyond the first they ask for
#pragma unroll 1
    for (int base = 0; base < p.nseq; base += 32) {
        const int i = base + lane, here = min(p.nseq - base, 32);
        LinSpan r{};
        if (i < p.nseq) r = lin_span(p, i);
        int incl = r.more;      // at most 32 * 2^30 / 64
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        // the lanes within the reserve come first: incl ascends
        const unsigned fits = __ballot_sync(0xffffffffu, asked + incl <= reserve);
        const int most = __shfl_sync(0xffffffffu, incl, fits ? 31 - __clz(fits) : 0), cap = fits ? most : 0;
        const int upto = min(lane + 1, here) + min(incl, cap);      // blocks up to and with this lane's sequence
        const unsigned hit = __ballot_sync(0xffffffffu, before + upto > static_cast<int64_t>(x));
        if (hit) {
            const int src = __ffs(hit) - 1, n = (fits >> lane & 1) ? r.more + 1 : 1;
            w.seq = base + src;
            w.seg = static_cast<int>(x - before) - __shfl_sync(0xffffffffu, upto - n, src);
            w.nseg = __shfl_sync(0xffffffffu, n, src);
            w.row0 = __shfl_sync(0xffffffffu, r.s, src);
            w.len = __shfl_sync(0xffffffffu, r.e - r.s, src);
            w.valid = true;
            return;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
        asked += __shfl_sync(0xffffffffu, incl, 31);
    }
}
// and this the one without the bound, which finds the same for a sequence whose segments are within the reserve
// (those before it then are too).
__device__ __forceinline__ LinWhere lin_locate(const LinParams& p, unsigned x) {
    LinWhere w{};
    if (!p.cu) {
        const unsigned nseg = static_cast<unsigned>(p.nseg), seq = x / nseg;
        w.seq = w.batch = static_cast<int>(seq);
        w.seg = static_cast<int>(x - seq * nseg);
        w.nseg = p.nseg;
        w.len = static_cast<int>(p.L);
        w.valid = w.seq < p.nseq;
        return w;
    }
    if (p.starts) {
        const int at = static_cast<int>(x);         // (the grid has fewer than 2^31 blocks)
        if (at >= __ldg(p.starts + p.nseq)) return w;
        int lo = 0, hi = p.nseq;                    // starts[lo] <= at < starts[hi]
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (__ldg(p.starts + m) <= at) lo = m;
            else hi = m;
        }
        const LinSpan r = lin_span(p, lo);
        w.seq = lo;
        w.seg = at - __ldg(p.starts + lo);
        w.nseg = __ldg(p.starts + lo + 1) - __ldg(p.starts + lo);
        w.row0 = r.s;
        w.len = r.e - r.s;
        w.valid = true;
        return w;
    }
    const int lane = threadIdx.x & 31;
    int64_t before = 0;
#pragma unroll 1
    for (int base = 0; base < p.nseq; base += 32) {
        const int i = base + lane;
        LinSpan r{};
        if (i < p.nseq) r = lin_span(p, i);
        const int n = i < p.nseq ? r.more + 1 : 0;
        int incl = n;           // at most 32 (2^30 / 64 + 1)
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + incl > static_cast<int64_t>(x));
        if (hit) {
            const int src = __ffs(hit) - 1;
            w.seq = base + src;
            w.nseg = __shfl_sync(0xffffffffu, n, src);
            const int64_t end = before + __shfl_sync(0xffffffffu, incl, src);
            if (end - w.seq - 1 > p.blocks_x - p.nseq) {
                LinWhere any{};
                lin_locate_any(p, x, any);
                return any;
            }
            w.seg = static_cast<int>(x - (end - w.nseg));
            w.row0 = __shfl_sync(0xffffffffu, r.s, src);
            w.len = __shfl_sync(0xffffffffu, r.e - r.s, src);
            w.valid = true;
            return w;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return w;
}

// The end of a segment that starts at token seg0: the only one of a sequence reaches its end.
__device__ __forceinline__ int64_t lin_seg_end(const LinParams& p, const LinWhere& w, int64_t seg0) {
    const int64_t end = seg0 + p.seg_len;
    return w.nseg == 1 || end > w.len ? w.len : end;
}

// a^n from log2(a): exact at n = 0 whatever a is (a = 0 included).
__device__ __forceinline__ float lin_pow(float g2, float n) { return n == 0.f ? 1.f : exp2f(g2 * n); }

#endif

}  // namespace m3
