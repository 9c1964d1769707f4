// Linear attention's pass on the sm_100a tensor cores (bf16 tensors, Dk <= 128).
//
// One CTA per (sequence, segment, head, 64-column tile of v) and SM; chunks of 128 tokens. With q, k, v
// the pass's operands, H the state (Dk x 64, fp32) and a the head's decay:
//     S  = q k^T                                   M128 N128 K=Dk   (A, B in shared memory)
//     P  = bf16(p_scale a^{|i - j|} S), masked     TMEM -> registers -> TMEM
//     O1 = q bf16(H)                               M128 N64  K=Dk
//     O2 = P v                                     M128 N64  K=128  (A = P in TMEM)
//     y  = o_scale a^{e(i)} O1 + O2
//     H  <- a^n H + k^T v',  v' = x_scale a^{w(j)} v      M128 N=64 parts K=128
// The mask's powers of a multiply the scores in fp32, in two factors per 32 columns that are both at
// most 1 for a <= 1 (a^{t - last column} of the thread's row, a^{last - column} of the column), so
// nothing overflows however strong the decay; the diagonal blocks take theirs from the same table,
// shifted by the row. q, k and v enter the products as stored. Roundings to bf16: P and H as operands of the
// output's products (the output is rounded to bf16 itself), and v' as the sum of bf16 parts: two
// (2^-17) for a state that only feeds bf16 operands, three (2^-25) for one that is returned. The
// parts lie side by side as one operand of 128 or 192 columns, so k is read once for all of them,
// and their products are summed in registers: the tensor core's accumulator drops the bits below
// its sum's last, and a state kept there would shrink by them at every step (relative to
// the state after 4096 tokens with a = 0.9999: 1.5e-6, against 1.7e-7 here).
//
// What bounds it: shared memory and the hand-offs of a chunk, about alike. The products read 1800 cycles
// of shared memory a chunk (S 64 KB, O1 48, k^T v' 80, O2 16, at 128 bytes a cycle); the loads' writes, v',
// its parts and the state's operand take it to some 2900. Measured are 3600 to 3900 cycles from chunk to
// chunk, with the data pipe in front of shared memory and TMEM busy for 78 % of a launch of the gradients (in the
// forward the warps' share of it is 40 %, against 50); 96 KB of HBM (per-head q, k, v and y of K 128, V 64) would
// take 4200 if all 148 SMs asked at once. Only H <- a^n H + ... is serial from chunk to chunk, so everything else runs ahead of it: q, k
// and v are double-buffered, v' and its product do not wait for the state, and S and P of a chunk do not
// wait for the outputs of the one before. A CTA's start (launch, TMEM, tables, first loads, the first
// chunk's chain of products) is some 11 000 cycles until its first output: short sequences are bound by that.
// Measured: 4 x 2048 tokens of 64 heads (K 128, V 64, q and k shared) 84 us, its three gradients with q and
// k of every head 330 us (2.3 TB/s); 65 536 tokens of 64 heads 965 us (3.3 TB/s). These are bursts of four calls;
// for seconds, under the power cap, 90, 370 and 1077.
//
// Warps: 0-3 and 4-7 the rows of the even and of the odd chunks (S -> P, then y), 8-15 the state (in
// registers, half a row a thread), 16-23 v', 24 TMA loads, 25 issues S and O2, 26 O1, 27 k^T v'.
// Hand-offs are mbarriers. All waits are bounded: one that gives up marks the library's timeout word,
// and every role leaves its loop at its next wait.
#include <cstdlib>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "m3_common.cuh"
#include "m3_internal.h"
#include "m3_linattn.h"
#include "m3_sm100.cuh"

namespace m3 {

__device__ int g_lin_timeout;       // set by a wait that gave up

namespace {

using namespace sm100;

constexpr int kC = 128, kVT = kLinTile;
constexpr int kRowWarps = 8, kStateWarp0 = 8, kPartWarp0 = 16, kLoadWarp = 24, kOutWarp = 25, kReadWarp = 26;
constexpr int kThreads = 28 * 32;
constexpr uint32_t kSlab = 16384;                    // 64 columns of 128 rows
// q and k of both stages (two slabs each), v of both stages, the three parts of v', the state's operand
constexpr uint32_t S_Q = 0, S_K = 4 * kSlab, S_V = 8 * kSlab, S_VP = 10 * kSlab, S_H = 13 * kSlab;
constexpr uint32_t kSmem = 14 * kSlab + 1024;
constexpr uint32_t kTmemCols = 512;
// S of both stages (P over its first half, O2 in its second), O1, the products k^T v' of the parts
constexpr uint32_t T_S = 0, T_O2 = 64, T_O1 = 256, T_H = 320;
constexpr int kMaps = 9;

// Pairs alternate with the chunk (phase chunk / 2); the others have a phase per chunk.
enum {
    B_QK, B_QK1, B_V, B_V1,             // loads landed
    B_S, B_S1, B_O1, B_O11, B_O2, B_O21, B_DH,      // products done
    B_P, B_P1, B_H0, B_VP,              // operands written: P, the state's, v'
    B_SFREE, B_SFREE1, B_OFREE, B_HFREE,            // accumulators read: S and O2, O1, k^T v'
    B_QKFREE, B_QKFREE1, B_VFREE, B_VFREE1,         // stages free for the next load
    B_CLEAN,                            // rows behind the last token zeroed (once)
    B_DRAIN, B_DRAIN1, B_DRAIN2, kNumBars
};
__host__ __device__ constexpr uint32_t bar_count(int b) {
    return (b == B_H0 || b == B_VP || b == B_HFREE || b == B_CLEAN) ? 8
         : (b == B_P || b == B_P1 || b == B_SFREE || b == B_SFREE1 || b == B_OFREE) ? 4
         : (b == B_QKFREE || b == B_QKFREE1) ? 3      // S, O1 and k^T v' done
         : (b == B_VFREE || b == B_VFREE1) ? 9        // read by the v' warps, O2 done
         : 1;
}

struct LinMaps {
    CUtensorMap m[kMaps];
};
struct LinTcParams {
    LinParams p;
    int map[3][3];              // [job][q, k, v]
    int head_ratio[3][3];       // head coordinate = h / ratio
    int batched[3][3];          // batch coordinate = sequence (0: one entry for all)
    int parts[3];               // bf16 parts of v'
    // Test hook: > 0 makes CTA 0 skip the load of that chunk's v, so that its bounded waits run out and
    // the timeout path is exercised. Set only from the M3_TEST_LINATTN_SKIP_LOAD environment variable.
    int test_skip;
};

// Waits for the phase of `bar` with the given parity, giving up after kMaxPolls polls (the thread is
// suspended for up to a microsecond in each: about a second). The loop is in the code a dozen times,
// so it reads neither a clock nor the flag: a role that gave up makes the others run out of polls too.
constexpr int kMaxPolls = 1 << 21;
constexpr long long kDrainCycles = 200000000LL;
__device__ __forceinline__ bool lwait(uint64_t* bar, int parity, volatile int* abort_flag) {
    const uint32_t a = smem_u32(bar);
#pragma unroll 1
    for (int i = 0; i < kMaxPolls; ++i)
        if (mbar_try_wait_sleep(a, parity & 1, 1000u)) return true;
    *abort_flag = 1;
    return false;
}
// The same for a whole warp, with one answer for all of its lanes.
__device__ __forceinline__ bool lwait_warp(uint64_t* bar, int parity, volatile int* abort_flag) {
    return __all_sync(0xffffffffu, lwait(bar, parity, abort_flag));
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(const float2& v) { return pack2(v.x, v.y); }
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// The products and commits below run in convergent code of one warp, predicated on its first lane
// (`el`), so that descriptors stay in uniform registers: inside a branch of one lane each product
// took some 200 cycles to issue.
// Four K steps of one product: descriptors given by their low words (the high word is the layout's),
// which advance by kA and kB a step; the first step accumulates if acc.
template <uint32_t kA, uint32_t kB>
__device__ __forceinline__ void mma4_el(uint32_t el, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    constexpr uint32_t hi = desc_hi_sw128(1024);
    asm volatile(
        "{\n\t.reg .pred p, q, t;\n\t.reg .b64 x, y;\n\t.reg .b32 u, v;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "mov.b64 x, {%1, %6};\n\tmov.b64 y, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t"
        "add.u32 u, %1, %7;\n\tadd.u32 v, %2, %8;\n\tmov.b64 x, {u, %6};\n\tmov.b64 y, {v, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
        "add.u32 u, %1, %9;\n\tadd.u32 v, %2, %10;\n\tmov.b64 x, {u, %6};\n\tmov.b64 y, {v, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
        "add.u32 u, %1, %11;\n\tadd.u32 v, %2, %12;\n\tmov.b64 x, {u, %6};\n\tmov.b64 y, {v, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t}\n"
        :: "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(el), "r"(hi), "n"(kA), "n"(kB), "n"(2 * kA), "n"(2 * kB),
           "n"(3 * kA), "n"(3 * kB));
}
// The same with the A operand in TMEM, eight columns a step.
template <uint32_t kB>
__device__ __forceinline__ void mma4_ts_el(uint32_t el, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    constexpr uint32_t hi = desc_hi_sw128(1024);
    asm volatile(
        "{\n\t.reg .pred p, q, t;\n\t.reg .b64 y;\n\t.reg .b32 u, v;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "mov.b64 y, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t"
        "add.u32 u, %1, 8;\n\tadd.u32 v, %2, %7;\n\tmov.b64 y, {v, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %3, t;\n\t"
        "add.u32 u, %1, 16;\n\tadd.u32 v, %2, %8;\n\tmov.b64 y, {v, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %3, t;\n\t"
        "add.u32 u, %1, 24;\n\tadd.u32 v, %2, %9;\n\tmov.b64 y, {v, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %3, t;\n\t}\n"
        :: "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(el), "r"(hi), "n"(kB), "n"(2 * kB), "n"(3 * kB));
}
// Steps of the operands' low words: 16 columns of a row (K-major), 16 rows (MN-major)
constexpr uint32_t kStepK = 2, kStepMN = 128, kNextSlab = kSlab >> 4;
__device__ __forceinline__ void commit_el(uint32_t el, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n"
        :: "r"(smem_u32(bar)), "r"(el) : "memory");
}

// The 72 registers a thread that 28 warps leave are dealt out again by what the roles hold. Spills are
// what to avoid: beside 227 KB of shared memory the L1 cache is too small to hold them.
constexpr int kRegsLaunch = 72, kRegsRow = 88, kRegsState = 64, kRegsPart = 80, kRegsIssue = 40;
static_assert(2 * kRegsRow + 2 * kRegsState + 2 * kRegsPart + kRegsIssue == 7 * kRegsLaunch,
              "an increase beyond what the block was launched with would wait for ever");
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N));
}

// 32 bytes to global memory (32-byte aligned)
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// 32 lanes x 32 bits, 8 consecutive columns: thread i of the warp gets lane (base + i).
__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

constexpr float kInf = __builtin_huge_valf();

// The outputs of a warp's 32 rows from P, O2 (lp) and O1 (lo) in TMEM and v in global memory: where O2 is not
// finite, row t's sum over the tokens up to its own alone. v: the chunk's first token; y: this thread's row.
__device__ __noinline__ void sum_rows(const LinJob& j, const __nv_bfloat16* v, uint8_t* y, uint32_t lp, uint32_t lo, int t,
                                      int n, int cols, float f1) {
#pragma unroll 1
    for (int c = 0; c < kVT && c < cols; c += 8) {
        float o[8], a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = 0.f;
#pragma unroll 1
        for (int s0 = 0; s0 < n; s0 += 32) {
            float p[16];        // 32 tokens' scores
            tmem_ld_32x32b_x16(lp + (s0 >> 1), p);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                const int s = s0 + k;
                const uint4 raw = s < n ? *reinterpret_cast<const uint4*>(v + s * j.v.token + c) : make_uint4(0u, 0u, 0u, 0u);
                // (selects, not a branch: the loads from TMEM need the whole warp)
                const uint32_t on = (s < n && (j.reverse ? s >= t : s <= t)) ? 0xFFFFFFFFu : 0u, p2 = __float_as_uint(p[k >> 1]);
                const float pr = __uint_as_float((k & 1 ? p2 & 0xFFFF0000u : p2 << 16) & on);
                const uint32_t u[4] = {raw.x & on, raw.y & on, raw.z & on, raw.w & on};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack2(u[i]);
                    o[2 * i] = fmaf(pr, f.x, o[2 * i]);
                    o[2 * i + 1] = fmaf(pr, f.y, o[2 * i + 1]);
                }
            }
        }
        tmem_ld_x8(lp + T_O2 + c, a);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = fabsf(a[i]) < kInf ? a[i] : o[i];
        tmem_ld_x8(lo + c, a);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = fmaf(f1, a[i], o[i]);
        if (t >= n) {
            // (no token)
        } else if (j.y_f32) {
            float4* at = reinterpret_cast<float4*>(y + 4 * c);
            at[0] = make_float4(o[0], o[1], o[2], o[3]);
            at[1] = make_float4(o[4], o[5], o[6], o[7]);
        } else {
            *reinterpret_cast<uint4*>(y + 2 * c) = make_uint4(pack2(o[0], o[1]), pack2(o[2], o[3]), pack2(o[4], o[5]), pack2(o[6], o[7]));
        }
        __syncwarp();
    }
}

template <bool kStateOnly>
__global__ void __launch_bounds__(kThreads, 1)
lin_tc_kernel(const __grid_constant__ LinTcParams tp, const __grid_constant__ LinMaps maps) {
    const LinParams& p = tp.p;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t bars[kNumBars];
    __shared__ __align__(16) float pw[kC + 4];
    // a^{31 - k} (reverse: a^{k - 31}), zero where the exponent is negative: entries 31 - r + i are row r
    // of the mask's diagonal blocks; and the columns' factors of the other blocks, a^{31 - i} (a^i)
    __shared__ float mask[64];
    __shared__ __align__(16) float colw[32];
    __shared__ uint32_t tslot;
    __shared__ volatile int s_abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const unsigned per_x = static_cast<unsigned>(p.H) * p.rtiles;
    const unsigned x = blockIdx.x / per_x;
    const int rem = static_cast<int>(blockIdx.x - x * per_x);
    const int h = rem / p.rtiles, rt = rem % p.rtiles;
    int ji = 0, tile = rt;
    while (ji + 1 < p.njobs && tile >= p.job[ji].tiles) tile -= p.job[ji++].tiles;
    const LinJob& j = p.job[ji];
    const LinWhere w = lin_locate(p, x);
    if (!w.valid) return;
    if (kStateOnly) grid_dep_launch_dependents();
    const bool rev = j.reverse;
    const int order = rev ? w.nseg - 1 - w.seg : w.seg;
    const bool last_seg = order == w.nseg - 1;
    if (kStateOnly && last_seg) return;              // nobody reads the last one's
    const int seg0 = w.seg * p.seg_len;
    const int seg_end = static_cast<int>(lin_seg_end(p, w, seg0));
    const int nchunks = (seg_end - seg0 + kC - 1) / kC;
    const bool want_final = !kStateOnly && j.final_state && last_seg;
    // chunks whose state product runs: the last one's only for a state that somebody wants
    const int nupdates = (kStateOnly || want_final) ? nchunks : nchunks - 1;
    const int slabs = j.Dk > 64 ? 2 : 1;     // of 64 columns of q and k (zeros beyond Dk)
    const int parts = tp.parts[ji];
    const float g2 = p.log_decay[h] * 1.4426950408889634f;
    // token 0 and length of the c-th chunk in processing order
    auto chunk_t0 = [&](int c) { return seg0 + kC * (rev ? nchunks - 1 - c : c); };
    auto chunk_n = [&](int c) { const int n = seg_end - chunk_t0(c); return n < kC ? n : kC; };

    // ---------------- set-up ----------------
    // The load warp needs nothing but its barriers: its first loads are issued ahead of the block's
    // barrier, while other warps allocate TMEM and fill the tables.
    const int nloads = kStateOnly ? nupdates : nchunks;
    int hq = 0, hk = 0, hv_ = 0, bq = 0, bk = 0, bv = 0;
    const void *mq = nullptr, *mk = nullptr, *mv = nullptr;
    auto load = [&](int c) {
        const int st = c & 1, at = w.row0 + chunk_t0(c);
        if (c > 1 && !lwait(&bars[B_QKFREE + st], (c >> 1) - 1, &s_abort)) return false;
        mbar_arrive_expect_tx(&bars[B_QK + st], (kStateOnly ? 1 : 2) * slabs * kSlab);
#pragma unroll 1
        for (int s = 0; s < slabs; ++s) {
            tma_load_4d(sm + S_K + (2 * st + s) * kSlab, mk, &bars[B_QK + st], 64 * s, hk, at, bk);
            if (!kStateOnly) tma_load_4d(sm + S_Q + (2 * st + s) * kSlab, mq, &bars[B_QK + st], 64 * s, hq, at, bq);
        }
        if (c > 1 && !lwait(&bars[B_VFREE + st], (c >> 1) - 1, &s_abort)) {
            (void)mbar_wait(&bars[B_QK + st], (c >> 1) & 1, kDrainCycles);
            return false;
        }
        if (blockIdx.x == 0 && c > 0 && c == tp.test_skip) return true;     // (test hook)
        mbar_arrive_expect_tx(&bars[B_V + st], kSlab);
        tma_load_4d(sm + S_V + st * kSlab, mv, &bars[B_V + st], tile * kVT, hv_, at, bv);
        return true;
    };
    if (warp == kLoadWarp) {
        if (lane == 0) {
            mq = &maps.m[tp.map[ji][0]];
            mk = &maps.m[tp.map[ji][1]];
            mv = &maps.m[tp.map[ji][2]];
            asm volatile("prefetch.tensormap [%0];" :: "l"(mk) : "memory");
            if (!kStateOnly) asm volatile("prefetch.tensormap [%0];" :: "l"(mq) : "memory");
            asm volatile("prefetch.tensormap [%0];" :: "l"(mv) : "memory");
            for (int i = 0; i < kNumBars; ++i) mbar_init(&bars[i], bar_count(i));
            fence_mbar_init();
            fence_proxy_async();
            hq = h / tp.head_ratio[ji][0];
            hk = h / tp.head_ratio[ji][1];
            hv_ = h / tp.head_ratio[ji][2];
            bq = tp.batched[ji][0] ? w.batch : 0;
            bk = tp.batched[ji][1] ? w.batch : 0;
            bv = tp.batched[ji][2] ? w.batch : 0;
            if (nloads > 0) load(0);
        }
        __syncwarp();
    } else if (warp == kOutWarp) {
        if (lane == 0) s_abort = 0;
        tmem_alloc(&tslot, kTmemCols);
    }
    if (tid <= kC) pw[tid] = lin_pow(g2, static_cast<float>(tid));
    if (tid >= 256 && tid < 320) {
        const int d = rev ? tid - 287 : 287 - tid;
        const float m = d >= 0 ? lin_pow(g2, static_cast<float>(d)) : 0.f;
        mask[tid - 256] = m;
        if (rev ? tid >= 287 && tid < 319 : tid < 288) colw[rev ? tid - 287 : tid - 256] = m;
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = tslot;

    if (warp < kRowWarps) {
        // ================= rows: S -> P, then y =================
        if constexpr (!kStateOnly) regs_inc<kRegsRow>();
        if (!kStateOnly) {
            const int g = warp >> 2, rw = warp & 3, t = 32 * rw + lane;
            const uint32_t ls = tmem + ((32u * rw) << 16) + T_S + 128u * g;     // S, P and (+64) O2
            const uint32_t lo = tmem + ((32u * rw) << 16) + T_O1;
            const float ps = j.p_scale;
            const int sgn = rev ? 1 : -1;
            const int es = j.y_f32 ? 4 : 2;
            const int cols = j.Dv - tile * kVT;
            uint8_t* ybase = static_cast<uint8_t*>(j.y) +
                             (w.batch * j.y_batch + w.row0 * j.y_token + h * j.y_head + tile * kVT) * es;
            // whether every row's pieces are whole 32-byte sectors
            const bool wide = ((reinterpret_cast<uintptr_t>(ybase) | static_cast<uintptr_t>(j.y_token * es)) & 31u) == 0;
            // what the output adds to P v: the state's share of row t
            auto state_factor = [&](int c) {
                const int e = (rev ? chunk_n(c) - t : t + 1) - ((rev && order == 0 && c == 0) ? 1 : 0);
                return j.o_scale * pw[e < 0 ? 0 : e];
            };
            int c = g;
            // P v runs over all of the chunk's tokens, and zero times what is not finite is NaN: a later token's
            // would reach the rows before it (and a growing decay's overflow, from tokens that are not there).
            // A warp that finds such sums leaves the loop, sums its rows again over the tokens up to theirs,
            // and comes back: inside the loop the sums' 64 registers would be spilled around that. The look costs
            // nothing in the forward and 4 % in the gradients (316 -> 330 us for 4 x 2048 tokens of 64 heads),
            // where it delays O1's release. Elsewhere it cost more: v looked through by the v' warps, which run
            // behind P, 350 us; O2 read before O1 is there, 368.
            bool again;
#pragma unroll 1
            do {
                again = false;
#pragma unroll 1
                for (; c < nchunks; c += 2) {
                    const int t0 = chunk_t0(c), n = chunk_n(c);
                    if (!lwait_warp(&bars[B_S + g], c >> 1, &s_abort)) break;
                    fence_after_sync();
                    // 32 columns at a time, as far as the product reads (scores behind the last token are zero)
#pragma unroll 1
                    for (int b = 0; b < (n > 64 ? 4 : 2); ++b) {
                        uint32_t pk[16];
                        const int ahead = sgn * (b - rw);           // 0: the diagonal block
                        if (ahead < 0) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) pk[i] = 0u;
                        } else {
                            float v[32];
                            tmem_ld_32x32b_x32(ls + 32u * b, v);
                            if (ahead > 0) {
                                const float f = ps * pw[sgn * (32 * b - t) - (rev ? 0 : 31)];
                                const float2 f2 = make_float2(f, f);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const float4 m = reinterpret_cast<const float4*>(colw)[i];
                                    pk[2 * i] = pack2(__fmul2_rn(__fmul2_rn(make_float2(v[4 * i], v[4 * i + 1]), f2), make_float2(m.x, m.y)));
                                    pk[2 * i + 1] = pack2(__fmul2_rn(__fmul2_rn(make_float2(v[4 * i + 2], v[4 * i + 3]), f2), make_float2(m.z, m.w)));
                                }
                            } else {
                                const float* m = mask + 31 - lane;
                                const float2 f2 = make_float2(ps, ps);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    pk[i] = pack2(__fmul2_rn(__fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), f2),
                                                             make_float2(m[2 * i], m[2 * i + 1])));
                            }
                        }
                        // block b of P lies over S's block b / 2, which has been read
                        tmem_st_32x32b_x16(ls + 16u * b, pk);
                    }
                    tmem_wait_st();
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[B_P + g]);
                    const float f1 = state_factor(c);
                    uint8_t* y = ybase + static_cast<int64_t>(t0 + t) * j.y_token * es;
                    if (!lwait_warp(&bars[B_O1 + g], c >> 1, &s_abort) || !lwait_warp(&bars[B_O2 + g], c >> 1, &s_abort)) break;
                    fence_after_sync();
                    float most = 0.f;       // of the sums of O2, NaN if one is
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
                        float a[32], o[32];
                        tmem_ld_32x32b_x32(lo + 32u * q, a);
                        tmem_ld_32x32b_x32(ls + T_O2 + 32u * q, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i += 2) asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(most) : "f"(o[i]), "f"(o[i + 1]));
                        if (q == 1) {
                            again = __any_sync(0xffffffffu, !(most < kInf));
                            if (again) break;
                            // O1, O2 and P have been read
                            fence_before_sync();
                            __syncwarp();
                            if (lane == 0) {
                                mbar_arrive(&bars[B_OFREE]);
                                mbar_arrive(&bars[B_SFREE + g]);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 y2 = __ffma2_rn(make_float2(f1, f1), make_float2(a[i], a[i + 1]), make_float2(o[i], o[i + 1]));
                            o[i] = y2.x;
                            o[i + 1] = y2.y;
                        }
                        const int left = t < n ? cols - 32 * q : 0;
                        if (j.y_f32) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t u[8];
#pragma unroll
                                for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(o[8 * i + k]);
                                if (8 * i < left) store32(y + 128 * q + 32 * i, u);     // always whole sectors
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint32_t u[8];
#pragma unroll
                                for (int k = 0; k < 8; ++k) u[k] = pack2(o[16 * i + 2 * k], o[16 * i + 2 * k + 1]);
                                uint8_t* at = y + 64 * q + 32 * i;
                                if (wide && left >= 16 * i + 16) {
                                    store32(at, u);
                                } else {
                                    if (left > 16 * i) *reinterpret_cast<uint4*>(at) = make_uint4(u[0], u[1], u[2], u[3]);
                                    if (left > 16 * i + 8) *reinterpret_cast<uint4*>(at + 16) = make_uint4(u[4], u[5], u[6], u[7]);
                                }
                            }
                        }
                    }
                    if (again) break;
                }
                if (again) {
                    const int t0 = chunk_t0(c), n = chunk_n(c);
                    sum_rows(j, static_cast<const __nv_bfloat16*>(j.v.p) + w.batch * j.v.batch + (w.row0 + t0) * j.v.token +
                                    (h / j.v.ratio) * j.v.head + tile * kVT,
                             ybase + static_cast<int64_t>(t0 + t) * j.y_token * es, ls, lo, t, n, cols, state_factor(c));
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bars[B_OFREE]);
                        mbar_arrive(&bars[B_SFREE + g]);
                    }
                    c += 2;
                }
            } while (again);
        }
    } else if (warp < kPartWarp0) {
        // ================= the state: half of row r (32 columns) in a thread's registers =================
        if constexpr (!kStateOnly) regs_dec<kRegsState>();
        const int r = 32 * (warp & 3) + lane, c0 = (warp - kStateWarp0) >> 2 << 5;
        const uint32_t lb = tmem + ((32u * (warp & 3)) << 16) + T_H + c0;
        const int cols = j.Dv - tile * kVT - c0;        // of this thread's that exist
        float hv[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) hv[i] = 0.f;
        // the state as the next chunk's bf16 operand
        auto publish = [&]() {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4*>(sm + S_H + swz128(r, c0 + 8 * i)) =
                    make_uint4(pack2(hv[8 * i], hv[8 * i + 1]), pack2(hv[8 * i + 2], hv[8 * i + 3]),
                               pack2(hv[8 * i + 4], hv[8 * i + 5]), pack2(hv[8 * i + 6], hv[8 * i + 7]));
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_H0]);
        };
        if (!kStateOnly) {
            // the state before this segment: the given one and the segments before, decayed
            const int before = rev ? (order == 0 ? 0 : w.len - (seg0 + p.seg_len)) : seg0;
            const float fi = lin_pow(g2, static_cast<float>(rev && before > 0 ? before - 1 : before));
            const bool live = r < j.Dk;
            if (j.init && live && fi != 0.f) {
                const float* src = j.init + (static_cast<int64_t>(w.seq) * p.H + h) * j.Dk * j.Dv + r * j.init_k +
                                   (tile * kVT + c0) * j.init_v;
                if (j.init_v == 1) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        if (i < cols) {         // Dv is a multiple of 8
                            const float4 v4 = *reinterpret_cast<const float4*>(src + i);
                            hv[i] = fi * v4.x; hv[i + 1] = fi * v4.y; hv[i + 2] = fi * v4.z; hv[i + 3] = fi * v4.w;
                        }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i, src += j.init_v)
                        if (i < cols) hv[i] = fi * *src;
                }
            }
            if (order > 0) grid_dep_wait();     // the segments' end states are there
#pragma unroll 1
            for (int o = 0; o < order && live; ++o) {
                const int sg = rev ? w.nseg - 1 - o : o;
                const int gap = rev ? sg * p.seg_len - (seg0 + p.seg_len) : seg0 - (sg + 1) * p.seg_len;
                const float f = lin_pow(g2, static_cast<float>(gap));
                if (f == 0.f) continue;
                const float* e = p.seg + (((static_cast<int64_t>(x - w.seg + sg) * p.H + h) * p.rtiles + rt) * p.seg_rows + r) * kVT + c0;
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 v4 = *reinterpret_cast<const float4*>(e + i);
                    hv[i] = fmaf(f, v4.x, hv[i]); hv[i + 1] = fmaf(f, v4.y, hv[i + 1]);
                    hv[i + 2] = fmaf(f, v4.z, hv[i + 2]); hv[i + 3] = fmaf(f, v4.w, hv[i + 3]);
                }
            }
            __syncwarp();
            if (nchunks > 0) publish();
        }
        bool good = true;
#pragma unroll 1
        for (int c = 0; c < nupdates; ++c) {
            const float decay = pw[chunk_n(c) - ((rev && order == 0 && c == 0) ? 1 : 0)];
            if (!lwait_warp(&bars[B_DH], c, &s_abort)) { good = false; break; }
            fence_after_sync();
#pragma unroll 1
            for (int part = 0; part < parts; ++part) {
                const float dc = part == 0 ? decay : 1.f;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float d[16];
                    tmem_ld_32x32b_x16(lb + 64u * part + 16u * q, d);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        float* at = hv + 16 * q + i;
                        const float2 h2 = __ffma2_rn(make_float2(dc, dc), make_float2(at[0], at[1]), make_float2(d[i], d[i + 1]));
                        at[0] = h2.x;
                        at[1] = h2.y;
                    }
                }
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_HFREE]);
            if (kStateOnly || c + 1 >= nchunks) continue;
            // the next chunk's operand, once O1 has read this chunk's
            if (!lwait_warp(&bars[B_O1 + (c & 1)], c >> 1, &s_abort)) { good = false; break; }
            publish();
        }
        if (good && (kStateOnly || want_final)) {
            // through the accumulator once more, so that the copy out is a short loop
            // (an empty sequence's state passes through)
            const float ff = rev && w.len > 0 && !kStateOnly ? pw[1] : 1.f;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t u[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(ff * hv[16 * q + i]);
                tmem_st_32x32b_x16(lb + 16u * q, u);
            }
            tmem_wait_st();
            float* dst = kStateOnly ? p.seg + (((static_cast<int64_t>(x) * p.H + h) * p.rtiles + rt) * p.seg_rows + r) * kVT + c0
                                    : j.final_state + ((static_cast<int64_t>(w.seq) * p.H + h) * j.Dk + r) * j.Dv +
                                          tile * kVT + c0;
            const int lim = r >= j.Dk ? 0 : (kStateOnly ? 32 : cols);
#pragma unroll 1
            for (int c = 0; c < 32; c += 16) {
                float v[16];
                tmem_ld_32x32b_x16(lb + c, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    if (c + i < lim)
                        *reinterpret_cast<float4*>(dst + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
        }
    } else if (warp < kLoadWarp) {
        // ================= v', the weighted v in bf16 parts =================
        if constexpr (!kStateOnly) regs_inc<kRegsPart>();
        // Half of token r's columns a thread. The parts are formed in registers while the product of
        // the chunk before still reads theirs.
        const int r = 32 * (warp & 3) + lane, half = (warp - kPartWarp0) >> 2;
#pragma unroll 1
        for (int c = 0; c < nchunks; ++c) {
            const int st = c & 1, n = chunk_n(c);
            if (c >= nupdates && (n == kC || !p.cu)) break;
            if (!lwait_warp(&bars[B_V + st], c >> 1, &s_abort)) break;
            if (n < kC && p.cu) {
                // Packed: rows of k and v behind the last token, another sequence's or anything, become zeros
                // before a product reads them: their weights are, but zero times NaN is not. (In a batch they
                // lie outside the tensor map, whose loads fill in zeros.)
                if (!lwait_warp(&bars[B_QK + st], c >> 1, &s_abort)) break;
                if (r >= n) {
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        *reinterpret_cast<uint4*>(sm + S_K + (2 * st + half) * kSlab + r * 128 + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
                        if (i < 4)
                            *reinterpret_cast<uint4*>(sm + S_V + st * kSlab + swz128(r, 32 * half + 8 * i)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_CLEAN]);
                if (c >= nupdates) break;
            }
            const float wt = r < n ? j.x_scale * pw[rev ? r : n - 1 - r] : 0.f;
            uint32_t p0[16], p1[16], p2[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 raw = *reinterpret_cast<const uint4*>(sm + S_V + st * kSlab + swz128(r, 32 * half + 8 * i));
                p0[4 * i] = raw.x; p0[4 * i + 1] = raw.y; p0[4 * i + 2] = raw.z; p0[4 * i + 3] = raw.w;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_VFREE + st]);
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const float2 ab = __fmul2_rn(make_float2(wt, wt), unpack2(p0[u])), minus = make_float2(-1.f, -1.f);
                p0[u] = pack2(ab);
                const float2 ab1 = __ffma2_rn(unpack2(p0[u]), minus, ab);       // exact
                p1[u] = pack2(ab1);
                p2[u] = pack2(__ffma2_rn(unpack2(p1[u]), minus, ab1));
            }
            if (c > 0 && !lwait_warp(&bars[B_DH], c - 1, &s_abort)) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint8_t* at = sm + S_VP + swz128(r, 32 * half + 8 * i);
                *reinterpret_cast<uint4*>(at) = make_uint4(p0[4 * i], p0[4 * i + 1], p0[4 * i + 2], p0[4 * i + 3]);
                *reinterpret_cast<uint4*>(at + kSlab) = make_uint4(p1[4 * i], p1[4 * i + 1], p1[4 * i + 2], p1[4 * i + 3]);
                if (parts > 2)
                    *reinterpret_cast<uint4*>(at + 2 * kSlab) = make_uint4(p2[4 * i], p2[4 * i + 1], p2[4 * i + 2], p2[4 * i + 3]);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_VP]);
        }
    } else {
        if constexpr (!kStateOnly) regs_dec<kRegsIssue>();
        if (warp == kLoadWarp) {
            // ================= TMA loads (one lane) =================
            if (lane == 0) {
                int done = nloads < 1 ? nloads : 1;
#pragma unroll 1
                for (int c = done; c < nloads; ++c) {
                    if (!load(c)) break;
                    done = c + 1;
                }
                // every copy has landed before the CTA exits (at once, unless a wait gave up)
                for (int c = done > 2 ? done - 2 : 0; c < done; ++c) {
                    (void)mbar_wait(&bars[B_QK + (c & 1)], (c >> 1) & 1, kDrainCycles);
                    (void)mbar_wait(&bars[B_V + (c & 1)], (c >> 1) & 1, kDrainCycles);
                }
            }
            __syncwarp();
        } else if (warp == kOutWarp) {
            // ================= S and O2 (issued by the first lane) =================
            // Every commit is waited for by somebody: one that arrived after the CTA's end would write
            // into the next one's barriers.
            if (!kStateOnly) {
                const uint32_t el = lane == 0;
                constexpr uint32_t id_s = idesc_bf16(128, 128, false, false);
                constexpr uint32_t id_o = idesc_bf16(128, 64, false, true);
                bool issued = false;
#pragma unroll 1
                for (int c = -1; c < nchunks; ++c) {
                    if (c + 1 < nchunks) {
                        const int st = (c + 1) & 1, ph = (c + 1) >> 1;
                        if (!lwait_warp(&bars[B_QK + st], ph, &s_abort)) break;
                        if (c > 0 && !lwait_warp(&bars[B_SFREE + st], ph - 1, &s_abort)) break;
                        if (p.cu && chunk_n(c + 1) < kC && !lwait_warp(&bars[B_CLEAN], 0, &s_abort)) break;
                        fence_after_sync();
                        issued = true;
                        const uint32_t loQ = desc_lo(smem_u32(sm + S_Q + 2 * st * kSlab), 16);
                        const uint32_t loK = desc_lo(smem_u32(sm + S_K + 2 * st * kSlab), 16);
                        mma4_el<kStepK, kStepK>(el, tmem + T_S + 128u * st, loQ, loK, id_s, 0);
                        if (slabs == 2)
                            mma4_el<kStepK, kStepK>(el, tmem + T_S + 128u * st, loQ + kNextSlab, loK + kNextSlab, id_s, 1);
                        commit_el(el, &bars[B_S + st]);
                        if (c + 3 < nchunks) commit_el(el, &bars[B_QKFREE + st]);
                    }
                    if (c >= 0) {
                        const int st = c & 1, ph = c >> 1;
                        const bool far = chunk_n(c) > 64;       // tokens in the chunk's second half
                        if (!lwait_warp(&bars[B_P + st], ph, &s_abort) || !lwait_warp(&bars[B_V + st], ph, &s_abort)) break;
                        fence_after_sync();
                        const uint32_t loV = desc_lo(smem_u32(sm + S_V + st * kSlab), kSlab);
                        mma4_ts_el<kStepMN>(el, tmem + T_S + 128u * st + T_O2, tmem + T_S + 128u * st, loV, id_o, 0);
                        if (far)
                            mma4_ts_el<kStepMN>(el, tmem + T_S + 128u * st + T_O2, tmem + T_S + 128u * st + 32u,
                                                loV + 4 * kStepMN, id_o, 1);
                        commit_el(el, &bars[B_O2 + st]);
                        if (c + 2 < nchunks) commit_el(el, &bars[B_VFREE + st]);
                    }
                }
                if (s_abort && issued) {    // products in flight end before their TMEM is released
                    commit_el(el, &bars[B_DRAIN]);
                    (void)mbar_wait(&bars[B_DRAIN], 0, kDrainCycles);
                }
            }
        } else if (warp == kReadWarp) {
            // ================= O1 (issued by the first lane) =================
            if (!kStateOnly) {
                const uint32_t el = lane == 0;
                constexpr uint32_t id_o = idesc_bf16(128, 64, false, true);
                const uint32_t loH = desc_lo(smem_u32(sm + S_H), kSlab);
                bool issued = false;
#pragma unroll 1
                for (int c = 0; c < nchunks; ++c) {
                    const int st = c & 1;
                    if (!lwait_warp(&bars[B_QK + st], c >> 1, &s_abort) || !lwait_warp(&bars[B_H0], c, &s_abort) ||
                        (c > 0 && !lwait_warp(&bars[B_OFREE], c - 1, &s_abort)))
                        break;
                    fence_after_sync();
                    issued = true;
                    const uint32_t loQ = desc_lo(smem_u32(sm + S_Q + 2 * st * kSlab), 16);
                    mma4_el<kStepK, kStepMN>(el, tmem + T_O1, loQ, loH, id_o, 0);
                    if (slabs == 2) mma4_el<kStepK, kStepMN>(el, tmem + T_O1, loQ + kNextSlab, loH + 4 * kStepMN, id_o, 1);
                    commit_el(el, &bars[B_O1 + st]);
                    if (c + 2 < nchunks) commit_el(el, &bars[B_QKFREE + st]);
                }
                if (s_abort && issued) {
                    commit_el(el, &bars[B_DRAIN1]);
                    (void)mbar_wait(&bars[B_DRAIN1], 0, kDrainCycles);
                }
            }
        } else {
            // ================= k^T v' (issued by the first lane) =================
            {
                const uint32_t el = lane == 0;
                const uint32_t id_h = parts > 2 ? idesc_bf16(128, 192, true, true) : idesc_bf16(128, 128, true, true);
                const uint32_t loVP = desc_lo(smem_u32(sm + S_VP), kSlab);
                bool issued = false;
#pragma unroll 1
                for (int c = 0; c < nupdates; ++c) {
                    const int st = c & 1;
                    const bool far = chunk_n(c) > 64;
                    if (!lwait_warp(&bars[B_QK + st], c >> 1, &s_abort) || !lwait_warp(&bars[B_VP], c, &s_abort) ||
                        (c > 0 && !lwait_warp(&bars[B_HFREE], c - 1, &s_abort)))
                        break;
                    fence_after_sync();
                    issued = true;
                    const uint32_t loK = desc_lo(smem_u32(sm + S_K + 2 * st * kSlab), kSlab);
                    mma4_el<kStepMN, kStepMN>(el, tmem + T_H, loK, loVP, id_h, 0);
                    if (far) mma4_el<kStepMN, kStepMN>(el, tmem + T_H, loK + 4 * kStepMN, loVP + 4 * kStepMN, id_h, 1);
                    commit_el(el, &bars[B_DH]);
                    if (c + 2 < nchunks) {
                        commit_el(el, &bars[B_QKFREE + st]);
                        if (kStateOnly && el) { // nobody else reads a stage
                            mbar_arrive(&bars[B_QKFREE + st]);
                            mbar_arrive(&bars[B_QKFREE + st]);
                            mbar_arrive(&bars[B_VFREE + st]);
                        }
                    }
                }
                if (s_abort && issued) {
                    commit_el(el, &bars[B_DRAIN2]);
                    (void)mbar_wait(&bars[B_DRAIN2], 0, kDrainCycles);
                }
            }
        }
    }

    // no CTA ends before the launch before it: what comes after this grid comes after both
    if (!kStateOnly && tid == 0) grid_dep_wait();
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (s_abort && tid == 0) atomicExch(&g_lin_timeout, 1);
    if (warp == kOutWarp) tmem_dealloc(tmem, kTmemCols);
}

bool aligned(const LinTensor& t) {
    return ((reinterpret_cast<uintptr_t>(t.p) | static_cast<uintptr_t>(t.batch * 2) |
             static_cast<uintptr_t>(t.token * 2) | static_cast<uintptr_t>(t.head * 2)) & 15u) == 0;
}

// Strides a tensor map can hold: below 2^40 bytes, and rows that do not repeat (a broadcast head or
// batch entry becomes a dimension of one).
bool mappable(const LinTensor& t, int64_t L) {
    const int64_t lim = int64_t(1) << 38;
    return aligned(t) && t.batch >= 0 && t.token >= 0 && t.head >= 0 && t.batch < lim && t.token < lim &&
           t.head < lim && (t.token > 0 || L <= 1);
}

}  // namespace

// a shorter segment's set-up costs as much as its chunks
LinForm lin_tc_form() { return LinForm{device_sm_count(), kC, 2, 2.f, 0.6f, 0.2f, 1.f}; }

bool lin_tc_supported(const LinParams& p) {
    for (int i = 0; i < p.njobs; ++i) {
        const LinJob& j = p.job[i];
        const int es = j.y_f32 ? 4 : 2;
        if (j.Dk > 128 || j.Dk % 8 != 0 || j.Dv % 8 != 0) return false;
        if (!mappable(j.q, p.L) || !mappable(j.k, p.L) || !mappable(j.v, p.L)) return false;
        if (((reinterpret_cast<uintptr_t>(j.y) | static_cast<uintptr_t>(j.y_batch * es) |
              static_cast<uintptr_t>(j.y_token * es) | static_cast<uintptr_t>(j.y_head * es)) & 15u) != 0)
            return false;
    }
    return true;
}

cudaError_t launch_lin_tc(const LinParams& p, bool cut, cudaStream_t s) {
    LinTcParams tp;
    LinMaps maps;
    tp.p = p;
    const char* skip = std::getenv("M3_TEST_LINATTN_SKIP_LOAD");
    tp.test_skip = skip ? std::atoi(skip) : 0;
    int used = 0;
    LinTensor seen[kMaps];
    int seen_dim[kMaps];
    for (int i = 0; i < p.njobs; ++i) {
        const LinJob& j = p.job[i];
        tp.parts[i] = j.final_state ? 3 : 2;
        const LinTensor* ts[3] = {&j.q, &j.k, &j.v};
        const int dims[3] = {j.Dk, j.Dk, j.Dv};
        for (int a = 0; a < 3; ++a) {
            const LinTensor& t = *ts[a];
            tp.head_ratio[i][a] = t.head == 0 ? p.H : t.ratio;
            tp.batched[i][a] = t.batch != 0 && !p.cu;
            int m = 0;
            while (m < used && !(seen[m].p == t.p && seen[m].batch == t.batch && seen[m].token == t.token &&
                                 seen[m].head == t.head && seen[m].ratio == t.ratio && seen_dim[m] == dims[a]))
                ++m;
            tp.map[i][a] = m;
            if (m < used) continue;
            seen[m] = t;
            seen_dim[m] = dims[a];
            ++used;
            // [batch][token][head][dim], box of 64 columns of 128 tokens of one head; a dimension of
            // one entry takes any legal stride
            const uint64_t nh = t.head == 0 ? 1 : p.H / t.ratio, nb = tp.batched[i][a] ? p.nseq : 1;
            const uint64_t d[4] = {static_cast<uint64_t>(dims[a]), nh, static_cast<uint64_t>(p.L), nb};
            const uint64_t st[3] = {nh > 1 ? static_cast<uint64_t>(t.head) * 2 : 16,
                                    p.L > 1 ? static_cast<uint64_t>(t.token) * 2 : 16,
                                    nb > 1 ? static_cast<uint64_t>(t.batch) * 2 : 16};
            const uint32_t box[4] = {64, 1, kC, 1};
            if (!encode_tmap(&maps.m[m], true, 4, t.p, d, st, box, true)) return cudaErrorInvalidValue;
        }
    }
    // the roles' register shares add up to a launch with exactly these
    static const int regs = [] {
        cudaFuncAttributes a{};
        return cudaFuncGetAttributes(&a, lin_tc_kernel<false>) == cudaSuccess ? a.numRegs : 0;
    }();
    if (regs != kRegsLaunch) return cudaErrorInvalidConfiguration;
    const unsigned grid = static_cast<unsigned>(p.blocks_x * p.H * p.rtiles);
    static std::atomic<uint64_t> done_state{0}, done{0};
    cudaError_t e = allow_smem(lin_tc_kernel<false>, kSmem, done);
    if (e != cudaSuccess) return e;
    if (!cut) {
        lin_tc_kernel<false><<<grid, kThreads, kSmem, s>>>(tp, maps);
        return cudaGetLastError();
    }
    if ((e = allow_smem(lin_tc_kernel<true>, kSmem, done_state)) != cudaSuccess) return e;
    lin_tc_kernel<true><<<grid, kThreads, kSmem, s>>>(tp, maps);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // may start while the end states' kernel runs; whoever reads them waits for it
    return launch_after_rms(lin_tc_kernel<false>, grid, kThreads, kSmem, s, tp, maps);
}

cudaError_t lin_tc_timeout(int* flag) {
    // the copy below waits for the default stream alone, not for streams that do not block on it
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(flag, g_lin_timeout, sizeof(int));
    if (e != cudaSuccess || *flag == 0) return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_lin_timeout, &zero, sizeof(int));
}

}  // namespace m3
