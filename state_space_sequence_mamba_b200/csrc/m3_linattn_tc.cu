// Linear attention's pass on the sm_100a tensor cores (bf16 tensors, Dk <= 128).
//
// One CTA per (sequence, segment, head, 64-column tile of v), two CTAs per SM; chunks of 128
// tokens. With q, k, v the pass's operands, H the state (Dk x 64, fp32) and pw[n] = a^n:
//     S  = q k^T                                   M128 N128 K=Dk   (A, B in shared memory)
//     O1 = q bf16(H)                               M128 N64  K=Dk
//     P  = bf16(p_scale a^{|i - j|} S), masked     TMEM -> registers -> TMEM
//     O2 = P v                                     M128 N64  K=128  (A = P in TMEM)
//     y  = o_scale a^{e(i)} O1 + O2
//     H  <- a^n H + k^T v',  v' = x_scale a^{w(j)} v
// The mask's powers of a multiply the scores in fp32, in two factors per 32-column block that are
// both at most 1 for a <= 1 (a^{t - last column} of the thread's row, a^{last - column} of the
// column), so nothing overflows however strong the decay; the diagonal block takes a^{t - j} from
// a table. q, k and v enter the products as stored. Roundings to bf16: P and H as operands of the
// output's products (the output is rounded to bf16 itself), and v' as the sum of bf16 parts: two
// (2^-17) for a state that only feeds bf16 operands, three (2^-25) for one that is returned,
// which keeps returned states as exact as fp32 sums are.
//
// What bounds it: with q, k, v, y per head (K 128, V 64) a chunk moves 96 KB against ~1800 tensor
// cycles, so HBM; with q and k shared by all heads 32 KB, so the tensor pipe and the chain of
// hand-offs S -> P -> O2 and H -> O1 -> v' -> H, which is why two CTAs share an SM. That leaves
// 104 KB a CTA: q, k (32 KB each), v, the state's bf16 operand (16 KB each), 8 KB to stage y.
// v' takes over q's place (and, its third part, the state operand's) once S and O1 are done.
//
// Two groups of four warps: 0-3 the rows (S -> P, y), 4-7 the state (H in registers, v'). One thread
// of each issues its group's products and loads right behind the group's named barrier (rows: S, O2
// and v's loads; state: O1, k^T v' and the loads of q and k); 8 warps leave 128 registers a thread.
// Hand-offs between the groups are mbarriers, one phase per chunk. All waits are bounded: one that
// gives up marks the library's timeout word, the groups' barriers carry the failure to every warp,
// and all leave their loops.
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
constexpr int kThreads = 256, kGroup = 128, kStateWarp0 = 4;
constexpr uint32_t kRowBar = 1, kStateBar = 2;      // named barriers of the two groups
constexpr uint32_t kSlab = 16384;
constexpr uint32_t S_Q = 0, S_K = 2 * kSlab, S_V = 4 * kSlab, S_H = 5 * kSlab, S_ST = 6 * kSlab;
constexpr uint32_t kStage = 2048;                    // y staging of one row warp
constexpr uint32_t kSmem = S_ST + 4 * kStage + 1024;
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t T_S = 0, T_P = 0, T_O2 = 64, T_O1 = 128, T_H = 192;
constexpr int kMaps = 9;

// One phase per chunk: loads landed (q and k; v), products done (S, O1, k^T v', O2), O1 read by the
// rows, v read by the state's warps; and two for draining.
enum { B_QK, B_V, B_S, B_O1, B_DH, B_O2, B_OFREE, B_VREAD, B_DRAIN, B_DRAIN2, kNumBars };
__host__ __device__ constexpr uint32_t bar_count(int b) { return b == B_VREAD ? 4 : 1; }

struct LinMaps {
    CUtensorMap m[kMaps];
};
struct LinTcParams {
    LinParams p;
    int map[3][3];              // [job][q, k, v]
    int head_ratio[3][3];       // head coordinate = h / ratio
    int batched[3][3];          // batch coordinate = sequence (0: one entry for all)
    int parts[3];               // bf16 parts of v'
};

// Waits for the phase of `bar` with the given parity, giving up when another role has or after
// kMaxPolls polls (the thread is suspended for up to a microsecond in each: about a second). No
// clock is read: the loop stays small, and it is in the code a dozen times.
constexpr int kMaxPolls = 1 << 21;
constexpr long long kDrainCycles = 200000000LL;
__device__ __forceinline__ bool lwait(uint64_t* bar, int parity, volatile int* abort_flag) {
    const uint32_t a = smem_u32(bar);
#pragma unroll 1
    for (int i = 0; i < kMaxPolls; ++i) {
        if (mbar_try_wait_sleep(a, parity & 1, 1000u)) return true;
        if (*abort_flag) return false;
    }
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
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void tma_prefetch_4d(const void* tmap, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];"
                 :: "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3) : "memory");
}

template <bool kStateOnly>
__global__ void __launch_bounds__(kThreads, 2)
lin_tc_kernel(const __grid_constant__ LinTcParams tp, const __grid_constant__ LinMaps maps) {
    const LinParams& p = tp.p;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t bars[kNumBars];
    __shared__ __align__(16) float pw[kC + 4];
    __shared__ __align__(16) float cf[32];
    __shared__ uint32_t tslot;
    __shared__ volatile int s_abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t per_x = static_cast<int64_t>(p.H) * p.rtiles;
    const int64_t x = blockIdx.x / per_x;
    const int rem = static_cast<int>(blockIdx.x - x * per_x);
    const int h = rem / p.rtiles, rt = rem % p.rtiles;
    int ji = 0, tile = rt;
    while (ji + 1 < p.njobs && tile >= p.job[ji].tiles) tile -= p.job[ji++].tiles;
    const LinJob& j = p.job[ji];
    const LinWhere w = lin_locate(p, x);
    if (!w.valid) return;
    const bool rev = j.reverse;
    const int order = rev ? w.nseg - 1 - w.seg : w.seg;
    const bool last_seg = order == w.nseg - 1;
    if (kStateOnly && last_seg) return;              // nobody reads the last one's
    const int seg0 = w.seg * p.seg_len;
    const int seg_end = seg0 + p.seg_len < w.len ? seg0 + p.seg_len : static_cast<int>(w.len);
    const int nchunks = (seg_end - seg0 + kC - 1) / kC;
    const bool want_final = !kStateOnly && j.final_state && last_seg;
    const int ksteps = (j.Dk + 15) / 16, slabs = j.Dk > 64 ? 2 : 1;
    const int parts = tp.parts[ji];
    const float g2 = p.log_decay[h] * 1.4426950408889634f;
    // token 0 and length of the cc-th chunk in processing order
    auto chunk_t0 = [&](int cc) { return seg0 + kC * (rev ? nchunks - 1 - cc : cc); };
    auto chunk_n = [&](int t0) { return seg_end - t0 < kC ? seg_end - t0 : kC; };

    // ---------------- set-up ----------------
    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) mbar_init(&bars[i], bar_count(i));
        fence_mbar_init();
        s_abort = 0;
    }
    if (warp == 0) tmem_alloc(&tslot, kTmemCols);
    for (int i = tid; i <= kC; i += kThreads) pw[i] = lin_pow(g2, static_cast<float>(i));
    if (tid < 32) cf[tid] = lin_pow(g2, static_cast<float>(rev ? tid : 31 - tid));
    if (slabs == 1) {   // the state's rows 64 .. 127: zeros (never loaded)
        for (int i = tid; i < static_cast<int>(kSlab / 16); i += kThreads)
            *reinterpret_cast<uint4*>(sm + S_K + kSlab + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = tslot;

    // operand descriptors and TMA coordinates (used by the two issuing threads)
    constexpr uint32_t hi = desc_hi_sw128(1024);
    const void* mv = &maps.m[tp.map[ji][2]];
    const int hv_ = h / tp.head_ratio[ji][2], bv = tp.batched[ji][2] ? static_cast<int>(w.batch) : 0;
    const int row0 = static_cast<int>(w.row0);
    auto load_v = [&](int cc) {
        mbar_arrive_expect_tx(&bars[B_V], kSlab);
        tma_load_4d(sm + S_V, mv, &bars[B_V], tile * kVT, hv_, row0 + chunk_t0(cc), bv);
    };

    if (warp < kStateWarp0) {
        // ================= rows: S -> P, then y =================
        if (!kStateOnly && nchunks > 0) {
            const bool lead = warp == 0 && lane == 0;
            const uint32_t lb = tmem + ((32u * warp) << 16);
            uint8_t* st = sm + S_ST + warp * kStage;
            const int t = 32 * warp + lane;
            const float ps = j.p_scale;
            int loads = 0, issued = 0;
            auto issue_s = [&](int cc) {
                constexpr uint32_t id_s = idesc_bf16(128, 128, false, false);
                const uint32_t loQ = desc_lo(smem_u32(sm + S_Q), 16), loK = desc_lo(smem_u32(sm + S_K), 16);
                if (!lwait(&bars[B_QK], cc, &s_abort)) return;
                fence_after_sync();
#pragma unroll 1
                for (int k = 0; k < ksteps; ++k)
                    mma_bf16(tmem + T_S, desc_pack(loQ + (kmajor_off(k, kSlab) >> 4), hi),
                             desc_pack(loK + (kmajor_off(k, kSlab) >> 4), hi), id_s, k > 0);
                mma_commit(smem_u32(&bars[B_S]));
                issued = 1;
            };
            if (lead) {
                load_v(0);
                loads = 1;
                issue_s(0);
            }
            __syncwarp();
#pragma unroll 1
            for (int cc = 0; cc < nchunks; ++cc) {
                const int t0 = chunk_t0(cc), n = chunk_n(t0);
                const int off = (rev && order == 0 && cc == 0) ? 1 : 0;
                bool fail = !lwait_warp(&bars[B_S], cc, &s_abort);
                if (!fail) {
                    fence_after_sync();
                    const int nblk = (n + 31) / 32;         // blocks of columns that hold tokens
#pragma unroll 1
                    for (int b = 0; b < nblk; ++b) {
                        uint32_t pk[16];
                        const int ahead = rev ? b - warp : warp - b;    // 0: the diagonal block
                        if (ahead < 0) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) pk[i] = 0u;
                        } else {
                            float v[32];
                            tmem_ld_32x32b_x32(lb + T_S + 32u * b, v);
                            tmem_wait_ld();
                            if (ahead > 0 && 32 * b + 32 <= n) {
                                const float f = ps * pw[rev ? 32 * b - t : t - 32 * b - 31];
#pragma unroll
                                for (int i = 0; i < 32; i += 4) {
                                    const float4 c4 = *reinterpret_cast<const float4*>(cf + i);
                                    pk[i / 2] = pack2(v[i] * f * c4.x, v[i + 1] * f * c4.y);
                                    pk[i / 2 + 1] = pack2(v[i + 2] * f * c4.z, v[i + 3] * f * c4.w);
                                }
                            } else {
                                // d = the distance of the block's column 0, lim = columns that hold tokens
                                const int sgn = rev ? 1 : -1, d = sgn * (32 * b - t), lim = n - 32 * b;
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    const int di = d + sgn * i;
                                    const bool on = di >= 0 && i < lim;
                                    v[i] = on ? v[i] * (ps * pw[on ? di : 0]) : 0.f;
                                }
#pragma unroll
                                for (int i = 0; i < 16; ++i) pk[i] = pack2(v[2 * i], v[2 * i + 1]);
                            }
                        }
                        // block b of P lies over S's block b / 2, which has been read
                        tmem_st_32x32b_x16(lb + T_P + 16u * b, pk);
                    }
                    tmem_wait_st();
                    if (n < kC) {
                        // rows of v behind the last token, as far as the product reads: another
                        // sequence's, or anything (their scores are zero, but zero times NaN is not)
                        fail = !lwait_warp(&bars[B_V], cc, &s_abort);
                        if (!fail && t >= n)
#pragma unroll 1
                            for (int i = 0; i < 8; ++i)
                                *reinterpret_cast<uint4*>(sm + S_V + t * 128 + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async();
                    }
                    fence_before_sync();
                }
                if (bar_sync_or(kRowBar, kGroup, fail)) break;
                if (lead && lwait(&bars[B_V], cc, &s_abort)) {
                    constexpr uint32_t id_o = idesc_bf16(128, 64, false, true);
                    const uint32_t loV = desc_lo(smem_u32(sm + S_V), kSlab);
                    fence_after_sync();
#pragma unroll 1
                    for (int k = 0; k < (n + 15) / 16; ++k)
                        mma_bf16_ts(tmem + T_O2, tmem + T_P + 8u * k, desc_pack(loV + (mnmajor_off(k) >> 4), hi),
                                    id_o, k > 0);
                    mma_commit(smem_u32(&bars[B_O2]));
                }
                __syncwarp();
                const int e = (rev ? n - t : t + 1) - off;
                const float f1 = j.o_scale * pw[e < 0 ? 0 : e];
                fail = !lwait_warp(&bars[B_O2], cc, &s_abort) || !lwait_warp(&bars[B_O1], cc, &s_abort);
                if (!fail) {
                    fence_after_sync();
                    const int64_t y0 = w.batch * j.y_batch + (w.row0 + t0 + 32 * warp) * j.y_token + h * j.y_head +
                                       tile * kVT;
                    const int rows = n - 32 * warp;         // of this warp that are tokens
                    const int cols = j.Dv - tile * kVT;
                    // 32 rows of 64 bytes at a time, 16-byte piece i of row r at piece i ^ (r >> 1 & 3)
                    uint8_t* put = st + lane * 64;
                    const int pr = lane >> 2, pc = lane & 3, sw = lane >> 1 & 3;
                    const uint8_t* get = st + pr * 64 + ((pc ^ (pr >> 1 & 3)) << 4);
                    const int per = j.y_f32 ? 4 : 8;        // columns of a piece
                    const int es = j.y_f32 ? 4 : 2;
                    uint8_t* out = static_cast<uint8_t*>(j.y) + (y0 + pr * j.y_token + pc * per) * es;
                    const int64_t step = 8 * j.y_token * es;
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        float a[16], b[16];
                        tmem_ld_32x32b_x16(lb + T_O1 + 16u * q, a);
                        tmem_ld_32x32b_x16(lb + T_O2 + 16u * q, b);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) b[i] = fmaf(f1, a[i], b[i]);
                        bool flush = true;
                        if (j.y_f32) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                *reinterpret_cast<float4*>(put + ((i ^ sw) << 4)) =
                                    make_float4(b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3]);
                        } else {
                            const int half = q & 1;
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                *reinterpret_cast<uint4*>(put + (((2 * half + i) ^ sw) << 4)) =
                                    make_uint4(pack2(b[8 * i], b[8 * i + 1]), pack2(b[8 * i + 2], b[8 * i + 3]),
                                               pack2(b[8 * i + 4], b[8 * i + 5]), pack2(b[8 * i + 6], b[8 * i + 7]));
                            flush = half == 1;
                        }
                        if (!flush) continue;
                        __syncwarp();
                        const int c = (j.y_f32 ? 16 * q : 16 * (q - 1)) + pc * per;
                        uint8_t* at = out + (c - pc * per) * es;
                        if (c < cols) {
#pragma unroll
                            for (int it = 0; it < 4; ++it)  // 8 rows further the pieces lie alike
                                if (8 * it + pr < rows)
                                    *reinterpret_cast<uint4*>(at + it * step) = *reinterpret_cast<const uint4*>(get + it * 512);
                        }
                        __syncwarp();
                    }
                    fence_before_sync();
                }
                if (bar_sync_or(kRowBar, kGroup, fail)) break;
                if (lead) {
                    mbar_arrive(&bars[B_OFREE]);
                    if (cc + 1 < nchunks && lwait(&bars[B_VREAD], cc, &s_abort)) {
                        load_v(cc + 1);
                        ++loads;
                    }
                }
                __syncwarp();
                if (lead && cc + 1 < nchunks) issue_s(cc + 1);
                __syncwarp();
            }
            if (lead) {     // every copy has landed, every product is done (at once, unless a wait gave up)
                if (loads > 0) (void)mbar_wait(&bars[B_V], (loads - 1) & 1, kDrainCycles);
                if (s_abort && issued) {
                    mma_commit(smem_u32(&bars[B_DRAIN]));
                    (void)mbar_wait(&bars[B_DRAIN], 0, kDrainCycles);
                }
            }
            __syncwarp();
        }
    } else {
        // ================= the state =================
        // Thread r holds row r in registers. The products of a chunk start from zero in TMEM and are
        // added here: the tensor core's accumulator drops the bits below its sum's last, and a state
        // kept there would shrink by them at every step (1e-6 over a long memory).
        const int sw = warp - kStateWarp0, r = 32 * sw + lane;
        const bool lead = sw == 0 && lane == 0;
        const uint32_t lb = tmem + ((32u * sw) << 16) + T_H;
        const void* mq = &maps.m[tp.map[ji][0]];
        const void* mk = &maps.m[tp.map[ji][1]];
        const int hq = h / tp.head_ratio[ji][0], hk = h / tp.head_ratio[ji][1];
        const int bq = tp.batched[ji][0] ? static_cast<int>(w.batch) : 0;
        const int bk = tp.batched[ji][1] ? static_cast<int>(w.batch) : 0;
        int loads = 0, issued = 0;
        auto load_qk = [&](int cc) {
            const int at = row0 + chunk_t0(cc);
            mbar_arrive_expect_tx(&bars[B_QK], (kStateOnly ? 1 : 2) * slabs * kSlab);
#pragma unroll 1
            for (int s = 0; s < slabs; ++s) {
                if (!kStateOnly) tma_load_4d(sm + S_Q + s * kSlab, mq, &bars[B_QK], 64 * s, hq, at, bq);
                tma_load_4d(sm + S_K + s * kSlab, mk, &bars[B_QK], 64 * s, hk, at, bk);
            }
            if (kStateOnly) load_v(cc);
            ++loads;
            if (cc + 1 < nchunks) {     // the next chunk on its way to L2
                const int tn = row0 + chunk_t0(cc + 1);
#pragma unroll 1
                for (int s = 0; s < slabs; ++s) {
                    if (!kStateOnly) tma_prefetch_4d(mq, 64 * s, hq, tn, bq);
                    tma_prefetch_4d(mk, 64 * s, hk, tn, bk);
                }
                tma_prefetch_4d(mv, tile * kVT, hv_, tn, bv);
            }
        };
        auto issue_o1 = [&](int cc) {
            constexpr uint32_t id_o = idesc_bf16(128, 64, false, true);
            const uint32_t loQ = desc_lo(smem_u32(sm + S_Q), 16), loH = desc_lo(smem_u32(sm + S_H), kSlab);
            if (!lwait(&bars[B_QK], cc, &s_abort) || (cc > 0 && !lwait(&bars[B_OFREE], cc - 1, &s_abort))) return;
            fence_after_sync();
#pragma unroll 1
            for (int k = 0; k < ksteps; ++k)
                mma_bf16(tmem + T_O1, desc_pack(loQ + (kmajor_off(k, kSlab) >> 4), hi),
                         desc_pack(loH + (mnmajor_off(k) >> 4), hi), id_o, k > 0);
            mma_commit(smem_u32(&bars[B_O1]));
            issued = 1;
        };
        if (lead && nchunks > 0) load_qk(0);
        __syncwarp();
        float hv[kVT];
#pragma unroll
        for (int i = 0; i < kVT; ++i) hv[i] = 0.f;
        // H <- decay H + the products in TMEM, and H as the next chunk's bf16 operand
        auto advance = [&](float decay, bool publish) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float d[16];
                tmem_ld_32x32b_x16(lb + 16u * q, d);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) hv[16 * q + i] = fmaf(decay, hv[16 * q + i], d[i]);
            }
            fence_before_sync();
            if (!publish) return;
#pragma unroll
            for (int i = 0; i < kVT / 8; ++i)
                *reinterpret_cast<uint4*>(sm + S_H + swz128(r, 8 * i)) =
                    make_uint4(pack2(hv[8 * i], hv[8 * i + 1]), pack2(hv[8 * i + 2], hv[8 * i + 3]),
                               pack2(hv[8 * i + 4], hv[8 * i + 5]), pack2(hv[8 * i + 6], hv[8 * i + 7]));
            fence_proxy_async();
        };
        const int cols = j.Dv - tile * kVT;
        if (!kStateOnly) {
            // the state before this segment (the given one and the segments before, decayed), four
            // columns at a time into the accumulator, from where the first chunk takes it as products
            const int64_t before = rev ? (order == 0 ? 0 : w.len - (seg0 + p.seg_len)) : seg0;
            const float fi = lin_pow(g2, static_cast<float>(rev && before > 0 ? before - 1 : before));
            const bool live = r < j.Dk, given = j.init && live && fi != 0.f;
            const float* src = given ? j.init + (static_cast<int64_t>(w.seq) * p.H + h) * j.Dk * j.Dv + r * j.init_k +
                                           tile * kVT * j.init_v
                                     : nullptr;
#pragma unroll 1
            for (int c = 0; c < kVT; c += 16) {
                float v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = 0.f;
                if (given && c < cols) {
                    if (j.init_v == 1) {        // Dv is a multiple of 8
#pragma unroll
                        for (int i = 0; i < 16; i += 4)
                            if (c + i < cols) {
                                const float4 v4 = *reinterpret_cast<const float4*>(src + c + i);
                                v[i] = fi * v4.x; v[i + 1] = fi * v4.y; v[i + 2] = fi * v4.z; v[i + 3] = fi * v4.w;
                            }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (c + i < cols) v[i] = fi * src[(c + i) * j.init_v];
                    }
                }
#pragma unroll 1
                for (int o = 0; o < order && live; ++o) {
                    const int sg = rev ? w.nseg - 1 - o : o;
                    const int64_t gap = rev ? static_cast<int64_t>(sg) * p.seg_len - (seg0 + p.seg_len)
                                            : seg0 - static_cast<int64_t>(sg + 1) * p.seg_len;
                    const float f = lin_pow(g2, static_cast<float>(gap));
                    if (f == 0.f) continue;
                    const float* e = p.seg + ((((x - w.seg + sg) * p.H + h) * p.rtiles + rt) * p.seg_rows + r) *
                                                 static_cast<int64_t>(kVT) + c;
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 v4 = *reinterpret_cast<const float4*>(e + i);
                        v[i] = fmaf(f, v4.x, v[i]); v[i + 1] = fmaf(f, v4.y, v[i + 1]);
                        v[i + 2] = fmaf(f, v4.z, v[i + 2]); v[i + 3] = fmaf(f, v4.w, v[i + 3]);
                    }
                }
                __syncwarp();
                uint32_t u[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(v[i]);
                tmem_st_32x32b_x16(lb + c, u);
            }
            tmem_wait_st();
        }
        // chunk -1 of the loop only takes up the state before the segment
        bool good = true;
#pragma unroll 1
        for (int cc = kStateOnly ? 0 : -1; cc < nchunks; ++cc) {
            const bool end = cc + 1 == nchunks;
            float decay = 0.f;
            bool fail = false;
            if (cc >= 0) {
                const int t0 = chunk_t0(cc), n = chunk_n(t0);
                decay = pw[n - ((rev && order == 0 && cc == 0) ? 1 : 0)];
                if (end && !kStateOnly && !want_final) {    // nobody wants the last chunk's state
                    good = false;
                    break;
                }
                fail = !lwait_warp(&bars[B_V], cc, &s_abort);
                // v' goes where q (and the state's operand) were read: S and O1 are done
                if (!kStateOnly)
                    fail = fail || !lwait_warp(&bars[B_S], cc, &s_abort) || !lwait_warp(&bars[B_O1], cc, &s_abort);
                else if (n < kC)
                    fail = fail || !lwait_warp(&bars[B_QK], cc, &s_abort);
                if (!fail) {
                    const float wt = r < n ? j.x_scale * pw[rev ? r : n - 1 - r] : 0.f;
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t at = swz128(r, 8 * i);
                        uint4 raw = *reinterpret_cast<const uint4*>(sm + S_V + at);
                        if (r >= n) {
                            // rows behind the last token, another sequence's or anything, are zeros: their
                            // weights are, but zero times NaN is not. k's too, as far as the product reads.
                            raw = make_uint4(0u, 0u, 0u, 0u);
                            *reinterpret_cast<uint4*>(sm + S_K + at) = raw;
                            *reinterpret_cast<uint4*>(sm + S_K + kSlab + at) = raw;
                        }
                        const uint32_t vw[4] = {raw.x, raw.y, raw.z, raw.w};
                        uint32_t p0[4], p1[4], p2[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float a = wt * lo_f(vw[u]), b = wt * hi_f(vw[u]);
                            p0[u] = pack2(a, b);
                            const float a1 = a - lo_f(p0[u]), b1 = b - hi_f(p0[u]);
                            p1[u] = pack2(a1, b1);
                            p2[u] = pack2(a1 - lo_f(p1[u]), b1 - hi_f(p1[u]));
                        }
                        *reinterpret_cast<uint4*>(sm + S_Q + at) = make_uint4(p0[0], p0[1], p0[2], p0[3]);
                        *reinterpret_cast<uint4*>(sm + S_Q + kSlab + at) = make_uint4(p1[0], p1[1], p1[2], p1[3]);
                        if (parts > 2) *reinterpret_cast<uint4*>(sm + S_H + at) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
                    }
                    fence_proxy_async();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_VREAD]);
                if (bar_sync_or(kStateBar, kGroup, fail)) { good = false; break; }
                if (lead && (!kStateOnly || lwait(&bars[B_QK], cc, &s_abort))) {
                    constexpr uint32_t id_h = idesc_bf16(128, 64, true, true);
                    const uint32_t loKt = desc_lo(smem_u32(sm + S_K), kSlab);
                    fence_after_sync();
#pragma unroll 1
                    for (int part = 0; part < parts; ++part) {
                        const uint32_t lo = desc_lo(smem_u32(sm + (part == 2 ? S_H : part * kSlab)), kSlab);
#pragma unroll 1
                        for (int k = 0; k < (n + 15) / 16; ++k)
                            mma_bf16(tmem + T_H, desc_pack(loKt + (mnmajor_off(k) >> 4), hi),
                                     desc_pack(lo + (mnmajor_off(k) >> 4), hi), id_h, part > 0 || k > 0);
                    }
                    mma_commit(smem_u32(&bars[B_DH]));
                    issued = 1;
                }
                __syncwarp();
                fail = !lwait_warp(&bars[B_DH], cc, &s_abort);
            }
            if (!fail) {
                if (lead && cc >= 0 && !end) load_qk(cc + 1);
                __syncwarp();
                fence_after_sync();
                advance(decay, !end && !kStateOnly);
            }
            if (bar_sync_or(kStateBar, kGroup, fail)) { good = false; break; }
            if (!kStateOnly && !end) {
                if (lead) issue_o1(cc + 1);
                __syncwarp();
            }
        }
        if (good && (kStateOnly || want_final)) {
            // through the accumulator once more, so that the copy out is a short loop
            // (an empty sequence's state passes through)
            const float ff = rev && w.len > 0 && !kStateOnly ? pw[1] : 1.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t u[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(ff * hv[16 * q + i]);
                tmem_st_32x32b_x16(lb + 16u * q, u);
            }
            tmem_wait_st();
            float* dst = kStateOnly ? p.seg + (((x * p.H + h) * p.rtiles + rt) * p.seg_rows + r) * static_cast<int64_t>(kVT)
                                    : j.final_state + ((static_cast<int64_t>(w.seq) * p.H + h) * j.Dk + r) * j.Dv +
                                          tile * kVT;
            const int lim = r >= j.Dk ? 0 : (kStateOnly ? kVT : cols);
#pragma unroll 1
            for (int c = 0; c < kVT; c += 16) {
                float v[16];
                tmem_ld_32x32b_x16(lb + c, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    if (c + i < lim)
                        *reinterpret_cast<float4*>(dst + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
        }
        if (lead) {
            if (loads > 0) {
                (void)mbar_wait(&bars[B_QK], (loads - 1) & 1, kDrainCycles);
                if (kStateOnly) (void)mbar_wait(&bars[B_V], (loads - 1) & 1, kDrainCycles);
            }
            if (s_abort && issued) {
                mma_commit(smem_u32(&bars[B_DRAIN2]));
                (void)mbar_wait(&bars[B_DRAIN2], 0, kDrainCycles);
            }
        }
        __syncwarp();
    }

    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (s_abort && tid == 0) atomicExch(&g_lin_timeout, 1);
    if (warp == 0) tmem_dealloc(tmem, kTmemCols);
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

int lin_tc_slots() { return 2 * device_sm_count(); }

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
    const unsigned grid = static_cast<unsigned>(p.blocks_x * p.H * p.rtiles);
    cudaError_t e;
    if (cut) {
        e = cudaFuncSetAttribute(lin_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        lin_tc_kernel<true><<<grid, kThreads, kSmem, s>>>(tp, maps);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    e = cudaFuncSetAttribute(lin_tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    lin_tc_kernel<false><<<grid, kThreads, kSmem, s>>>(tp, maps);
    return cudaGetLastError();
}

cudaError_t lin_tc_timeout(int* flag) {
    cudaError_t e = cudaMemcpyFromSymbol(flag, g_lin_timeout, sizeof(int));
    if (e != cudaSuccess || *flag == 0) return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_lin_timeout, &zero, sizeof(int));
}

}  // namespace m3
