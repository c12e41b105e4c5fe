// la_gated_bwd64.cuh — the whole backward of a 128-token block at D = 64 (bf16;
// formulas in la_gated_common.cuh, weights and rounding as la_gated_tc.cuh).
//
// Given the states S entering and R leaving the block, everything a block
// needs is local: with P = Q K^T and W = dO V^T (C x C, one product each for
// all three gradients), P~ = w P and W~ = w W,
//
//     dq = scale (W~ K + r dO S^T)         r_i = e^{G_i}
//     dk = scale W~^T Q + r' V R^T         r'_j = e^{G_C - G_j}
//     dv = scale P~^T dO + r' K R
//     M  = scale w P W                     (its row and column sums: dlog_gate)
//
// and q, k, v, dO are read and dq, dk, dv written once: 14 D bytes a token and
// head, and the two bf16 states (2 D bytes more at D = 64).  P~ and W~ are
// packed to bf16 in shared memory as row tiles [i][j]; the tensor core reads
// the same tile as rows (dq) and as columns (dk, dv), so each weight is formed
// and each product packed once.  Shared key/value heads: the block's group of
// query heads runs one after the other into the same dk, dv accumulators.
//
// Separate passes for dq, dk and dv read the four tensors again for each (and
// left dlog_gate's pieces to a fourth): 656 us at B8 H16 N8192.
#pragma once

#include "la_gated_tc.cuh"

namespace la {

struct GatedBwd64Params {
    CUtensorMap tm_q, tm_k, tm_v, tm_do, tm_s, tm_r, tm_dq, tm_dk, tm_dv;
    const __nv_bfloat16* lg;
    __nv_bfloat16* dlg;
    int64_t N, items;   // items: key/value heads * nblk
    int nblk, group;
    float scale;
};

struct alignas(16) GateTab64 {
    float loc[kGtC], fac[kGtC];
    double start[6];
};

struct GatedBwd64Cfg {
    static constexpr int C = 128, D = 64;
    static constexpr int TILE = C * D * 2;              // 16 KB
    static constexpr int OFF_KV = 0;                    // [2][K, V]
    static constexpr int OFF_QD = 4 * TILE;             // [2][Q, dO]
    static constexpr int OFF_PW = 8 * TILE;             // P~, W~: [128][128] bf16 each
    static constexpr int OFF_SR = OFF_PW + 2 * C * C * 2;  // S, R: [64][64] bf16 each
    static constexpr int OFF_TAB = OFF_SR + 2 * D * D * 2;
    static constexpr int OFF_RED = OFF_TAB + 2 * int(sizeof(GateTab64));
    static constexpr int RED = 12 * C;                  // floats: rows [4], cols [4], through [4]
    static constexpr int OFF_BAR = OFF_RED + RED * 4;
    static constexpr int NBAR = 24;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    // TMEM columns.  dq's two parts take P's columns once P~ is packed.
    static constexpr int T_P = 0, T_W = 128, T_DQS = 0, T_DQ = 64;
    static constexpr int T_DK = 256, T_DV = 320, T_DKR = 384, T_DVR = 448;
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

// Warps: 0 TMA loads, 1 MMA, 2 gate sums and dlog_gate, 3 TMA stores, 4-19
// weights, packing and epilogues: four groups of four warps, group h for the 32
// columns h of the C x C products and 16 columns of each gradient.  (Two groups
// with twice the columns each took 455 us instead of the time above: the chain
// pack - products - epilogue is latency, and more warps shorten its steps.)
constexpr int kGatedBwd64Threads = 640;
constexpr int kGatedBwd64Work = 512;

// STATE: S and R are given (both, zeros where there is none); without, the
// sequence is one block that nothing enters.
template <bool STATE>
__global__ void __launch_bounds__(kGatedBwd64Threads, 1)
gated_bwd64_kernel(const __grid_constant__ GatedBwd64Params prm) {
    using namespace sm100;
    using Cfg = GatedBwd64Cfg;
    constexpr int C = Cfg::C, D = Cfg::D, TILE = Cfg::TILE;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
    uint64_t* kv_full = bars;        // [2] TMA
    uint64_t* kv_free = bars + 2;    // [2] dk, dv stored, MMAs done       (store warp)
    uint64_t* qd_full = bars + 4;    // [2] TMA
    uint64_t* qd_free = bars + 6;    // [2] dq stored (store warp); MMAs done (commit)
    uint64_t* sr_full = bars + 8;    // TMA
    uint64_t* sr_free = bars + 9;    // products done (commit); <S, R> formed (warp 2)
    uint64_t* pw_raw = bars + 10;    // P, W complete                      (commit)
    uint64_t* pw_full = bars + 11;   // P~, W~ packed                      (512)
    uint64_t* a_full = bars + 12;    // dq and dk products complete        (commit)
    uint64_t* b_full = bars + 13;    // dv products complete               (commit)
    uint64_t* dq_read = bars + 14;   // dq accumulators read               (512)
    uint64_t* kv_read = bars + 15;   // dk, dv accumulators read           (512)
    uint64_t* dq_out = bars + 16;    // dq staged                          (512)
    uint64_t* kv_out = bars + 17;    // dk, dv staged; dlog_gate's sums written (512)
    uint64_t* red_free = bars + 18;  // ... read                           (32)
    uint64_t* tab_full = bars + 19;  // [2] gate tables written            (32)
    uint64_t* tab_free = bars + 21;  // [2] ... read                       (512)
    uint64_t* drain = bars + 23;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);
    GateTab64* tabs = reinterpret_cast<GateTab64*>(smem + Cfg::OFF_TAB);
    float* red = reinterpret_cast<float*>(smem + Cfg::OFF_RED);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(&kv_full[b], 1);
            mbar_init(&kv_free[b], 1);
            mbar_init(&qd_full[b], 1);
            mbar_init(&qd_free[b], 2);
            mbar_init(&tab_full[b], 32);
            mbar_init(&tab_free[b], kGatedBwd64Work);
        }
        mbar_init(sr_full, 1);
        mbar_init(sr_free, 2);
        mbar_init(pw_raw, 1);
        mbar_init(pw_full, kGatedBwd64Work);
        mbar_init(a_full, 1);
        mbar_init(b_full, 1);
        mbar_init(dq_read, kGatedBwd64Work);
        mbar_init(kv_read, kGatedBwd64Work);
        mbar_init(dq_out, kGatedBwd64Work);
        mbar_init(kv_out, kGatedBwd64Work);
        mbar_init(red_free, 32);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int G = prm.group;
    auto head_of = [&](int64_t it) { return int(unsigned(it) / unsigned(prm.nblk)); };
    auto blk_of = [&](int64_t it) { return int(unsigned(it) % unsigned(prm.nblk)); };

    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&prm.tm_q);
            tma_prefetch_desc(&prm.tm_k);
            tma_prefetch_desc(&prm.tm_v);
            tma_prefetch_desc(&prm.tm_do);
            uint32_t m = 0, u = 0;  // items, (item, query head) steps
            uint32_t srn = 0;  // state pairs issued
            bool ok = true;
            for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x, ++m) {
                const int head = head_of(it), blk = blk_of(it), row = blk * C;
                const int b = m & 1;
                if (m >= 2 && !(ok = mbar_wait(&kv_free[b], ((m >> 1) - 1) & 1, abort_flag))) break;
                uint8_t* kv = smem + Cfg::OFF_KV + b * 2 * TILE;
                mbar_arrive_expect_tx(&kv_full[b], 2 * TILE);
                tma_load_3d(kv, &prm.tm_k, &kv_full[b], 0, row, head);
                tma_load_3d(kv + TILE, &prm.tm_v, &kv_full[b], 0, row, head);
                for (int g = 0; g < G; ++g, ++u) {
                    const int s = u & 1;
                    if (u >= 2 && !(ok = mbar_wait(&qd_free[s], ((u >> 1) - 1) & 1, abort_flag)))
                        break;
                    uint8_t* qd = smem + Cfg::OFF_QD + s * 2 * TILE;
                    mbar_arrive_expect_tx(&qd_full[s], 2 * TILE);
                    tma_load_3d(qd, &prm.tm_q, &qd_full[s], 0, row, head * G + g);
                    tma_load_3d(qd + TILE, &prm.tm_do, &qd_full[s], 0, row, head * G + g);
                    if (g == 0 && STATE) {
                        if (srn > 0 && !(ok = mbar_wait(sr_free, (srn - 1) & 1, abort_flag))) break;
                        uint8_t* sr = smem + Cfg::OFF_SR;
                        mbar_arrive_expect_tx(sr_full, 2 * D * D * 2);
                        tma_load_3d(sr, &prm.tm_s, sr_full, 0, 0, head * prm.nblk + blk);
                        tma_load_3d(sr + D * D * 2, &prm.tm_r, sr_full, 0, 0, head * prm.nblk + blk);
                        ++srn;
                    }
                }
            }
            // copies in flight: at most the last two of each pair, and the states
            for (uint32_t i = m > 2 ? m - 2 : 0; i < m; ++i)
                mbar_wait_drain(&kv_full[i & 1], (i >> 1) & 1);
            for (uint32_t i = u > 2 ? u - 2 : 0; i < u; ++i)
                mbar_wait_drain(&qd_full[i & 1], (i >> 1) & 1);
            if (srn > 0) mbar_wait_drain(sr_full, (srn - 1) & 1);
        }
    } else if (warp == 1) {
        {
            const uint32_t one = elect_lane();
            constexpr uint32_t idP = idesc_bf16(C, C, 0, 0);
            constexpr uint32_t idQ = idesc_bf16(C, D, 0, 1);   // W~ K; K R
            constexpr uint32_t idT = idesc_bf16(C, D, 1, 1);   // W~^T Q; P~^T dO
            constexpr uint32_t idS = idesc_bf16(C, D, 0, 0);   // dO S^T; V R^T
            const uint32_t pt = sbase + Cfg::OFF_PW, wt = pt + C * C * 2;
            const uint32_t s_t = sbase + Cfg::OFF_SR, r_t = s_t + D * D * 2;
            uint32_t m = 0, u = 0;
            bool ok = true;
            for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x, ++m) {
                const uint32_t kt = sbase + Cfg::OFF_KV + (m & 1) * 2 * TILE, vt = kt + TILE;
                for (int g = 0; g < G; ++g, ++u) {
                    const int s = u & 1;
                    const uint32_t qt = sbase + Cfg::OFF_QD + s * 2 * TILE, ot = qt + TILE;
                    if (g == 0 && !(ok = warp_wait(&kv_full[m & 1], (m >> 1) & 1, abort_flag)))
                        break;
                    if (!(ok = warp_wait(&qd_full[s], (u >> 1) & 1, abort_flag))) break;
                    if (u > 0 && !(ok = warp_wait(dq_read, (u - 1) & 1, abort_flag))) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < D; k += 16)
                        umma_one(one, tmem + Cfg::T_P, desc_k_base(qt) + kstep_k(C, k),
                                  desc_k_base(kt) + kstep_k(C, k), idP, k > 0);
#pragma unroll
                    for (int k = 0; k < D; k += 16)
                        umma_one(one, tmem + Cfg::T_W, desc_k_base(ot) + kstep_k(C, k),
                                  desc_k_base(vt) + kstep_k(C, k), idP, k > 0);
                    commit_one(one, pw_raw);
                    if (g == 0) {
                        if (m > 0 && !(ok = warp_wait(kv_read, (m - 1) & 1, abort_flag))) break;
                        if (STATE && !(ok = warp_wait(sr_full, m & 1, abort_flag))) break;
                        tc_fence_after();
                        if (STATE) {
#pragma unroll
                            for (int k = 0; k < D; k += 16)
                                umma_one(one, tmem + Cfg::T_DKR, desc_k_base(vt) + kstep_k(C, k),
                                          desc_k_base(r_t) + kstep_k(D, k), idS, k > 0);
#pragma unroll
                            for (int k = 0; k < D; k += 16)
                                umma_one(one, tmem + Cfg::T_DVR, desc_k_base(kt) + kstep_k(C, k),
                                          desc_mn_base(r_t, D) + kstep_mn(k), idQ, k > 0);
                        }
                    }
                    if (!(ok = warp_wait(pw_full, u & 1, abort_flag))) break;
                    tc_fence_after();
                    if (STATE) {
#pragma unroll
                        for (int k = 0; k < D; k += 16)
                            umma_one(one, tmem + Cfg::T_DQS, desc_k_base(ot) + kstep_k(C, k),
                                      desc_k_base(s_t) + kstep_k(D, k), idS, k > 0);
                    }
                    if (g == G - 1 && STATE) commit_one(one, sr_free);
#pragma unroll
                    for (int k = 0; k < C; k += 16)
                        umma_one(one, tmem + Cfg::T_DQ, desc_k_base(wt) + kstep_k(C, k),
                                  desc_mn_base(kt, C) + kstep_mn(k), idQ, k > 0);
#pragma unroll
                    for (int k = 0; k < C; k += 16)
                        umma_one(one, tmem + Cfg::T_DK, desc_mn_base(wt, C) + kstep_mn(k),
                                  desc_mn_base(qt, C) + kstep_mn(k), idT, g > 0 || k > 0);
                    commit_one(one, a_full);
#pragma unroll
                    for (int k = 0; k < C; k += 16)
                        umma_one(one, tmem + Cfg::T_DV, desc_mn_base(pt, C) + kstep_mn(k),
                                  desc_mn_base(ot, C) + kstep_mn(k), idT, g > 0 || k > 0);
                    commit_one(one, b_full);
                    commit_one(one, &qd_free[s]);
                }
            }
            commit_one(one, drain);
            if (lane == 0) mbar_wait_drain(drain, 0);
        }
    } else if (warp == 2) {
        // gate tables one item ahead; <S, R>; the finished item's dlog_gate
        auto tables = [&](int64_t it, int buf) {
            GateTab64& tab = tabs[buf];
            gate_sums(prm.lg + int64_t(head_of(it)) * prm.N, int64_t(blk_of(it)) * C, prm.N, 4,
                      lane, tab.start, [&](int t, double run, double before, double end, double) {
                          tab.loc[t] = float(run - before);
                          tab.fac[t] = ex2_fast(float(end - run));
                      });
            __syncwarp();
            mbar_arrive(&tab_full[buf]);
        };
        uint32_t m = 0;
        if (int64_t(blockIdx.x) < prm.items) tables(blockIdx.x, 0);
        bool ok = true;
        for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x, ++m) {
            if (it + gridDim.x < prm.items) {
                const int nb = (m + 1) & 1;
                if (!(ok = __all_sync(0xffffffffu,
                                      m + 1 < 2 || mbar_wait(&tab_free[nb],
                                                             (((m + 1) >> 1) - 1) & 1, abort_flag))))
                    break;
                tables(it + gridDim.x, nb);
            }
            float x = 0.f;
            if (STATE) {
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(sr_full, m & 1, abort_flag)))) break;
                const uint4* s4 = reinterpret_cast<const uint4*>(smem + Cfg::OFF_SR);
                const uint4* r4 = s4 + D * D / 8;  // same swizzle: same places
#pragma unroll 4
                for (int i = lane; i < D * D / 8; i += 32) {
                    const uint4 a = s4[i], b = r4[i];
                    const uint32_t p[4] = {a.x, a.y, a.z, a.w}, q[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = unpack_bf16(p[j]), h = unpack_bf16(q[j]);
                        x = fmaf(f.x, h.x, x);
                        x = fmaf(f.y, h.y, x);
                    }
                }
                x = warp_sum(x) * ex2_fast(float(tabs[m & 1].start[4]));
                __syncwarp();
                if (lane == 0) mbar_arrive(sr_free);
            }
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(kv_out, m & 1, abort_flag)))) break;
            // tokens 4 l .. 4 l + 3 of lane l
            float d[4], t[4], ds = 0.f, ts = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = 4 * lane + j;
                d[j] = t[j] = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    d[j] += red[w * C + n] - red[(4 + w) * C + n];
                    t[j] += red[(8 + w) * C + n];
                }
                ds += d[j];
                ts += t[j];
            }
            __syncwarp();
            mbar_arrive(red_free);
            float behind = ds, before = ts;  // sums over the lanes behind / before
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float a = __shfl_down_sync(0xffffffffu, behind, o);
                const float b = __shfl_up_sync(0xffffffffu, before, o);
                if (lane + o < 32) behind += a;
                if (lane >= o) before += b;
            }
            behind = __shfl_down_sync(0xffffffffu, behind, 1);
            before = __shfl_up_sync(0xffffffffu, before, 1);
            if (lane == 31) behind = 0.f;
            if (lane == 0) before = 0.f;
            float g[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                g[j] = before + x;
                before += t[j];
            }
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                behind += d[j];
                g[j] += behind;
            }
            const int64_t n0 = int64_t(blk_of(it)) * C + 4 * lane;
            __nv_bfloat16* out = prm.dlg + int64_t(head_of(it)) * prm.N;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n0 + j < prm.N) out[n0 + j] = __float2bfloat16_rn(g[j]);
        }
    } else if (warp == 3) {
        if (lane == 0) {
            uint32_t m = 0, u = 0;
            bool ok = true;
            for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x, ++m) {
                const int head = head_of(it), row = blk_of(it) * C;
                for (int g = 0; g < G; ++g, ++u) {
                    if (!(ok = mbar_wait(dq_out, u & 1, abort_flag))) break;
                    tma_store_3d(&prm.tm_dq, smem + Cfg::OFF_QD + (u & 1) * 2 * TILE, 0, row,
                                 head * G + g);
                    bulk_commit();
                    bulk_wait_read0();
                    mbar_arrive(&qd_free[u & 1]);
                }
                if (!ok || !(ok = mbar_wait(kv_out, m & 1, abort_flag))) break;
                const uint8_t* kv = smem + Cfg::OFF_KV + (m & 1) * 2 * TILE;
                tma_store_3d(&prm.tm_dk, kv, 0, row, head);
                tma_store_3d(&prm.tm_dv, kv + TILE, 0, row, head);
                bulk_commit();
                bulk_wait_read0();
                mbar_arrive(&kv_free[m & 1]);
            }
            bulk_wait0();
        }
    } else {
        const int sp = warp & 3, grp = (warp - 4) >> 2;
        const uint32_t lane_base = uint32_t(32 * sp) << 16;
        const int irow = 32 * sp + lane;
        uint8_t* pt = smem + Cfg::OFF_PW;
        uint8_t* wt = pt + C * C * 2;
        uint32_t m = 0, u = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
        };
        // output columns of this thread: through a state (times rr) and inside the
        // block, into row irow of `tile`; returns the dot of what came through the
        // state with what the tile held there
        auto finish = [&](int t_in, int t_st, float rr, uint8_t* tile) {
            const int c0 = 16 * grp;
            float ov[16], sv[16], dot = 0.f;
            if (STATE) tmem_ld16(tmem + lane_base + t_st + c0, sv);
            tmem_load<16>(tmem + lane_base + t_in + c0, ov);
#pragma unroll
            for (int t = 0; t < 16; ++t) ov[t] *= prm.scale;
            if (STATE) {
#pragma unroll
                for (int t = 0; t < 16; t += 8) {
                    const uint4 x = *reinterpret_cast<const uint4*>(
                        tile + tile_chunk_off(C, irow, (c0 + t) / 8));
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = unpack_bf16(w[j]);
                        sv[t + 2 * j] *= rr;
                        sv[t + 2 * j + 1] *= rr;
                        dot = fmaf(f.x, sv[t + 2 * j], dot);
                        dot = fmaf(f.y, sv[t + 2 * j + 1], dot);
                        ov[t + 2 * j] += sv[t + 2 * j];
                        ov[t + 2 * j + 1] += sv[t + 2 * j + 1];
                    }
                }
            }
            store_row_bf16<16>(tile, C, irow, c0, ov);
            return dot;
        };
        for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x, ++m) {
            const GateTab64& tab = tabs[m & 1];
            if (!(ok = wait(&tab_full[m & 1], (m >> 1) & 1))) break;
            const float gi = tab.loc[irow];
            const double gI = tab.start[sp];
            const float r_q = prm.scale * ex2_fast(gi + float(gI));
            const float r_k = ex2_fast(float(tab.start[4] - gI) - gi);
            float rsum = 0.f, csum = 0.f, through = 0.f;
            uint8_t* kv = smem + Cfg::OFF_KV + (m & 1) * 2 * TILE;
            for (int g = 0; g < G; ++g, ++u) {
                if (!(ok = wait(pw_raw, u & 1))) break;
                tc_fence_after();
                // The last step's dv products have read P~, and its dk products W~:
                // this thread waited for both before it left that step.
                uint32_t mp[16];  // M, in bf16 pairs (see below)
                const int J = grp;
                const float r = J < sp ? ex2_fast(gi + float(gI - tab.start[J + 1])) : 0.f;
#pragma unroll
                for (int s = 0; s < 2; ++s) {  // 16 columns at a time
                    const int c0 = 32 * J + 16 * s;
                    float pv[16], wv[16];
                    float ms[16];
                    if (J <= sp) {
                        tmem_ld16(tmem + lane_base + Cfg::T_P + c0, pv);
                        tmem_load<16>(tmem + lane_base + Cfg::T_W + c0, wv);
                        if (J == sp) {
#pragma unroll
                            for (int t = 0; t < 16; ++t) {
                                const int tt = 16 * s + t;
                                const float e = ex2_fast(gi - tab.loc[c0 + t]);
                                const float a = tt <= lane ? pv[t] * e : 0.f;
                                ms[t] = tt < lane ? a * wv[t] : 0.f;  // the diagonal passes no gate
                                pv[t] = a;
                                wv[t] = tt <= lane ? wv[t] * e : 0.f;
                            }
                        } else {
#pragma unroll
                            for (int t = 0; t < 16; t += 4) {
                                const float4 f = *reinterpret_cast<const float4*>(tab.fac + c0 + t);
                                const float fj[4] = {r * f.x, r * f.y, r * f.z, r * f.w};
#pragma unroll
                                for (int w = 0; w < 4; ++w) {
                                    pv[t + w] *= fj[w];
                                    ms[t + w] = pv[t + w] * wv[t + w];
                                    wv[t + w] *= fj[w];
                                }
                            }
                        }
                    } else {
#pragma unroll
                        for (int t = 0; t < 16; ++t) pv[t] = wv[t] = ms[t] = 0.f;
                    }
#pragma unroll
                    for (int t = 0; t < 8; ++t) mp[8 * s + t] = pack_bf16(ms[2 * t], ms[2 * t + 1]);
                    store_row_bf16<16>(pt, C, irow, c0, pv);
                    store_row_bf16<16>(wt, C, irow, c0, wv);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(pw_full);
                if (J <= sp) {  // M's sums while the products run
                    // rows and columns add the same rounded values, so what cancels
                    // between them still does
                    float mm[32], rs = 0.f;
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        const float2 f = unpack_bf16(mp[t]);
                        mm[2 * t] = f.x;
                        mm[2 * t + 1] = f.y;
                        rs += f.x + f.y;
                    }
                    rsum = fmaf(prm.scale, rs, rsum);
                    // lane l ends with the sum of column l over the warp's rows
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
                        for (int t = 0; t < off; ++t) {
                            const bool up = (lane & off) != 0;
                            const float give = up ? mm[t] : mm[t + off];
                            const float keep = up ? mm[t + off] : mm[t];
                            mm[t] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                        }
                    csum = fmaf(prm.scale, mm[0], csum);
                }
                // dq, then (last head of the group) dk: their products are done
                uint8_t* qt = smem + Cfg::OFF_QD + (u & 1) * 2 * TILE;
                if (!(ok = wait(&qd_full[u & 1], (u >> 1) & 1) && wait(a_full, u & 1) &&
                           (u == 0 || wait(&qd_free[(u - 1) & 1], ((u - 1) >> 1) & 1))))
                    break;
                tc_fence_after();
                rsum += finish(Cfg::T_DQ, Cfg::T_DQS, r_q, qt);
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(dq_read);
                mbar_arrive(dq_out);
                if (g == G - 1) {
                    if (!(ok = wait(&kv_full[m & 1], (m >> 1) & 1))) break;
                    through = finish(Cfg::T_DK, Cfg::T_DKR, r_k, kv);
                }
                if (!(ok = wait(b_full, u & 1))) break;
                tc_fence_after();
                if (g == G - 1) (void)finish(Cfg::T_DV, Cfg::T_DVR, r_k, kv + TILE);
            }
            if (!ok) break;
            if (!(ok = m == 0 || (wait(red_free, (m - 1) & 1) &&
                                  wait(&kv_free[(m - 1) & 1], ((m - 1) >> 1) & 1))))
                break;
            red[grp * C + irow] = rsum;
            red[(4 + sp) * C + 32 * grp + lane] = csum;
            red[(8 + grp) * C + irow] = through;
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(kv_read);
            mbar_arrive(kv_out);
            mbar_arrive(&tab_free[m & 1]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace la
