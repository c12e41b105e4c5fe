// la_gated_bwd.cuh — the whole backward of a 128-token block of gated linear
// attention (bf16, D = 64 or 128; formulas in la_gated_common.cuh, weights and
// rounding as la_gated_tc.cuh).
//
// Given the states S entering and R leaving the block, everything a block
// needs is local: with P = Q K^T and W = dO V^T (C x C, one product each for
// all three gradients), P~ = scale w P and W~ = scale w W,
//
//     dq = scale r dO S^T + W~ K           r_i = e^{G_i}
//     dk = r' V R^T + W~^T Q               r'_j = e^{G_C - G_j}
//     dv = r' K R + P~^T dO
//     M  = scale w P W                     (its row and column sums: dlog_gate)
//
// and q, k, v, dO are read and dq, dk, dv written once: 14 D bytes a token and
// head, and the two bf16 states (4 D^2 / 128 bytes).  P~ and W~ are packed to
// bf16 in shared memory as row tiles [i][j]; the tensor core reads the same tile
// as rows (dq) and as columns (dk, dv), so each weight is formed and each product
// packed once.  What comes through a state is formed first, in the gradient's own
// accumulator; its rows are multiplied by their gates there (TMEM -> registers ->
// TMEM), and the products inside the block add to it.  Shared key/value heads:
// the group's query heads run one after the other into the same dk and dv.
//
// D = 64: two blocks' tiles in shared memory; TMEM holds P, W (128 columns each)
// and the three gradients (64 each), so the next block's P and W are formed while
// this one's gradients are read.  D = 128: one block's tiles (128 KB), the states
// stand where P~ and W~ go later (64 KB), and dq takes P's columns once P is in
// registers; the loads of a block wait for the stores of the one before.
//
// Separate passes for dq, dk and dv read the four tensors again for each and left
// dlog_gate's pieces to a fourth kernel: 656 us at B8 H16 N8192 D64 and 322 us at
// B4 H16 N4096 D128, where this kernel takes 299 and 143 us.  It moves 1.07 GB and
// 0.60 GB (3.6 and 4.2 TB/s, 0.55 and 0.64 of a copy's bandwidth).  D = 64: the
// warps of rows 96 to 127, which have most of the triangle, issue almost without
// pause, and pack, product and epilogue of a block follow each other.  D = 128: one
// block's tiles at a time (the next block's are brought to L2 ahead).
#pragma once

#include "la_gated_tc.cuh"

namespace la {

struct GatedBwdParams {
    CUtensorMap tm_q, tm_k, tm_v, tm_do, tm_s, tm_r, tm_dq, tm_dk, tm_dv;
    const __nv_bfloat16* lg;
    __nv_bfloat16* dlg;
    int64_t N, items;   // items: key/value heads * nblk
    const float* dots;  // [kvh][nblk][ndots]: parts of <S, R>
    int nblk, group, ndots;
    float scale;
};

struct alignas(16) GateTabBlock {
    float loc[kGtC], fac[kGtC];
    double start[6];
};

template <int HEAD>
struct GatedBwdCfg {
    static constexpr int C = 128, D = HEAD;
    static constexpr int NB = D == 64 ? 2 : 1;           // blocks of tiles
    static constexpr int TILE = C * D * 2;
    static constexpr int PT = C * C * 2;                 // P~, W~
    static constexpr int OFF_KV = 0;                     // [NB][K, V]
    static constexpr int OFF_QD = 2 * NB * TILE;         // [NB][Q, dO]
    static constexpr int OFF_PW = 4 * NB * TILE;         // P~, W~
    static constexpr int ST = D * D * 2;                 // S, R
    static constexpr int OFF_SR = D == 64 ? OFF_PW + 2 * PT : OFF_PW;
    static constexpr int OFF_TAB = D == 64 ? OFF_SR + 2 * ST : OFF_PW + 2 * PT;
    static constexpr int OFF_RED = OFF_TAB + 2 * int(sizeof(GateTabBlock));
    static constexpr int RED = 12 * C;                   // rows [4], cols [4], through [4]
    static constexpr int OFF_BAR = OFF_RED + RED * 4;
    static constexpr int NBAR = 26;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static constexpr int T_P = 0, T_W = 128;
    static constexpr int T_DQ = D == 64 ? 256 : T_P, T_DK = D == 64 ? 320 : 256, T_DV = 384;
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

// Warps: 0 TMA loads, 1 MMA, 2 gate sums and dlog_gate, 3 TMA stores, 4-19
// weights, packing and epilogues: four groups of four warps, group h for the
// columns 32 h .. 32 h + 31 of the C x C products and a quarter of each gradient's.
constexpr int kGatedBwdThreads = 640;
constexpr int kGatedBwdWork = 512;

// STATE: S and R are given (both, zeros where there is none); without, the
// sequence is one block that nothing enters.
template <int HEAD, bool STATE>
__global__ void __launch_bounds__(kGatedBwdThreads, 1)
gated_bwd_kernel(const __grid_constant__ GatedBwdParams prm) {
    using namespace sm100;
    using Cfg = GatedBwdCfg<HEAD>;
    constexpr int C = Cfg::C, D = Cfg::D, TILE = Cfg::TILE, NB = Cfg::NB;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
    uint64_t* kv_full = bars;        // [2] TMA
    uint64_t* kv_free = bars + 2;    // [2] dk, dv stored                  (store warp)
    uint64_t* qd_full = bars + 4;    // [2] TMA
    uint64_t* qd_free = bars + 6;    // [2] dq stored (store warp); MMAs done (commit)
    uint64_t* sr_full = bars + 8;    // TMA
    uint64_t* sr_free = bars + 9;    // S, R (D = 128: and P~, W~) read    (commit)
    uint64_t* pw_raw = bars + 10;    // P, W complete                      (commit)
    uint64_t* p_read = bars + 11;    // P, W in registers                  (16 warps)
    uint64_t* s_full = bars + 12;    // products with S and R complete     (commit)
    uint64_t* pw_full = bars + 13;   // P~, W~ packed, state parts scaled  (16 warps)
    uint64_t* a_full = bars + 14;    // dq, dk complete                    (commit)
    uint64_t* b_full = bars + 15;    // dv complete                        (commit)
    uint64_t* dq_read = bars + 16;   // dq accumulator read                (16 warps)
    uint64_t* kv_read = bars + 17;   // dk, dv accumulators read           (16 warps)
    uint64_t* dq_out = bars + 18;    // dq staged                          (16 warps)
    uint64_t* kv_out = bars + 19;    // dk, dv staged; dlog_gate's sums written (16 warps)
    uint64_t* red_free = bars + 20;  // ... read                           (1)
    uint64_t* tab_full = bars + 21;  // [2] gate tables written            (1)
    uint64_t* tab_free = bars + 23;  // [2] ... read                       (16 warps)
    uint64_t* drain = bars + 25;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);
    GateTabBlock* tabs = reinterpret_cast<GateTabBlock*>(smem + Cfg::OFF_TAB);
    float* red = reinterpret_cast<float*>(smem + Cfg::OFF_RED);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(&kv_full[b], 1);
            mbar_init(&kv_free[b], 1);
            mbar_init(&qd_full[b], 1);
            mbar_init(&qd_free[b], 2);
        }
        mbar_init(sr_full, 1);
        mbar_init(sr_free, 1);
        mbar_init(pw_raw, 1);
        mbar_init(p_read, kGatedBwdWork / 32);
        mbar_init(s_full, 1);
        mbar_init(pw_full, kGatedBwdWork / 32);
        mbar_init(a_full, 1);
        mbar_init(b_full, 1);
        mbar_init(dq_read, kGatedBwdWork / 32);
        mbar_init(kv_read, kGatedBwdWork / 32);
        mbar_init(dq_out, kGatedBwdWork / 32);
        mbar_init(kv_out, kGatedBwdWork / 32);
        mbar_init(red_free, 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tab_full[b], 1);
            mbar_init(&tab_free[b], kGatedBwdWork / 32);
        }
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
            auto load = [&](int off, const CUtensorMap* map, uint64_t* bar, int rows, int row,
                            int head) {
                for (int a = 0; a < D / 64; ++a)
                    tma_load_3d(smem + off + a * rows * 128, map, bar, 64 * a, row, head);
            };
            // D = 128: the tiles of the next item, brought to L2 while this one's space
            // is still taken
            auto ahead = [&](const CUtensorMap* map, int row, int head) {
                for (int a = 0; a < D / 64; ++a) tma_prefetch_3d(map, 64 * a, row, head);
            };
            uint32_t m = 0, u = 0;              // items, (item, query head) steps
            uint32_t kvn = 0, qdn = 0, srn = 0;  // issued
            bool ok = true;
            for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x, ++m) {
                const int head = head_of(it), blk = blk_of(it), row = blk * C;
                for (int g = 0; g < G; ++g, ++u) {
                    const int s = u % NB, b = m % NB;
                    if (u >= NB && !(ok = mbar_wait(&qd_free[s], (u / NB - 1) & 1, abort_flag))) break;
                    mbar_arrive_expect_tx(&qd_full[s], 2 * TILE);
                    load(Cfg::OFF_QD + 2 * s * TILE, &prm.tm_q, &qd_full[s], C, row, head * G + g);
                    load(Cfg::OFF_QD + (2 * s + 1) * TILE, &prm.tm_do, &qd_full[s], C, row,
                         head * G + g);
                    ++qdn;
                    if (g == 0) {
                        if (m >= NB && !(ok = mbar_wait(&kv_free[b], (m / NB - 1) & 1, abort_flag)))
                            break;
                        mbar_arrive_expect_tx(&kv_full[b], 2 * TILE);
                        load(Cfg::OFF_KV + 2 * b * TILE, &prm.tm_k, &kv_full[b], C, row, head);
                        load(Cfg::OFF_KV + (2 * b + 1) * TILE, &prm.tm_v, &kv_full[b], C, row, head);
                        ++kvn;
                    }
                    if (STATE) {  // S for every query head, R for the first
                        if (u > 0 && !(ok = mbar_wait(sr_free, (u - 1) & 1, abort_flag))) break;
                        mbar_arrive_expect_tx(sr_full, (g == 0 ? 2 : 1) * Cfg::ST);
                        load(Cfg::OFF_SR, &prm.tm_s, sr_full, D, 0, head * prm.nblk + blk);
                        if (g == 0)
                            load(Cfg::OFF_SR + Cfg::ST, &prm.tm_r, sr_full, D, 0,
                                 head * prm.nblk + blk);
                        ++srn;
                    }
                    if (D == 128) {
                        const bool same = g + 1 < G;
                        const int64_t nx = same ? it : it + gridDim.x;
                        if (nx < prm.items) {
                            const int h2 = head_of(nx), b2 = blk_of(nx), qh = h2 * G + (same ? g + 1 : 0);
                            ahead(&prm.tm_q, b2 * C, qh);
                            ahead(&prm.tm_do, b2 * C, qh);
                            if (!same) {
                                ahead(&prm.tm_k, b2 * C, h2);
                                ahead(&prm.tm_v, b2 * C, h2);
                                if (STATE) {
                                    ahead(&prm.tm_s, 0, h2 * prm.nblk + b2);
                                    ahead(&prm.tm_r, 0, h2 * prm.nblk + b2);
                                }
                            }
                        }
                    }
                }
            }
            for (uint32_t i = qdn > NB ? qdn - NB : 0; i < qdn; ++i)
                mbar_wait_drain(&qd_full[i % NB], (i / NB) & 1);
            for (uint32_t i = kvn > NB ? kvn - NB : 0; i < kvn; ++i)
                mbar_wait_drain(&kv_full[i % NB], (i / NB) & 1);
            if (srn) mbar_wait_drain(sr_full, (srn - 1) & 1);
        }
    } else if (warp == 1) {
        const uint32_t one = elect_lane();
        constexpr uint32_t idP = idesc_bf16(C, C, 0, 0);   // P, W
        constexpr uint32_t idK = idesc_bf16(C, D, 0, 0);   // dO S^T; V R^T
        constexpr uint32_t idN = idesc_bf16(C, D, 0, 1);   // W~ K; K R
        constexpr uint32_t idT = idesc_bf16(C, D, 1, 1);   // W~^T Q; P~^T dO
        const uint32_t st = sbase + Cfg::OFF_SR, rt = st + Cfg::ST;
        const uint32_t pt = sbase + Cfg::OFF_PW, wt = pt + Cfg::PT;
        uint32_t m = 0, u = 0;
        bool ok = true;
        for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x, ++m) {
            const uint32_t kt = sbase + Cfg::OFF_KV + (m % NB) * 2 * TILE, vt = kt + TILE;
            for (int g = 0; g < G; ++g, ++u) {
                const uint32_t qt = sbase + Cfg::OFF_QD + (u % NB) * 2 * TILE, ot = qt + TILE;
                // P's and W's columns: read by the step before (D = 128: and its dq)
                if (!(ok = (g > 0 || warp_wait(&kv_full[m % NB], (m / NB) & 1, abort_flag)) &&
                           warp_wait(&qd_full[u % NB], (u / NB) & 1, abort_flag) &&
                           (u == 0 ||
                            warp_wait(D == 64 ? p_read : dq_read, (u - 1) & 1, abort_flag))))
                    break;
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
                auto dq_state = [&]() {
#pragma unroll
                    for (int k = 0; k < D; k += 16)
                        umma_one(one, tmem + Cfg::T_DQ, desc_k_base(ot) + kstep_k(C, k),
                                 desc_k_base(st) + kstep_k(D, k), idK, k > 0);
                };
                if (D == 64 && u > 0 && !(ok = warp_wait(dq_read, (u - 1) & 1, abort_flag))) break;
                if (STATE) {
                    if (!(ok = warp_wait(sr_full, u & 1, abort_flag))) break;
                    tc_fence_after();
                    if (D == 64) dq_state();
                }
                if (g == 0 && m > 0 && !(ok = warp_wait(kv_read, (m - 1) & 1, abort_flag))) break;
                if (STATE) {
                    tc_fence_after();
                    if (g == 0) {
#pragma unroll
                        for (int k = 0; k < D; k += 16)
                            umma_one(one, tmem + Cfg::T_DK, desc_k_base(vt) + kstep_k(C, k),
                                     desc_k_base(rt) + kstep_k(D, k), idK, k > 0);
#pragma unroll
                        for (int k = 0; k < D; k += 16)
                            umma_one(one, tmem + Cfg::T_DV, desc_k_base(kt) + kstep_k(C, k),
                                     desc_mn_base(rt, D) + kstep_mn(k), idN, k > 0);
                    }
                    if (D == 64) commit_one(one, s_full);
                    if (!(ok = warp_wait(p_read, u & 1, abort_flag))) break;
                    tc_fence_after();
                    if (D == 64) {
                        commit_one(one, sr_free);
                    } else {
                        dq_state();
                        commit_one(one, s_full);
                    }
                }
                if (!(ok = warp_wait(pw_full, u & 1, abort_flag))) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < C; k += 16)
                    umma_one(one, tmem + Cfg::T_DQ, desc_k_base(wt) + kstep_k(C, k),
                             desc_mn_base(kt, C) + kstep_mn(k), idN, STATE || k > 0);
#pragma unroll
                for (int k = 0; k < C; k += 16)
                    umma_one(one, tmem + Cfg::T_DK, desc_mn_base(wt, C) + kstep_mn(k),
                             desc_mn_base(qt, C) + kstep_mn(k), idT, STATE || g > 0 || k > 0);
                commit_one(one, a_full);
#pragma unroll
                for (int k = 0; k < C; k += 16)
                    umma_one(one, tmem + Cfg::T_DV, desc_mn_base(pt, C) + kstep_mn(k),
                             desc_mn_base(ot, C) + kstep_mn(k), idT, STATE || g > 0 || k > 0);
                commit_one(one, b_full);
                commit_one(one, &qd_free[u % NB]);
                if (STATE && D == 128) commit_one(one, sr_free);
            }
        }
        commit_one(one, drain);
        if (lane == 0) mbar_wait_drain(drain, 0);
    } else if (warp == 2) {
        // gate tables one item ahead; the finished item's dlog_gate
        auto tables = [&](int64_t it, int buf) {
            GateTabBlock& tab = tabs[buf];
            gate_sums(prm.lg + int64_t(head_of(it)) * prm.N, int64_t(blk_of(it)) * C, prm.N, 4,
                      lane, tab.start, [&](int t, double run, double before, double end, double) {
                          tab.loc[t] = float(run - before);
                          tab.fac[t] = ex2_fast(float(end - run));
                      });
            warp_arrive(&tab_full[buf]);
        };
        uint32_t m = 0;
        if (int64_t(blockIdx.x) < prm.items) tables(blockIdx.x, 0);
        bool ok = true;
        for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x, ++m) {
            if (it + gridDim.x < prm.items) {
                const int nb = (m + 1) & 1;
                if (!(ok = m + 1 < 2 ||
                           warp_wait(&tab_free[nb], (((m + 1) >> 1) - 1) & 1, abort_flag)))
                    break;
                tables(it + gridDim.x, nb);
            }
            float x = 0.f;  // e^{G_C} <S, R>
            if (STATE) {
                const float* dots = prm.dots + it * prm.ndots;
                for (int i = lane; i < prm.ndots; i += 32) x += dots[i];
                x = warp_sum(x) * ex2_fast(float(tabs[m & 1].start[4]));
            }
            if (!(ok = warp_wait(kv_out, m & 1, abort_flag))) break;
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
            warp_arrive(red_free);
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
            float gr[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                gr[j] = before + x;
                before += t[j];
            }
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                behind += d[j];
                gr[j] += behind;
            }
            const int64_t n0 = int64_t(blk_of(it)) * C + 4 * lane;
            __nv_bfloat16* out = prm.dlg + int64_t(head_of(it)) * prm.N;
            // the gates once more, as differences of their sums in the table
            const float4 l4 = *reinterpret_cast<const float4*>(&tabs[m & 1].loc[4 * lane]);
            const float up = __shfl_up_sync(0xffffffffu, l4.w, 1);
            const float l[5] = {lane % 8 ? up : 0.f, l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n0 + j < prm.N)
                    out[n0 + j] =
                        __float2bfloat16_rn(gate_is_zero(l[j + 1] - l[j]) ? 0.f : gr[j]);
        }
    } else if (warp == 3) {
        if (lane == 0) {
            auto store = [&](const CUtensorMap* map, int off, int row, int head) {
                for (int a = 0; a < D / 64; ++a)
                    tma_store_3d(map, smem + off + a * C * 128, 64 * a, row, head);
            };
            uint32_t m = 0, u = 0;
            bool ok = true;
            for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x, ++m) {
                const int head = head_of(it), row = blk_of(it) * C;
                for (int g = 0; g < G; ++g, ++u) {
                    if (!(ok = mbar_wait(dq_out, u & 1, abort_flag))) break;
                    store(&prm.tm_dq, Cfg::OFF_QD + 2 * (u % NB) * TILE, row, head * G + g);
                    bulk_commit();
                    bulk_wait_read0();
                    mbar_arrive(&qd_free[u % NB]);
                }
                if (!ok || !(ok = mbar_wait(kv_out, m & 1, abort_flag))) break;
                store(&prm.tm_dk, Cfg::OFF_KV + 2 * (m % NB) * TILE, row, head);
                store(&prm.tm_dv, Cfg::OFF_KV + (2 * (m % NB) + 1) * TILE, row, head);
                bulk_commit();
                bulk_wait_read0();
                mbar_arrive(&kv_free[m % NB]);
            }
            bulk_wait0();
        }
    } else {
        const int sp = warp & 3, grp = (warp - 4) >> 2;
        const uint32_t lane_base = uint32_t(32 * sp) << 16;
        const int irow = 32 * sp + lane;
        const int c0 = 32 * grp;        // columns of the C x C products
        constexpr int GC = D / 4;       // columns of the gradients
        const int d0 = GC * grp;
        uint8_t* pt = smem + Cfg::OFF_PW;
        uint8_t* wt = pt + Cfg::PT;
        uint32_t m = 0, u = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity, abort_flag); };
        // this thread's columns of an accumulator times rr, in place; returns their
        // dot with the same columns of row irow of `tile` (null: none)
        auto scale_part = [&](int t_acc, float rr, const uint8_t* tile) {
            float2 dot = make_float2(0.f, 0.f);
#pragma unroll
            for (int s = 0; s < GC / 16; ++s) {
                float sv[16];
                const uint32_t at = tmem + lane_base + t_acc + d0 + 16 * s;
                tmem_load<16>(at, sv);
#pragma unroll
                for (int t = 0; t < 16; t += 2) {
                    const float2 x = mul2(make_float2(sv[t], sv[t + 1]), make_float2(rr, rr));
                    sv[t] = x.x, sv[t + 1] = x.y;
                }
                tmem_st16(at, sv);
                if (tile) {
#pragma unroll
                    for (int t = 0; t < 16; t += 8) {
                        const uint4 x = *reinterpret_cast<const uint4*>(
                            tile + tile_chunk_off(C, irow, (d0 + 16 * s + t) / 8));
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            dot = fma2(unpack_bf16(w[j]),
                                       make_float2(sv[t + 2 * j], sv[t + 2 * j + 1]), dot);
                        }
                    }
                }
            }
            return dot.x + dot.y;
        };
        // One step of the sums of columns over a warp's rows: of 2 n columns the lanes
        // with bit `off` keep the last n, the others the first.  M stays float32: the
        // first step is taken while its 16 columns are formed, so that half as many
        // registers hold it until the products run.  After steps of 16, 8, 4 and 2 for
        // each half of the 32 columns and one of 1 between the halves, lane l has the
        // sum of column 16 (l % 2) + l / 2.
        auto fold = [&](float* x, int n, int off) {
            const bool up = (lane & off) != 0;
#pragma unroll
            for (int t = 0; t < n; ++t) {
                const float give = up ? x[t] : x[t + n];
                const float keep = up ? x[t + n] : x[t];
                x[t] = keep + __shfl_xor_sync(0xffffffffu, give, off);
            }
        };
        auto put = [&](int t_acc, uint8_t* tile) {
#pragma unroll
            for (int s = 0; s < GC / 16; ++s) {
                float ov[16];
                tmem_load<16>(tmem + lane_base + t_acc + d0 + 16 * s, ov);
                store_row_bf16<16>(tile, C, irow, d0 + 16 * s, ov);
            }
        };
        for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x, ++m) {
            const GateTabBlock& tab = tabs[m & 1];
            if (!(ok = wait(&tab_full[m & 1], (m >> 1) & 1))) break;
            const float gi = tab.loc[irow];
            const double gI = tab.start[sp];
            const float r_q = prm.scale * ex2_fast(gi + float(gI));
            const float r_k = ex2_fast(float(tab.start[4] - gI) - gi);
            const int J = grp;
            const float rJ = J < sp ? ex2_fast(gi + float(gI - tab.start[J + 1])) : 0.f;
            float rsum = 0.f, csum = 0.f, through = 0.f;
            uint8_t* kt = smem + Cfg::OFF_KV + (m % NB) * 2 * TILE;
            for (int g = 0; g < G; ++g, ++u) {
                if (!(ok = wait(pw_raw, u & 1))) break;
                tc_fence_after();
                float mm[16];             // M, folded once: see fold
                uint32_t pp[16], wp[16];  // P~, W~ in bf16 pairs
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    float pv[16], wv[16], ms[16];
                    if (J <= sp) {
                        tmem_ld16(tmem + lane_base + Cfg::T_P + c0 + 16 * s, pv);
                        tmem_load<16>(tmem + lane_base + Cfg::T_W + c0 + 16 * s, wv);
                        if (J == sp) {
#pragma unroll
                            for (int t = 0; t < 16; ++t) {
                                const int tt = 16 * s + t;
                                const float e = prm.scale * ex2_fast(gi - tab.loc[c0 + tt]);
                                const float a = tt <= lane ? pv[t] * e : 0.f;
                                ms[t] = tt < lane ? a * wv[t] : 0.f;  // the diagonal passes no gate
                                pv[t] = a;
                                wv[t] = tt <= lane ? wv[t] * e : 0.f;
                            }
                        } else {
#pragma unroll
                            for (int t = 0; t < 16; t += 4) {
                                const float4 f =
                                    *reinterpret_cast<const float4*>(tab.fac + c0 + 16 * s + t);
                                const float2 r2 = make_float2(prm.scale * rJ, prm.scale * rJ);
                                const float2 fj[2] = {mul2(r2, make_float2(f.x, f.y)),
                                                      mul2(r2, make_float2(f.z, f.w))};
#pragma unroll
                                for (int w = 0; w < 2; ++w) {
                                    const int j = t + 2 * w;
                                    const float2 p = mul2(make_float2(pv[j], pv[j + 1]), fj[w]);
                                    const float2 x = make_float2(wv[j], wv[j + 1]);
                                    const float2 mv = mul2(p, x), y = mul2(x, fj[w]);
                                    pv[j] = p.x, pv[j + 1] = p.y;
                                    ms[j] = mv.x, ms[j + 1] = mv.y;
                                    wv[j] = y.x, wv[j + 1] = y.y;
                                }
                            }
                        }
                    } else {
#pragma unroll
                        for (int t = 0; t < 16; ++t) pv[t] = wv[t] = ms[t] = 0.f;
                    }
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        pp[8 * s + t] = pack_bf16(pv[2 * t], pv[2 * t + 1]);
                        wp[8 * s + t] = pack_bf16(wv[2 * t], wv[2 * t + 1]);
                    }
                    if (J <= sp) {
#pragma unroll
                        for (int t = 0; t < 16; ++t) rsum += ms[t];
                        fold(ms, 8, 16);
                    }
#pragma unroll
                    for (int t = 0; t < 8; ++t) mm[8 * s + t] = ms[t];
                }
                tc_fence_before();
                warp_arrive(p_read);
                uint8_t* qt = smem + Cfg::OFF_QD + (u % NB) * 2 * TILE;
                if (!(ok = wait(&qd_full[u % NB], (u / NB) & 1) &&
                           wait(&kv_full[m % NB], (m / NB) & 1)))
                    break;
                if (STATE) {
                    // the parts through the states are complete; D = 128: S and R are
                    // read, and their space takes P~ and W~
                    if (!(ok = wait(s_full, u & 1))) break;
                    tc_fence_after();
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t off = tile_chunk_off(C, irow, c0 / 8 + j);
                    *reinterpret_cast<uint4*>(pt + off) =
                        make_uint4(pp[4 * j], pp[4 * j + 1], pp[4 * j + 2], pp[4 * j + 3]);
                    *reinterpret_cast<uint4*>(wt + off) =
                        make_uint4(wp[4 * j], wp[4 * j + 1], wp[4 * j + 2], wp[4 * j + 3]);
                }
                if (STATE) {
                    rsum += scale_part(Cfg::T_DQ, r_q, qt);
                    if (g == 0) {
                        through = scale_part(Cfg::T_DK, r_k, kt);
                        (void)scale_part(Cfg::T_DV, r_k, nullptr);
                    }
                    tmem_wait_st();
                }
                fence_proxy_async_smem();
                tc_fence_before();
                warp_arrive(pw_full);
                if (J <= sp) {  // the rest of M's column sums while the products run
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        fold(mm + 8 * s, 4, 8);
                        fold(mm + 8 * s, 2, 4);
                        fold(mm + 8 * s, 1, 2);
                    }
                    mm[1] = mm[8];
                    fold(mm, 1, 1);
                    csum += mm[0];
                }
                // staged over the tiles that nothing reads any more; the store warp is
                // done with the step before
                if (!(ok = wait(a_full, u & 1) &&
                           (u == 0 || wait(&qd_free[(u - 1) % NB], ((u - 1) / NB) & 1))))
                    break;
                tc_fence_after();
                put(Cfg::T_DQ, qt);
                fence_proxy_async_smem();
                tc_fence_before();
                warp_arrive(dq_read);
                warp_arrive(dq_out);
                if (g == G - 1) put(Cfg::T_DK, kt);
                if (!(ok = wait(b_full, u & 1))) break;
                tc_fence_after();
                if (g == G - 1) put(Cfg::T_DV, kt + TILE);
            }
            if (!ok) break;
            if (!(ok = m == 0 || (wait(red_free, (m - 1) & 1) &&
                                  wait(&kv_free[(m - 1) % NB], ((m - 1) / NB) & 1))))
                break;
            red[grp * C + irow] = rsum;
            red[(4 + sp) * C + c0 + 16 * (lane & 1) + (lane >> 1)] = csum;
            red[(8 + grp) * C + irow] = through;
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(kv_read);
            warp_arrive(kv_out);
            warp_arrive(&tab_free[m & 1]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace la
