// la_gated_api.cuh — entry points of gated linear attention and the head-row
// group norm (declared in include/la_api.h): argument checks, workspace plans
// and launches.  Included by la_api.cu, whose checks and helpers it uses.
#pragma once

#include "la_gated_bwd.cuh"
#include "la_gated_chain.cuh"
#include "la_gated_decode.cuh"
#include "la_gated_generic.cuh"
#include "la_gated_tc.cuh"
#include "la_norm.cuh"

namespace {

constexpr int64_t kMaxBlocks = (int64_t(1) << 31) - 1;

// ------------------------------------------------------------------ the plan
// Records of D*D float32 per key/value head and 64-token chunk: the state
// entering each chunk (S), and for the backward the gradient of the state
// leaving it (R), each with its chunks' gate products.  A head of one chunk with
// neither state given leaves them unused; they are reserved all the same, since
// the size is asked for without saying which states are given.
struct GatedPlan {
    int64_t nchunk = 0;
    size_t rec_bytes = 0, tot_bytes = 0;
    size_t s_rec = 0, s_tot = 0, r_rec = 0, r_tot = 0, bytes = 0;
};

GatedPlan plan_gated(la_op op, int64_t B, int64_t Hkv, int64_t N, int64_t D) {
    GatedPlan p;
    const int64_t kvh = B * Hkv;
    p.nchunk = (N + la::kGatedC - 1) / la::kGatedC;
    p.rec_bytes = round_up(size_t(kvh) * size_t(p.nchunk) * size_t(D * D) * 4, 256);
    p.tot_bytes = round_up(size_t(kvh) * size_t(p.nchunk) * 4, 256);
    p.s_rec = 0;
    p.s_tot = p.rec_bytes;
    p.bytes = p.rec_bytes + p.tot_bytes;
    if (op == LA_OP_BACKWARD) {
        p.r_rec = p.bytes;
        p.r_tot = p.r_rec + p.rec_bytes;
        p.bytes += p.rec_bytes + p.tot_bytes;
    }
    return p;
}

// Tensor-core path (bf16, D = 64 or 128): 128-token blocks, spans of nb
// blocks.  One float32 record array serves both directions' parts in turn; the
// states entering the spans are bf16, one array each for S and R.
struct GatedTcPlan {
    int64_t nblk = 0;
    int nb = 0, nspan = 0;
    // value columns a CTA of the walk takes, for S and for R; 0: spans in parallel
    int chain = 0, chain_r = 0;
    size_t rec = 0, tot = 0, s_enter = 0, r_enter = 0, bytes = 0;
    // parts of <S, R> a block of the backward adds up, and where they are
    int ndots = 0;
    size_t dots = 0, dots_bytes = 0;
};

// How the border states are formed: spans in parallel (0; two launches and the
// float32 records) or a walk of CTAs of 64 or 32 value columns, whichever the
// model below says is sooner, in us.  G: tiles a block (a group's query heads,
// for R).  Measured for S, bf16 to the blocks only (spans; walk with 64; with
// 32): 128 heads of 8192 tokens, D = 64: 118, 94, 122; 64 of 4096, D = 128,
// single blocks: 89, 62, 79; 32 of 131072, D = 128: 763, 1326, 916; 8 of 777, D =
// 128, single blocks: 20, 19, 15; 8 of 16384, D = 64: 38, 174, 138.  With a
// float32 state for the caller 134, 104, 123 for the first.  For R with <S, R>,
// in the same order: 183, 129, 158; 155, 81, 101; 29, 37, 27 (groups of 4); 78,
// 239, 180.
int pick_chain(int64_t kvh, int64_t nblk, int64_t D, int64_t G) {
    const double sms = num_sms(), tiles = double(nblk) * double(G);
    const double spans = 10.0 + double(kvh) * tiles * (D == 64 ? 0.0134 : 0.0243);
    const double w64 = 4.0 + ceil(double(kvh) * double(D / 64) / sms) * tiles * 1.5;
    const double w32 = 4.0 + ceil(double(kvh) * double(D / 32) / sms) * tiles * 0.9;
    if (spans <= w64 && spans <= w32) return 0;
    return w64 <= w32 ? 64 : 32;
}

GatedTcPlan plan_gated_tc(la_op op, int64_t B, int64_t H, int64_t Hkv, int64_t N, int64_t D) {
    GatedTcPlan p;
    p.nblk = (N + la::kGtC - 1) / la::kGtC;
    // A sequence of one span needs no border states, so up to four blocks are
    // one.  Longer spans move fewer state bytes (D^2 a span) and take more C x C
    // products (nb + 1 over 2 a block) and more of L2: states and outputs of
    // 131072 tokens, 32 heads, D = 128 take 2024 us with one block a span, 1723
    // with two, 1866 with four; of 8192 tokens, 128 heads, D = 64: 209, 240, 273.
    // The backward kernels take single blocks.
    if (op == LA_OP_BACKWARD)
        p.nb = 1;
    else
        p.nb = p.nblk <= 1 ? 1 : p.nblk == 2 ? 2 : p.nblk <= 4 ? 4 : D == 64 ? 1 : 2;
    p.nspan = int((p.nblk + p.nb - 1) / p.nb);
    p.chain = pick_chain(B * Hkv, p.nblk, D, 1);
    p.chain_r = op == LA_OP_BACKWARD ? pick_chain(B * Hkv, p.nblk, D, H / Hkv) : p.chain;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += round_up(n, 256);
        return o;
    };
    const size_t states = size_t(B) * size_t(Hkv) * size_t(p.nspan) * size_t(D * D);
    if (!p.chain || !p.chain_r) {
        p.rec = take(states * 4);
        p.tot = take(size_t(B) * size_t(Hkv) * size_t(p.nspan) * 4);
    }
    p.s_enter = take(states * 2);
    if (op == LA_OP_BACKWARD) {
        p.r_enter = take(states * 2);
        p.ndots = int(p.chain_r ? 8 * D / p.chain_r : D * D / 128);
        p.dots_bytes = size_t(B) * size_t(Hkv) * size_t(p.nspan) * size_t(p.ndots) * 4;
        p.dots = take(p.dots_bytes);
    }
    p.bytes = at;
    return p;
}

template <typename T, int D>
constexpr bool gated_on_tensor_cores = std::is_same<T, __nv_bfloat16>::value && (D == 64 || D == 128);

// A few tokens that no state enters or leaves, of at most a head an SM, run on
// the plain cores in every type, so that a call of so few products is rounded
// once; a token more, a head more or a state, and the products and states are
// operands in bf16 again.  The kernels' times there, 16 tokens on the plain cores
// and 17 on the tensor cores, us: forward D = 64 with 1, 37 and 148 heads 4.7, 5.0,
// 5.1 and 6.5, 6.6, 7.4; D = 128: 6.4, 6.6, 6.6 and 6.8, 6.9, 7.5.  Backward, whose
// blocks are four a head: D = 64 6.6, 6.6, 14.1 and 7.6, 7.7, 8.1; D = 128: 9.3, 9.0,
// 28.9 and 8.3, 8.4, 9.0: above a block an SM it costs time for its rounding.
bool gated_few_tokens(int64_t B, int64_t H, int64_t N, bool states) {
    return !states && N <= 16 && B * H <= num_sms();
}

// Sizes a gated launch can take: at most four blocks per 64 tokens of a head.
la_status check_gated(int64_t B, int64_t H, int64_t Hkv, int64_t N, int64_t D, la_dtype dt) {
    la_status s;
    if (dt != LA_F32 && dt != LA_BF16) return LA_ERR_INVALID_ARG;
    if ((s = check_sizes(B, H, N, D)) != LA_OK) return s;
    if ((s = check_group(H, Hkv)) != LA_OK) return s;
    if (N > 0 && 4 * B * H > kMaxBlocks / ((N + la::kGatedC - 1) / la::kGatedC))
        return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

// Gates are read and written one by one, so a slice of a larger tensor will do.
la_status check_gate_ptr(const void* p, la_dtype dt) {
    const uintptr_t mask = dt == LA_F32 ? 3u : 1u;
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) & mask) ? LA_ERR_INVALID_ARG : LA_OK;
}

la_status check_opt(const void* p) {
    return p != nullptr && !aligned16(p) ? LA_ERR_INVALID_ARG : LA_OK;
}

template <typename K>
la_status allow_smem(K kern, size_t bytes) {
    if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             int(bytes)))
        return cuda_fail("cudaFuncSetAttribute", e);
    return LA_OK;
}

// ------------------------------------------------------ the plain-core kernels
// Border states of every chunk: parts, then the recurrence; the forward
// direction (S, from k and v) and the backward one (R, from q and dO) together.
// A job without records is left out; `last` (may be null) receives the state
// after the last chunk walked.
template <typename T, int D>
la_status gated_states(la::GatedPartJob f, la::GatedCarryJob fc, la::GatedPartJob r,
                       la::GatedCarryJob rc, const T* lg, int64_t kvh, int64_t N, int64_t nchunk,
                       cudaStream_t st) {
    la_status s;
    auto fill = [&](la::GatedPartJob& p, la::GatedCarryJob& c, bool rev) {
        p.run = int(!c.rec ? 0 : c.last ? nchunk : nchunk - 1);
        p.chunk0 = rev && !c.last ? 1 : 0;
        p.blocks = kvh * p.run;
        p.rec = reinterpret_cast<float*>(c.rec);
        p.gtot = const_cast<float*>(c.gtot);
    };
    fill(f, fc, false);
    fill(r, rc, true);
    if (f.blocks + r.blocks > 0) {
        const size_t smem = size_t(2) * la::kGatedC * la::GatedTile::ld(D) * 4;
        auto kern = la::gated_part_kernel<T, D>;
        if ((s = allow_smem(kern, smem)) != LA_OK) return s;
        la::LaunchScope scope("gated_part", st);
        kern<<<unsigned(f.blocks + r.blocks), la::kGatedThreads, smem, st>>>(f, r, lg, N,
                                                                            int(nchunk));
        if ((s = launch_status()) != LA_OK) return s;
    }
    const int per = D * D / 4;
    const int64_t total = kvh * per;
    la::LaunchScope scope("gated_carry", st);
    la::gated_carry_kernel<<<dim3(unsigned((total + 127) / 128), rc.rec ? 2 : 1), 128, 0, st>>>(
        fc, rc, total, per, int(nchunk));
    return launch_status();
}

// ---------------------------------------------------- the tensor-core kernels
template <int D, int EC, bool REV, int SPLIT>
la_status gated_tc_chain(const void* A, const void* Bm, const void* lg, const GatedTcPlan& p,
                         char* ws, size_t enter, const float* first, float* last, int64_t heads,
                         int64_t kvh, int64_t N, int group, float mul, cudaStream_t st) {
    using Cfg = la::GatedChainCfg<D, EC, SPLIT>;
    la_status s;
    la::GatedChainParams prm;
    memset(&prm, 0, sizeof(prm));
    if (!make_qkv_map(&prm.tm_a, A, heads, N, D, la::kGtC)) return LA_ERR_CUDA;
    prm.b = static_cast<const __nv_bfloat16*>(Bm), prm.lg = static_cast<const __nv_bfloat16*>(lg);
    prm.first = first, prm.last = last;
    if (REV && p.dots_bytes) {
        prm.S = reinterpret_cast<const __nv_bfloat16*>(ws + p.s_enter);
        prm.dots = reinterpret_cast<float*>(ws + p.dots);
    }
    prm.enter = reinterpret_cast<__nv_bfloat16*>(ws + enter);
    prm.N = N, prm.nblk = int(p.nblk), prm.nb = p.nb, prm.nspan = p.nspan, prm.group = group;
    prm.mul = mul;
    // without `last` the span walked last adds nothing that is asked for
    prm.blocks = last ? prm.nblk : REV ? std::max(0, prm.nblk - p.nb) : (p.nspan - 1) * p.nb;
    auto kern = la::gated_chain_kernel<D, EC, REV, SPLIT>;
    if ((s = allow_smem(kern, Cfg::SMEM)) != LA_OK) return s;
    la::LaunchScope scope(EC == 64 ? (REV ? "gated_chain64_rev" : "gated_chain64")
                                   : (REV ? "gated_chain32_rev" : "gated_chain32"),
                          st);
    kern<<<unsigned(kvh * (D / EC)), la::kGatedChainThreads, Cfg::SMEM, st>>>(prm);
    return launch_status();
}

template <int D, bool REV>
la_status gated_tc_states(const void* A, const void* Bm, const void* lg, const GatedTcPlan& p,
                          char* ws, size_t enter, const float* first, float* last, int64_t heads,
                          int64_t kvh, int64_t N, int group, float mul, cudaStream_t st) {
    la_status s;
    const int chain = REV ? p.chain_r : p.chain;
    auto walk = [&](auto ec, auto split) {
        return gated_tc_chain<D, decltype(ec)::value, REV, decltype(split)::value>(
            A, Bm, lg, p, ws, enter, first, last, heads, kvh, N, group, mul, st);
    };
    using std::integral_constant;
    if (chain == 32)
        return last ? walk(integral_constant<int, 32>{}, integral_constant<int, 3>{})
                    : walk(integral_constant<int, 32>{}, integral_constant<int, 2>{});
    if (chain)
        return last ? walk(integral_constant<int, 64>{}, integral_constant<int, 3>{})
                    : walk(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    const int run = last ? p.nspan : p.nspan - 1;
    float* rec = reinterpret_cast<float*>(ws + p.rec);
    float* tot = reinterpret_cast<float*>(ws + p.tot);
    if (run > 0) {
        la::GatedSpanParams prm;
        memset(&prm, 0, sizeof(prm));
        if (!make_qkv_map(&prm.tm_a, A, heads, N, D, la::kGtC) ||
            !make_qkv_map(&prm.tm_b, Bm, heads, N, D, la::kGtC))
            return LA_ERR_CUDA;
        prm.lg = static_cast<const __nv_bfloat16*>(lg);
        prm.rec = rec, prm.tot = tot, prm.N = N;
        prm.items = kvh * run, prm.nspan = p.nspan, prm.spans_run = run;
        prm.span0 = REV && !last ? 1 : 0;
        prm.nb = p.nb, prm.nblk = int(p.nblk), prm.group = group, prm.mul = mul;
        auto go = [&](auto split) -> la_status {
            using Cfg = la::GatedSpanCfg<D, decltype(split)::value>;
            auto kern = la::gated_span_kernel<D, REV, decltype(split)::value>;
            if (la_status e = allow_smem(kern, Cfg::SMEM)) return e;
            const unsigned grid =
                unsigned(std::min<int64_t>(prm.items, int64_t(num_sms()) * Cfg::CTAS));
            la::LaunchScope scope(REV ? "gated_span_rev" : "gated_span", st);
            kern<<<grid, la::kGatedSpanThreads, Cfg::SMEM, st>>>(prm);
            return launch_status();
        };
        s = last ? go(std::integral_constant<int, 3>{}) : go(std::integral_constant<int, 2>{});
        if (s != LA_OK) return s;
    }
    const int per = D * D / 4;
    const int64_t total = kvh * per;
    la::LaunchScope scope(REV ? "gated_border_rev" : "gated_border", st);
    la::gated_border_kernel<REV><<<unsigned((total + 127) / 128), 128, 0, st>>>(
        reinterpret_cast<const float4*>(rec), tot, reinterpret_cast<const float4*>(first),
        reinterpret_cast<float4*>(last), reinterpret_cast<uint2*>(ws + enter),
        REV && p.dots_bytes ? reinterpret_cast<const uint2*>(ws + p.s_enter) : nullptr,
        reinterpret_cast<float*>(ws + p.dots), total, per, p.nspan);
    return launch_status();
}

template <int D>
la_status run_gated_fwd_tc(const void* q, const void* k, const void* v, const void* lg, void* o,
                           const float* S_in, float* S_out, float scale, int64_t B, int64_t H,
                           int64_t Hkv, int64_t N, char* ws, cudaStream_t st) {
    const GatedTcPlan p = plan_gated_tc(LA_OP_FORWARD, B, H, Hkv, N, D);
    const int64_t kvh = B * Hkv;
    const bool through = p.nspan > 1 || S_in || S_out;
    if (through) {
        la_status s = gated_tc_states<D, false>(k, v, lg, p, ws, p.s_enter, S_in, S_out, kvh, kvh,
                                                N, 1, 1.f, st);
        if (s != LA_OK) return s;
    }
    const bool state = p.nspan > 1 || S_in;
    using Cfg = la::GatedBlockCfg<D>;
    la::GatedBlockParams prm;
    memset(&prm, 0, sizeof(prm));
    constexpr int C = la::kGtC;
    if (!make_qkv_map(&prm.tm_q, q, B * H, N, D, C) || !make_qkv_map(&prm.tm_k, k, kvh, N, D, C) ||
        !make_qkv_map(&prm.tm_v, v, kvh, N, D, C) || !make_qkv_map(&prm.tm_o, o, B * H, N, D, C) ||
        (state && !make_qkv_map(&prm.tm_st, ws + p.s_enter, kvh * p.nspan, D, D, D)))
        return LA_ERR_CUDA;
    prm.lg = static_cast<const __nv_bfloat16*>(lg);
    prm.N = N, prm.items = B * H * p.nblk;
    prm.nblk = int(p.nblk), prm.nb = p.nb, prm.nspan = p.nspan, prm.group = int(H / Hkv);
    prm.has_state = state, prm.scale = scale;
    auto kern = la::gated_block_kernel<D>;
    la_status s;
    if ((s = allow_smem(kern, Cfg::SMEM)) != LA_OK) return s;
    const unsigned grid = unsigned(std::min<int64_t>(prm.items, int64_t(num_sms()) * Cfg::CTAS));
    la::LaunchScope scope("gated_o", st);
    kern<<<grid, Cfg::THREADS, Cfg::SMEM, st>>>(prm);
    return launch_status();
}

template <int D>
la_status run_gated_bwd_tc(const void* q, const void* k, const void* v, const void* lg,
                           const void* dO, const float* S_in, const float* dS_out, void* dq,
                           void* dk, void* dv, void* dlg, float* dS_in, float scale, int64_t B,
                           int64_t H, int64_t Hkv, int64_t N, char* ws, cudaStream_t st) {
    la_status s;
    GatedTcPlan p = plan_gated_tc(LA_OP_BACKWARD, B, H, Hkv, N, D);
    const int group = int(H / Hkv);
    const int64_t kvh = B * Hkv, qh = B * H;
    // the blocks take both border states or, a single block that nothing enters
    // or leaves, none
    const bool state = p.nspan > 1 || S_in || dS_out;
    if (!state) p.dots_bytes = 0;  // S is not formed
    if (state && (s = gated_tc_states<D, false>(k, v, lg, p, ws, p.s_enter, S_in, nullptr, kvh, kvh,
                                                N, 1, 1.f, st)) != LA_OK)
        return s;
    if ((state || dS_in) &&
        (s = gated_tc_states<D, true>(q, dO, lg, p, ws, p.r_enter, dS_out, dS_in, qh, kvh, N, group,
                                      scale, st)) != LA_OK)
        return s;
    la::GatedBwdParams prm;
    memset(&prm, 0, sizeof(prm));
    constexpr int C = la::kGtC;
    if (!make_qkv_map(&prm.tm_q, q, qh, N, D, C) || !make_qkv_map(&prm.tm_k, k, kvh, N, D, C) ||
        !make_qkv_map(&prm.tm_v, v, kvh, N, D, C) || !make_qkv_map(&prm.tm_do, dO, qh, N, D, C) ||
        !make_qkv_map(&prm.tm_dq, dq, qh, N, D, C) || !make_qkv_map(&prm.tm_dk, dk, kvh, N, D, C) ||
        !make_qkv_map(&prm.tm_dv, dv, kvh, N, D, C) ||
        (state && (!make_qkv_map(&prm.tm_s, ws + p.s_enter, kvh * p.nspan, D, D, D) ||
                   !make_qkv_map(&prm.tm_r, ws + p.r_enter, kvh * p.nspan, D, D, D))))
        return LA_ERR_CUDA;
    prm.lg = static_cast<const __nv_bfloat16*>(lg), prm.dlg = static_cast<__nv_bfloat16*>(dlg);
    prm.N = N, prm.items = kvh * p.nblk, prm.nblk = int(p.nblk), prm.group = group;
    prm.dots = reinterpret_cast<const float*>(ws + p.dots), prm.ndots = p.ndots;
    prm.scale = scale;
    auto kern = state ? la::gated_bwd_kernel<D, true> : la::gated_bwd_kernel<D, false>;
    constexpr size_t kSmem = la::GatedBwdCfg<D>::SMEM;
    if ((s = allow_smem(kern, kSmem)) != LA_OK) return s;
    la::LaunchScope scope("gated_bwd", st);
    kern<<<unsigned(std::min<int64_t>(prm.items, num_sms())), la::kGatedBwdThreads, kSmem, st>>>(prm);
    return launch_status();
}

template <typename T, int D>
la_status run_gated_fwd(const void* q, const void* k, const void* v, const void* lg, void* o,
                        const float* S_in, float* S_out, float scale, int64_t B, int64_t H,
                        int64_t Hkv, int64_t N, char* ws, cudaStream_t st) {
    la_status s;
    const GatedPlan p = plan_gated(LA_OP_FORWARD, B, Hkv, N, D);
    la::GatedTensors<T> t{};
    t.q = static_cast<const T*>(q), t.k = static_cast<const T*>(k), t.v = static_cast<const T*>(v);
    t.lg = static_cast<const T*>(lg), t.o = static_cast<T*>(o);
    t.N = N, t.qheads = B * H, t.kvh = B * Hkv, t.nchunk = int(p.nchunk);
    t.group = int(H / Hkv), t.scale = scale;
    if (p.nchunk > 1 || S_in || S_out) {
        t.S = reinterpret_cast<float*>(ws + p.s_rec);
        const la::GatedPartJob f{k, v, nullptr, nullptr, 0, 0, 0, 1, 1.f};
        const la::GatedCarryJob fc{reinterpret_cast<float4*>(ws + p.s_rec),
                                   reinterpret_cast<float*>(ws + p.s_tot),
                                   reinterpret_cast<const float4*>(S_in),
                                   reinterpret_cast<float4*>(S_out)};
        if ((s = gated_states<T, D>(f, fc, {}, {}, t.lg, t.kvh, N, p.nchunk, st)) != LA_OK) return s;
    }
    const size_t smem = (size_t(3) * la::kGatedC * la::GatedTile::ld(D) +
                         la::kGatedC * la::GatedTile::ld(la::kGatedC)) * 4;
    auto kern = la::gated_o_kernel<T, D>;
    if ((s = allow_smem(kern, smem)) != LA_OK) return s;
    la::LaunchScope scope("gated_o", st);
    kern<<<unsigned(t.qheads * p.nchunk), la::kGatedThreads, smem, st>>>(t);
    return launch_status();
}

template <typename T, int D>
la_status run_gated_bwd(const void* q, const void* k, const void* v, const void* lg,
                        const void* dO, const float* S_in, const float* dS_out, void* dq,
                        void* dk, void* dv, void* dlg, float* dS_in, float scale, int64_t B,
                        int64_t H, int64_t Hkv, int64_t N, char* ws, cudaStream_t st) {
    la_status s;
    const GatedPlan p = plan_gated(LA_OP_BACKWARD, B, Hkv, N, D);
    la::GatedTensors<T> t{};
    t.q = static_cast<const T*>(q), t.k = static_cast<const T*>(k), t.v = static_cast<const T*>(v);
    t.lg = static_cast<const T*>(lg), t.dO = static_cast<const T*>(dO);
    t.dq = static_cast<T*>(dq), t.dk = static_cast<T*>(dk), t.dv = static_cast<T*>(dv);
    t.dlg = static_cast<T*>(dlg);
    t.N = N, t.qheads = B * H, t.kvh = B * Hkv, t.nchunk = int(p.nchunk);
    t.group = int(H / Hkv), t.scale = scale;
    la::GatedCarryJob fc{}, rc{};
    if (p.nchunk > 1 || S_in) {
        t.S = reinterpret_cast<float*>(ws + p.s_rec);
        fc = {reinterpret_cast<float4*>(ws + p.s_rec), reinterpret_cast<float*>(ws + p.s_tot),
              reinterpret_cast<const float4*>(S_in), nullptr};
    }
    if (p.nchunk > 1 || dS_out || dS_in) {
        t.R = reinterpret_cast<float*>(ws + p.r_rec);
        rc = {reinterpret_cast<float4*>(ws + p.r_rec), reinterpret_cast<float*>(ws + p.r_tot),
              reinterpret_cast<const float4*>(dS_out), reinterpret_cast<float4*>(dS_in)};
    }
    if (t.S || t.R) {
        const la::GatedPartJob f{k, v, nullptr, nullptr, 0, 0, 0, 1, 1.f};
        const la::GatedPartJob r{q, dO, nullptr, nullptr, 0, 0, 0, t.group, scale};
        if ((s = gated_states<T, D>(f, fc, r, rc, t.lg, t.kvh, N, p.nchunk, st)) != LA_OK) return s;
    }
    // dlog_gate's four tiles, or three and the C x C product
    const size_t smem = (size_t(3) * la::kGatedC * la::GatedTile::ld(D) +
                         la::kGatedC * la::GatedTile::ld(std::max(D, la::kGatedC))) * 4;
    auto kern = la::gated_grad_kernel<T, D>;
    if ((s = allow_smem(kern, smem)) != LA_OK) return s;
    la::LaunchScope scope("gated_grad", st);
    kern<<<unsigned((3 * t.kvh + t.qheads) * p.nchunk), la::kGatedThreads, smem, st>>>(t);
    return launch_status();
}

// fn.template operator()<T, D>() for the call's type and head size
template <typename Fn>
la_status with_type_and_size(la_dtype dt, int64_t D, Fn&& fn) {
    auto size = [&](auto t) {
        using T = decltype(t);
        switch (D) {
            case 16: return fn(t, std::integral_constant<int, 16>{});
            case 32: return fn(t, std::integral_constant<int, 32>{});
            case 64: return fn(t, std::integral_constant<int, 64>{});
            default: return fn(T{}, std::integral_constant<int, 128>{});
        }
    };
    return dt == LA_F32 ? size(float{}) : size(__nv_bfloat16{});
}

template <typename T, int D>
la_status run_gated_step(float* S, const void* q, const void* k, const void* v, const void* lg,
                         void* o, float scale, int64_t kvh, int G, cudaStream_t st) {
    const T *tq = static_cast<const T*>(q), *tk = static_cast<const T*>(k),
            *tv = static_cast<const T*>(v), *tl = static_cast<const T*>(lg);
    la::LaunchScope scope("gated_step", st);
    constexpr int DC = la::gated_step_columns<D>;
    la::gated_step_kernel<T, D, DC><<<unsigned(kvh * (D / DC)), 2 * D, 0, st>>>(
        S, tq, tk, tv, tl, static_cast<T*>(o), G, scale);
    return launch_status();
}

// ------------------------------------------------------------------ group norm
struct NormPlan {
    int groups = 0, span = 0, slots = 0, threads = 0, spans = 0, blocks = 0;
    size_t bytes = 0;  // backward: partial sums
};

// A block covers 256 groups of 16 bytes of a token's channels, or several
// tokens of fewer.  The tokens are dealt over as many blocks as keep every SM
// full (kNormBlocks), each block at least one.
NormPlan plan_norm(int64_t B, int64_t H, int64_t N, int64_t D, la_dtype dt, bool bwd) {
    NormPlan p;
    p.groups = int(H * D * (dt == LA_F32 ? 4 : 2) / 16);
    p.span = std::min(p.groups, 256);
    p.slots = std::max(1, 256 / p.span);
    p.threads = (p.span * p.slots + 31) / 32 * 32;
    p.spans = (p.groups + p.span - 1) / p.span;
    const int64_t tokens = B * N;
    const int per_sm = dt == LA_F32 ? (bwd ? la::kNormBlocks<float, true> : la::kNormBlocks<float, false>)
                                    : (bwd ? la::kNormBlocks<__nv_bfloat16, true>
                                           : la::kNormBlocks<__nv_bfloat16, false>);
    const int64_t want = std::max<int64_t>(1, int64_t(num_sms()) * per_sm / p.spans);
    p.blocks = int(std::max<int64_t>(1, std::min(want, (tokens + p.slots - 1) / p.slots)));
    if (bwd) p.bytes = size_t(2) * size_t(p.blocks) * size_t(H * D) * 4;
    return p;
}

la_status check_norm(int64_t B, int64_t H, int64_t N, int64_t D, la_dtype dt, la_act act,
                     float eps) {
    if (dt != LA_F32 && dt != LA_BF16) return LA_ERR_INVALID_ARG;
    if (act != LA_ACT_IDENTITY && act != LA_ACT_SILU) return LA_ERR_INVALID_ARG;
    if (!(eps > 0.f) || eps > 3.0e38f) return LA_ERR_INVALID_ARG;  // NaN fails too
    la_status s = check_sizes(B, H, N, D);
    if (s != LA_OK) return s;
    return H * D > (int64_t(1) << 24) ? LA_ERR_UNSUPPORTED : LA_OK;
}

template <typename T, int D, bool BWD>
la_status launch_norm(const la::NormParams& prm, const NormPlan& p, bool gate, la_act act,
                      cudaStream_t st) {
    const dim3 grid(unsigned(p.blocks), unsigned(p.spans));
    const size_t smem = size_t(la::kNormStages) * size_t(1 + gate + BWD) * size_t(p.threads) * 16;
    auto go = [&](auto G, auto A) {
        auto kern = la::group_norm_kernel<T, D, BWD, decltype(G)::value, decltype(A)::value>;
        if (la_status s = allow_smem(kern, smem)) return s;
        la::LaunchScope scope(BWD ? "group_norm_bwd" : "group_norm", st);
        kern<<<grid, unsigned(p.threads), smem, st>>>(prm);
        return launch_status();
    };
    using std::integral_constant;
    if (gate)
        return act == LA_ACT_SILU ? go(std::true_type{}, integral_constant<int, la::ACT_SILU>{})
                                  : go(std::true_type{}, integral_constant<int, la::ACT_IDENTITY>{});
    return act == LA_ACT_SILU ? go(std::false_type{}, integral_constant<int, la::ACT_SILU>{})
                              : go(std::false_type{}, integral_constant<int, la::ACT_IDENTITY>{});
}

}  // namespace

extern "C" {

size_t la_workspace_size_gated(la_op op, int64_t B, int64_t H, int64_t Hkv, int64_t N, int64_t D,
                               la_dtype dt) {
    if (op != LA_OP_FORWARD && op != LA_OP_BACKWARD) return 0;
    if (check_gated(B, H, Hkv, N, D, dt) != LA_OK || B == 0 || H == 0 || N == 0) return 0;
    return fast_path(dt, D) ? plan_gated_tc(op, B, H, Hkv, N, D).bytes
                            : plan_gated(op, B, Hkv, N, D).bytes;
}

la_status la_forward_gated(const void* q, const void* k, const void* v, const void* log_gate,
                           void* o, const float* S_in, float* S_out, float scale, int64_t B,
                           int64_t H, int64_t Hkv, int64_t N, int64_t D, la_dtype dt,
                           void* workspace, size_t workspace_bytes, la_stream_t stream) {
    la_status s;
    if ((s = check_gated(B, H, Hkv, N, D, dt)) != LA_OK) return s;
    if ((s = check_opt(S_in)) != LA_OK || (s = check_opt(S_out)) != LA_OK) return s;
    if (S_in && S_in == S_out) return LA_ERR_INVALID_ARG;
    if ((s = check_opt(workspace)) != LA_OK) return s;
    if (B == 0 || H == 0) return LA_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t state = size_t(B) * size_t(Hkv) * size_t(D * D) * 4;
    if (N == 0) {  // the state passes through
        if (!S_out) return LA_OK;
        const cudaError_t e = S_in ? cudaMemcpyAsync(S_out, S_in, state,
                                                     cudaMemcpyDeviceToDevice, st)
                                   : cudaMemsetAsync(S_out, 0, state, st);
        return e == cudaSuccess ? LA_OK : cuda_fail("la_forward_gated: state copy", e);
    }
    if ((s = check_ptr(q)) || (s = check_ptr(k)) || (s = check_ptr(v)) ||
        (s = check_gate_ptr(log_gate, dt)) || (s = check_ptr(o)))
        return s;
    if (workspace == nullptr ||
        workspace_bytes < la_workspace_size_gated(LA_OP_FORWARD, B, H, Hkv, N, D, dt))
        return LA_ERR_WORKSPACE;
    if ((s = bind_context()) != LA_OK) return s;
    char* ws = static_cast<char*>(workspace);
    return with_type_and_size(dt, D, [&](auto t, auto d) {
        using T = decltype(t);
        constexpr int kD = decltype(d)::value;
        if constexpr (gated_on_tensor_cores<T, kD>)
            if (!gated_few_tokens(B, H, N, S_in || S_out))
                return run_gated_fwd_tc<kD>(q, k, v, log_gate, o, S_in, S_out, scale, B, H, Hkv, N,
                                            ws, st);
        return run_gated_fwd<T, kD>(q, k, v, log_gate, o, S_in, S_out, scale, B, H, Hkv, N, ws, st);
    });
}

la_status la_backward_gated(const void* q, const void* k, const void* v, const void* log_gate,
                            const void* dO, const float* S_in, const float* dS_out, void* dq,
                            void* dk, void* dv, void* dlog_gate, float* dS_in, float scale,
                            int64_t B, int64_t H, int64_t Hkv, int64_t N, int64_t D, la_dtype dt,
                            void* workspace, size_t workspace_bytes, la_stream_t stream) {
    la_status s;
    if ((s = check_gated(B, H, Hkv, N, D, dt)) != LA_OK) return s;
    if ((s = check_opt(S_in)) != LA_OK || (s = check_opt(dS_out)) != LA_OK ||
        (s = check_opt(dS_in)) != LA_OK)
        return s;
    if (dS_in && (dS_in == dS_out || dS_in == S_in)) return LA_ERR_INVALID_ARG;
    if ((s = check_opt(workspace)) != LA_OK) return s;
    if (B == 0 || H == 0) return LA_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t state = size_t(B) * size_t(Hkv) * size_t(D * D) * 4;
    if (N == 0) {  // the state's gradient passes through
        if (!dS_in) return LA_OK;
        const cudaError_t e = dS_out ? cudaMemcpyAsync(dS_in, dS_out, state,
                                                       cudaMemcpyDeviceToDevice, st)
                                     : cudaMemsetAsync(dS_in, 0, state, st);
        return e == cudaSuccess ? LA_OK : cuda_fail("la_backward_gated: state copy", e);
    }
    if ((s = check_ptr(q)) || (s = check_ptr(k)) || (s = check_ptr(v)) ||
        (s = check_gate_ptr(log_gate, dt)) || (s = check_ptr(dO)) || (s = check_ptr(dq)) ||
        (s = check_ptr(dk)) || (s = check_ptr(dv)) || (s = check_gate_ptr(dlog_gate, dt)))
        return s;
    if (workspace == nullptr ||
        workspace_bytes < la_workspace_size_gated(LA_OP_BACKWARD, B, H, Hkv, N, D, dt))
        return LA_ERR_WORKSPACE;
    if ((s = bind_context()) != LA_OK) return s;
    char* ws = static_cast<char*>(workspace);
    return with_type_and_size(dt, D, [&](auto t, auto d) {
        using T = decltype(t);
        constexpr int kD = decltype(d)::value;
        if constexpr (gated_on_tensor_cores<T, kD>)
            if (!gated_few_tokens(B, H, N, S_in || dS_out || dS_in))
                return run_gated_bwd_tc<kD>(q, k, v, log_gate, dO, S_in, dS_out, dq, dk, dv,
                                            dlog_gate, dS_in, scale, B, H, Hkv, N, ws, st);
        return run_gated_bwd<T, kD>(q, k, v, log_gate, dO, S_in, dS_out, dq, dk, dv, dlog_gate,
                                    dS_in, scale, B, H, Hkv, N, ws, st);
    });
}

la_status la_decode_step_gated(float* S, const void* q, const void* k, const void* v,
                               const void* log_gate, void* o, float scale, int64_t B, int64_t H,
                               int64_t Hkv, int64_t D, la_dtype dt, la_stream_t stream) {
    la_status s;
    if ((s = check_gated(B, H, Hkv, 1, D, dt)) != LA_OK) return s;
    if (B == 0 || H == 0) return LA_OK;
    if (B * Hkv > kMaxBlocks / 8) return LA_ERR_UNSUPPORTED;
    if ((s = check_ptr(S)) || (s = check_ptr(q)) || (s = check_ptr(k)) || (s = check_ptr(v)) ||
        (s = check_gate_ptr(log_gate, dt)) || (s = check_ptr(o)))
        return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return with_type_and_size(dt, D, [&](auto t, auto d) {
        return run_gated_step<decltype(t), decltype(d)::value>(S, q, k, v, log_gate, o, scale,
                                                               B * Hkv, int(H / Hkv), st);
    });
}

la_status la_group_norm(const void* x, const void* gate, const float* weight, const float* bias,
                        void* y, float eps, la_act act, int64_t B, int64_t H, int64_t N,
                        int64_t D, la_dtype dt, la_stream_t stream) {
    la_status s;
    if ((s = check_norm(B, H, N, D, dt, act, eps)) != LA_OK) return s;
    if ((s = check_opt(gate)) != LA_OK || (s = check_opt(bias)) != LA_OK) return s;
    if (B == 0 || H == 0 || N == 0) return LA_OK;
    if ((s = check_ptr(x)) || (s = check_ptr(weight)) || (s = check_ptr(y))) return s;
    const NormPlan p = plan_norm(B, H, N, D, dt, false);
    la::NormParams prm{};
    prm.x = x, prm.gate = gate, prm.weight = weight, prm.bias = bias, prm.y = y;
    prm.tokens = B * N, prm.N = N, prm.H = int(H), prm.groups = p.groups;
    prm.span = p.span, prm.slots = p.slots, prm.eps = eps;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return with_type_and_size(dt, D, [&](auto t, auto d) {
        return launch_norm<decltype(t), decltype(d)::value, false>(prm, p, gate != nullptr, act,
                                                                   st);
    });
}

size_t la_workspace_size_group_norm(int64_t B, int64_t H, int64_t N, int64_t D, la_dtype dt) {
    if (check_norm(B, H, N, D, dt, LA_ACT_IDENTITY, 1.f) != LA_OK) return 0;
    if (B == 0 || H == 0 || N == 0) return 0;
    return plan_norm(B, H, N, D, dt, true).bytes;
}

la_status la_group_norm_backward(const void* x, const void* gate, const float* weight,
                                 const float* bias, const void* dy, void* dx, void* dgate,
                                 float* dweight, float* dbias, float eps, la_act act, int64_t B,
                                 int64_t H, int64_t N, int64_t D, la_dtype dt, void* workspace,
                                 size_t workspace_bytes, la_stream_t stream) {
    la_status s;
    if ((s = check_norm(B, H, N, D, dt, act, eps)) != LA_OK) return s;
    if ((s = check_opt(gate)) || (s = check_opt(bias)) || (s = check_opt(dgate)) ||
        (s = check_opt(dbias)) || (s = check_opt(workspace)))
        return s;
    if ((gate == nullptr) != (dgate == nullptr)) return LA_ERR_INVALID_ARG;
    if (H == 0) return LA_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = check_ptr(weight)) || (s = check_ptr(dweight))) return s;
    if (B == 0 || N == 0) {  // no rows: the channel sums are empty, and outputs still
        cudaError_t e = cudaMemsetAsync(dweight, 0, size_t(H * D) * 4, st);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, size_t(H * D) * 4, st);
        return e == cudaSuccess ? LA_OK : cuda_fail("la_group_norm_backward: zeros", e);
    }
    if ((s = check_ptr(x)) || (s = check_ptr(dy)) || (s = check_ptr(dx))) return s;
    const NormPlan p = plan_norm(B, H, N, D, dt, true);
    if (workspace == nullptr || workspace_bytes < p.bytes) return LA_ERR_WORKSPACE;
    la::NormParams prm{};
    prm.x = x, prm.gate = gate, prm.dy = dy, prm.weight = weight, prm.bias = bias;
    prm.dx = dx, prm.dgate = dgate, prm.part = static_cast<float*>(workspace);
    prm.tokens = B * N, prm.N = N, prm.H = int(H), prm.groups = p.groups;
    prm.span = p.span, prm.slots = p.slots, prm.eps = eps;
    s = with_type_and_size(dt, D, [&](auto t, auto d) {
        return launch_norm<decltype(t), decltype(d)::value, true>(prm, p, gate != nullptr, act,
                                                                  st);
    });
    if (s != LA_OK) return s;
    const int C = int(H * D);
    la::LaunchScope scope("norm_sum", st);
    la::norm_sum_kernel<<<dim3(unsigned((C + 31) / 32), 2), 512, 0, st>>>(prm.part, dweight, dbias,
                                                                         p.blocks, C);
    return launch_status();
}

}  // extern "C"
