// decode_fp8.cu -- decode attention over the 8-bit paged cache (bdfp8.h), to the
// whole context or through a sliding window with visible first tokens.
//
// The mathematics.  With codes k', v' and block scales a_t (keys), c_t (values),
// out = sum_t p_t c_t v'_t / sum_t p_t, p_t = exp(sm_scale a_t q.k'_t - m).  The
// tensor cores multiply 8-bit floats, so the cache's bytes are MMA operands as they
// stand and only the two small factors are split to fit:
//  - q = (q1 + q2 / 16) / 2^s: two E4M3 terms.  A bf16 element has 8 significant
//    bits, an E4M3 term 4, and the rest after rounding to 4 bits fits 4 bits: exact
//    for elements down to 2^-13 of the row's largest.
//  - p c = (P1 + P2 + P3) 2^(m-11): three E5M2 terms, cut from an fp16 one after another
//    (e5m2_terms: relative error 2^-9, which is bf16's own on average), with a floor at
//    2^-28 of the row's largest p c, so a sink with a hundred thousand faint tokens behind it
//    keeps their mass.  (E4M3 terms would be finer, 2^-12, but end at 2^-22.)  2^m bounds
//    the row's p c so far (decode_fp8.cuh).
// The terms are stacked as columns of one MMA (N = 2 rows of q, 3 rows of P), S^T =
// K q^T with M = 128 tokens and O^T = V^T P^T with M = 128 channels.
//
// One CTA per (sequence, KV head, split), for up to 16 stacked query rows, the G
// T_q (token, head) rows of the KV head (more take decode_fp8_wide.cu): eight softmax
// warps in two groups that each own half of the rows (thread = token, then thread =
// channel), a producer warp (bulk copies into a key and a value ring; keys run one
// tile ahead) and an MMA warp.
//
// Two blocks would do for the bandwidth; three of two 16 KB key and two value stages hide a
// tile's chain (900 to 1000 ns alone: logits, maximum over four warps, probabilities,
// value product) behind one another's.  Measured at 32 / 8 heads: 16 x 32768 tokens 168 us
// (6410 GB/s; 154 to 159 as graph replays, above the copy rate of 6545, which writes
// half), 64 ragged contexts of 8 to 131 thousand (32 / 4 heads) 577 to 606, 1024 tokens of
// one sequence 5.9.  A tile fed from L2 takes an SM 381, 449 and 580 ns at 4, 8 and 16 rows,
// memory 741 at d = 128 and 371 at d = 64: so d = 64 is bound by the softmax's instructions, and
// 16 rows at d = 128 (16 sequences of 20 to 33 thousand tokens 176 us, 157 to 165 as graph
// replays, 125 at the copy rate) by how well two blocks an SM and 256 uneven blocks in
// 296 places keep the memory busy.
//
// A row group's tiles are those of the first `sinks` tokens and those from its oldest
// window token on, numbered one after another and cut into splits, so a window
// costs what it shows, wherever it stands.

#include <algorithm>
#include <climits>

#include "decode_fp8.cuh"

namespace bdfp4 {
namespace fp8 {

// Each row's maximum (or sum) over the warp, x[g] of the lanes for row g: lane l gets row l % HG's.  Lanes trade
// rows, half of what they hold in each step, until each holds one (four rows: six shuffles; a redux.sync for each
// row took 340 cycles a tile).
template <int HG, bool SUM>
__device__ __forceinline__ float rows_reduce(const float (&x)[HG], int lane) {
    constexpr uint32_t all = 0xffffffffu;
    auto join = [](float a, float b) { return SUM ? a + b : fmaxf(a, b); };
    float r[HG];
#pragma unroll
    for (int g = 0; g < HG; ++g) r[g] = x[g];
#pragma unroll
    for (int d = 1, n = HG / 2; d < HG; d *= 2, n /= 2) {   // n rows left: those with bit d of the lane
        const bool odd = lane & d;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = odd ? r[2 * i + 1] : r[2 * i], give = odd ? r[2 * i] : r[2 * i + 1];
            r[i] = join(keep, __shfl_xor_sync(all, give, d));
        }
    }
#pragma unroll
    for (int d = HG; d < 32; d *= 2) r[0] = join(r[0], __shfl_xor_sync(all, r[0], d));
    return r[0];
}

template <int FMT, int D, int ROWS, bool MT>
struct Cfg {
    static constexpr int NQ = 2 * ROWS < 16 ? 16 : 2 * ROWS;      // N of QK: q1 and q2 columns
    static constexpr int NP = (3 * ROWS + 15) / 16 * 16;          // N of PV: three probability terms
    static constexpr int KS = D / 32;                             // MMA K steps of QK
    static constexpr int NSG = 2;                                 // softmax groups of four warps
    static constexpr int HG = ROWS / NSG;                         // rows per group
    static constexpr int NSW = 4 * NSG;
    static constexpr int PRODUCER = NSW, MMA_WARP = NSW + 1;
    static constexpr int THREADS = 32 * (NSW + 2);
    // Up to eight rows an SM holds three blocks of two 16 KB key and two value stages (192 KB in flight).
    static constexpr int CTAS = ROWS == 16 ? 2 : 3;
    static constexpr int NSK = ROWS == 16 ? 3 : 2, NSV = 2;
    static constexpr int NSC = ROWS == 16 ? 8 : 4;                  // scale slots (at least NSK + 2, see the producer)
    // P: [token/16][row][16 tokens] with chunks an odd multiple of 64 bytes apart, so that a warp's byte
    // stores (32 tokens of a row, two chunks) meet no bank twice.  MMA rows behind 3 ROWS read on into
    // what follows; their columns are not used.
    static constexpr int P_CHUNK = (3 * ROWS * 16) % 128 == 64 ? 3 * ROWS * 16 : 3 * ROWS * 16 + 64;
    static_assert(P_CHUNK % 128 == 64, "bank spread");
    static constexpr int PAGE = kPageSlots * D;
    static constexpr int TILE = 2 * PAGE;
    static constexpr int P_BUF = 8 * P_CHUNK;
    static constexpr int SM_K = 0;
    static constexpr int SM_V = SM_K + NSK * TILE;
    // D = 64: the value MMA's M = 128 rows run 4 KB past a page, into the bytes that follow the
    // ring; those products land in TMEM lanes that nothing reads
    static constexpr int SM_P = SM_V + NSV * TILE;
    static constexpr int SM_Q = SM_P + 2 * P_BUF;
    static constexpr int SM_SC = SM_Q + NQ * D;                                // [NSC][2 pages][8] scales
    static constexpr int SM_RED = SM_SC + NSC * 2 * kScalePage * 4;           // [2][4][ROWS] a quadrant's maxima
    static constexpr int SM_VM = (SM_RED + 2 * 4 * ROWS * 4 + 15) / 16 * 16;   // [2][NSG][4] masks of visible tokens
    static constexpr int SM_LSC = SM_VM + 2 * NSG * 16;                       // [ROWS] logit factors
    static constexpr int SM_ROWS = SM_LSC + ROWS * 4;                         // [ROWS] their rows in the output
    static constexpr int SM_POK = SM_ROWS + ROWS * 4;                         // [NSC] page flags
    static constexpr int SM_BARS = (SM_POK + NSC * 4 + 7) / 8 * 8;
    static constexpr int NBARS = 2 * NSK + 2 * NSV + 7;
    static constexpr int SM_MISC = SM_BARS + NBARS * 8;
    static constexpr int SMEM = SM_MISC + 16;
    static_assert(2 * P_BUF + NQ * D >= 4096, "the value MMA's overrun at D = 64 stays inside the block's memory");
    static_assert((NP - 3 * ROWS) * 16 <= NQ * D, "P's overrun too");
    static_assert(SMEM <= 233472 / CTAS - 1024, "shared memory");
    static_assert(NSC >= NSK + 2, "scale slots");
    static constexpr int T_S = 0;                                 // TMEM columns: S^T double buffer, O^T
    static constexpr int T_O = 2 * NQ;
    static constexpr int T_USED = T_O + NP;
    static constexpr int T_ALLOC = ROWS == 16 ? 128 : 64;
    static_assert(T_USED <= T_ALLOC && T_ALLOC * CTAS <= 512, "tensor memory");
    static_assert(ROWS == 4 || ROWS == 8 || ROWS == 16, "more rows take the wide kernel");
};

constexpr int kMaxCluster = 8;   // blocks of a cluster, the portable limit

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// HOOK: the unwind test's instantiation (bdfp8_debug.h).
template <int FMT, int D, int ROWS, bool MT, bool HOOK>
__global__ void __launch_bounds__(Cfg<FMT, D, ROWS, MT>::THREADS, Cfg<FMT, D, ROWS, MT>::CTAS)
    decode_fp8_kernel(const Args a) {
    using C = Cfg<FMT, D, ROWS, MT>;
    const long long wlim = HOOK ? a.wait_limit : kWaitLimit;
    constexpr int HG = C::HG;
    follow_grid();
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* const p_op = smem + C::SM_P;
    uint8_t* const q_op = smem + C::SM_Q;
    float* const sc_ring = reinterpret_cast<float*>(smem + C::SM_SC);
    float* const red = reinterpret_cast<float*>(smem + C::SM_RED);
    uint32_t* const vmask = reinterpret_cast<uint32_t*>(smem + C::SM_VM);
    float* const lsc = reinterpret_cast<float*>(smem + C::SM_LSC);
    int* const rows = reinterpret_cast<int*>(smem + C::SM_ROWS);
    int* const pok = reinterpret_cast<int*>(smem + C::SM_POK);
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + C::SM_BARS);
    uint64_t* const kfull = bars;
    uint64_t* const kempty = kfull + C::NSK;
    uint64_t* const vfull = kempty + C::NSK;
    uint64_t* const vempty = vfull + C::NSV;
    uint64_t* const s_full = vempty + C::NSV;   // [2] QK done, and the tile's scales seen -> softmax
    uint64_t* const p_ready = s_full + 2;       // [2] P written, dead value columns zeroed -> MMA
    uint64_t* const o_full = p_ready + 2;       // [2] PV done -> softmax
    uint64_t* const q_ready = o_full + 2;
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SM_MISC);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + C::SM_MISC + 4);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Place at = place_of(a);
    const int b = at.b, hk = at.hk, split = at.split;   // one row group
    const int nrows = a.G * a.T_q;
    // row of the [B][T_q][H_q] arrays of stacked row r
    auto row_of = [&](int r) -> int {
        if constexpr (!MT) return b * a.H_q + hk * a.G + r;
        return (b * a.T_q + r / a.G) * a.H_q + hk * a.G + r % a.G;
    };
    // what does not depend on the sequence's length is loaded while that is on its way
    int early[2] = {-1, -1};
    float qx[ROWS > C::NSW ? ROWS / C::NSW : 1][D / 32];
    if (warp == C::PRODUCER) early_pages(a, at, lane, early);
    else if (warp < C::NSW)
#pragma unroll
        for (int i = 0; i * C::NSW < ROWS; ++i) {
            const int r = warp + i * C::NSW;
            load_query<D>(r < nrows ? a.q + (int64_t)row_of(r) * D : nullptr, lane, qx[i]);
        }

    const int N = checked_len(a, b);
    const Tiles tl = tiles_of(N, a.T_q, a.G, 0, nrows - 1, a.window, a.sinks);
    const int nspl = splits_of(tl, a.chunk_tiles);
    if (tid == 0 && split == 0 && hk == 0 && (N != a.seq_lens[b] || (N > 0 && N < a.T_q)))
        set_status(a.dev_status, BDFP4_DEV_BAD_SEQLEN);
    if (split > 0 && split >= nspl) return;
    if (tl.total == 0) {
        for (int i = tid; i < nrows * D; i += C::THREADS) a.out[(int64_t)row_of(i / D) * D + i % D] = __float2bfloat16(0.0f);
        return;
    }
    const int tile0 = split * a.chunk_tiles;
    const int n = min(a.chunk_tiles, tl.total - tile0);   // tiles of this split (>= 1)

    if (tid == 0) {
        for (int s = 0; s < C::NSK; ++s) {
            tc::mbar_init(&kfull[s], 1);
            tc::mbar_init(&kempty[s], 1);
        }
        for (int s = 0; s < C::NSV; ++s) {
            tc::mbar_init(&vfull[s], 1);
            tc::mbar_init(&vempty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&s_full[i], 2);   // the MMAs' commit, and the MMA lane itself
            tc::mbar_init(&p_ready[i], C::NSW);
            tc::mbar_init(&o_full[i], 1);
        }
        tc::mbar_init(q_ready, C::NSW);
        *abort_flag = 0;
        tc::fence_mbar_init();
    }
    if (warp == C::MMA_WARP) {
        tc::tmem_alloc(tmem_slot, C::T_ALLOC);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tbase = *tmem_slot;

    if (warp == C::PRODUCER) {
        produce<C, HOOK>(a, tl, tile0, n, b, hk, lane, smem, sc_ring, pok, kfull, kempty, vfull, vempty, abort_flag, early);
    } else if (warp == C::MMA_WARP) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc_qk = idesc_f8(Fmt8<FMT>::mma, Fmt8<BDFP8_E4M3>::mma, C::NQ);
            constexpr uint32_t idesc_pv = idesc_f8(Fmt8<FMT>::mma, Fmt8<BDFP8_E5M2>::mma, C::NP);
            // keys and queries: 8-row groups 8 D bytes apart, 16-element chunks 128 bytes apart; values: 8-channel
            // groups 512 bytes apart, 16-slot chunks 128; P: 8-row groups 128 bytes apart, chunks P_CHUNK
            constexpr uint32_t qk_hi = desc_hi(8 * D), v_hi = desc_hi(512), p_hi = desc_hi(128);
            const uint32_t q_lo = desc_lo(tc::smem_u32(q_op), 128);
            const uint32_t p_lo = desc_lo(tc::smem_u32(p_op), C::P_CHUNK);
            const uint32_t k_lo = desc_lo(tc::smem_u32(smem + C::SM_K), 128);
            const uint32_t v_lo = desc_lo(tc::smem_u32(smem + C::SM_V), 128);
            // the last commit: its phase completes once every tcgen05 operation issued before it has
            uint64_t* last_bar = nullptr;
            uint32_t last_par = 0;
            auto issue_qk = [&](int j) -> bool {
                const int s = j % C::NSK, buf = j & 1;
                if (!tc::mbar_wait(&kfull[s], (j / C::NSK) & 1, abort_flag, wlim)) return false;
                tc::tc_fence_after();
                const uint32_t kt = k_lo + s * (C::TILE / 16), d = tbase + C::T_S + buf * C::NQ;
                mma_f8<false>(d, kt, qk_hi, q_lo, qk_hi, idesc_qk);
#pragma unroll
                for (int ks = 1; ks < C::KS; ++ks) mma_f8<true>(d, kt + ks * 16, qk_hi, q_lo + ks * 16, qk_hi, idesc_qk);
                tc::mma_commit(&s_full[buf]);
                tc::mma_commit(&kempty[s]);
                // passes on this thread's view of the copied scales and the page flags
                tc::mbar_arrive(&s_full[buf]);
                last_bar = &kempty[s];
                last_par = (uint32_t)(j / C::NSK) & 1u;
                return true;
            };
            bool ok = tc::mbar_wait(q_ready, 0, abort_flag, wlim);
            if (ok) tc::tc_fence_after();
            ok = ok && issue_qk(0);
            for (int j = 0; ok && j < n; ++j) {
                if (j + 1 < n && !(ok = issue_qk(j + 1))) break;
                const int s = j % C::NSV, buf = j & 1;
                if (!(ok = tc::mbar_wait(&p_ready[buf], (j >> 1) & 1, abort_flag, wlim))) break;
                if (!(ok = tc::mbar_wait(&vfull[s], (j / C::NSV) & 1, abort_flag, wlim))) break;
                tc::tc_fence_after();
                const uint32_t vt = v_lo + s * (C::TILE / 16), pt = p_lo + buf * (C::P_BUF / 16), d = tbase + C::T_O;
                // O^T accumulates over the split's tiles (the softmax warps rescale it)
                if (j > 0) mma_f8<true>(d, vt, v_hi, pt, p_hi, idesc_pv);
                else mma_f8<false>(d, vt, v_hi, pt, p_hi, idesc_pv);
#pragma unroll
                for (int ks = 1; ks < 4; ++ks)
                    mma_f8<true>(d, vt + (ks >> 1) * (C::PAGE / 16) + (ks & 1) * 16, v_hi, pt + ks * 2 * (C::P_CHUNK / 16), p_hi,
                                 idesc_pv);
                tc::mma_commit(&o_full[buf]);
                tc::mma_commit(&vempty[s]);
                last_bar = &vempty[s];
                last_par = (uint32_t)(j / C::NSV) & 1u;
            }
            if (!ok) {
                *abort_flag = 1;
                // the tensor memory is freed below: the MMAs into it must have finished
                if (last_bar) tc::mbar_wait_drain(last_bar, last_par, wlim);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax warps
        const int grp = warp >> 2;
        const int qd = warp & 3;                   // TMEM lane quadrant: tokens 32 qd .. 32 qd + 31 of a tile
        const int gb = grp * HG;                   // first row of the group
        const int bar_id = 1 + grp;
        const uint32_t tq = tbase + ((uint32_t)(32 * qd) << 16);
        bool bad = false, grp_abort = false;

        // query rows as two E4M3 terms: q 2^(7-e) in [128, 256) for the row's largest, the rest times 16
#pragma unroll
        for (int i = 0; i * C::NSW < ROWS; ++i) {
            const int r = warp + i * C::NSW;
            if (r >= ROWS) break;
            uint32_t c1w, c2w;
            const float f = split_query<D, 4>(qx[i], a.sm_scale, c1w, c2w);
            const int col = 2 * HG * (r / HG) + r % HG;   // a group's q1 columns, then its q2 columns
            put_query<D>(q_op, col, lane, c1w);
            put_query<D>(q_op, col + HG, lane, c2w);
            if (lane == 0) {
                lsc[r] = f;
                rows[r] = row_of(r);
            }
        }
        tc::fence_proxy_async_smem();
        tc::named_bar_sync(1 + C::NSG, 32 * C::NSW);
        if (lane == 0) tc::mbar_arrive(q_ready);

        // The reference of row gb + hl lives in lanes hl, hl + HG, ... of the group's warps; the warp takes a new one
        // by shuffle.
        const int hl = lane % HG;
        float m_l = -INFINITY;
        float l_part[HG], mz[HG];   // mz: the references (0 where there is none yet) less kLift
#pragma unroll
        for (int g = 0; g < HG; ++g) {
            l_part[g] = 0.0f;
            mz[g] = -(float)kLift;
        }
        const int pg = qd >> 1;                                // page of this thread's token in the tile
        const int blk = 2 * (qd & 1) + (lane >> 4);            // its scale block in the page
        const int tok = 32 * qd + lane;
        const int chan = tok;                                  // O^T lane = value channel
        uint8_t* const pslot = p_op + (tok >> 4) * C::P_CHUNK + 3 * gb * 16 + (tok & 15);
        float lr[HG];
#pragma unroll
        for (int g = 0; g < HG; ++g) lr[g] = lsc[gb + g];
        const uint32_t t_o = tq + C::T_O + 3 * gb;             // a group's first, second and third terms

        // tiles all of whose tokens all rows see need no masks
        const int all_end = N - a.T_q + 1, all_lo = a.window > 0 ? N - a.window : 0;

        // One tile's logits to probabilities; FULL: every row sees every token of it.  False: a warp of the group gave up.
        auto tile = [&](auto full_c, int j, int t0, int good) -> bool {
            constexpr bool full = decltype(full_c)::value;
            const int buf = j & 1;
            uint32_t s12[2 * HG];
            tc::tmem_ld<2 * HG>(tq + C::T_S + buf * C::NQ + 2 * gb, s12);
            const float* sc = sc_ring + ((j % C::NSC) * 2 + pg) * kScalePage + blk;
            const float ka = sc[0];
            float va = sc[kBlocksPerPage];
            const int t = t0 + tok;
            const bool valid = full || (t < tl.end && (t >= tl.lo || t < a.sinks) && ((good >> pg) & 1));
            // several query tokens: row r sees t iff r / G >= t - (N - T_q) and, in a window, r / G < t + W - (N - T_q)
            // or t < sinks: rows [vis0, vis1) of the group
            [[maybe_unused]] int vis0 = 0, vis1 = HG;
            if constexpr (MT && !full) {
                const int d = t - (N - a.T_q);
                vis0 = min(max(d, 0), a.T_q) * a.G - gb;
                if (a.window > 0 && t >= a.sinks) vis1 = min(max(d + a.window, 0), a.T_q) * a.G - gb;
            }
            const uint32_t seen = full ? 0xffffffffu : __ballot_sync(0xffffffffu, valid);   // the warp's visible tokens
            float ve, v_down;
            scale_parts(va, ve, v_down);
            tc::tmem_wait_ld();
            float x[HG];   // x + e
#pragma unroll
            for (int g = 0; g < HG; ++g) {
                const float s = fmaf(fmaf(__uint_as_float(s12[HG + g]), 0.0625f, __uint_as_float(s12[g])), ka * lr[g], ve);
                const bool see = full || (valid && (!MT || (g >= vis0 && g < vis1)));
                x[g] = see ? s : -INFINITY;
            }
            float wm_l = rows_reduce<HG, false>(x, lane);   // row hl's maximum over the warp's tokens
            // blocks of zeros (see kZeroScale): each half of the warp looks at its tokens' block
            if (__any_sync(0xffffffffu, valid && va == kZeroScale) && __any_sync(0xffffffffu, wm_l > m_l + kRise)) {
                const int s = j % C::NSV;
                if (!tc::mbar_wait(&vfull[s], (j / C::NSV) & 1, abort_flag, wlim)) bad = true;
                const uint8_t* const vb = smem + C::SM_V + s * C::TILE + pg * C::PAGE + blk * 128;
                bool some = false;
#pragma unroll 1
                for (int c = lane & 15; c < D; c += 16)
                    some |= any_value(*reinterpret_cast<const uint4*>(vb + (c >> 3) * 512 + (c & 7) * 16), seen >> (lane & 16));
                some = (__ballot_sync(0xffffffffu, some) >> (lane & 16)) & 0xffffu;
                if (va == kZeroScale && !some) {
                    const float one = ve;
                    va = 0.0f;
                    scale_parts(va, ve, v_down);
#pragma unroll
                    for (int g = 0; g < HG; ++g) x[g] += ve - one;
                }
                wm_l = rows_reduce<HG, false>(x, lane);
            }
            float* const rw = red + (buf * 4 + qd) * ROWS;
            if (lane < HG) rw[gb + lane] = wm_l;
            if constexpr (!full) {
                if (lane == 0) vmask[(buf * C::NSG + grp) * 4 + qd] = seen;
            }
            // one decision for the group's four warps, taken by the barrier itself
            if (tc::named_bar_or(bar_id, 128, bad)) return false;
            const float* const rr = red + buf * 4 * ROWS;
            const float mt = fmaxf(fmaxf(rr[gb + hl], rr[ROWS + gb + hl]),
                                   fmaxf(rr[2 * ROWS + gb + hl], rr[3 * ROWS + gb + hl]));
            const bool rise = mt > m_l + kRise;
            const bool rose = __any_sync(0xffffffffu, rise);
            float corr_l = 1.0f;
            if (rose) {
                corr_l = rise ? ex2_down(m_l - mt) : 1.0f;   // 0 before the first visible token
                m_l = rise ? mt : m_l;
#pragma unroll
                for (int g = 0; g < HG; ++g) {
                    l_part[g] *= __shfl_sync(0xffffffffu, corr_l, g);
                    const float m = __shfl_sync(0xffffffffu, m_l, g);
                    mz[g] = (m == -INFINITY ? 0.0f : m) - (float)kLift;
                }
            }
            // r in units of 2^-kTopExp; nothing of a token that no row sees goes in
            const float vy = valid ? va * v_down * (float)(1 << kTopExp) : 0.0f;
            uint8_t* const pb = pslot + buf * C::P_BUF;
#pragma unroll
            for (int g = 0; g < HG; g += 2) {
                const float p0 = tc::ex2_approx(x[g] - mz[g]);
                const float p1 = tc::ex2_approx(x[g + 1] - mz[g + 1]);
                l_part[g] = fmaf(p0, v_down, l_part[g]);
                l_part[g + 1] = fmaf(p1, v_down, l_part[g + 1]);
                float y0 = p0 * vy, y1 = p1 * vy;
                if constexpr (MT && !full) {   // a token that another row sees, with a scale that is no number
                    y0 = x[g] == -INFINITY ? 0.0f : y0;
                    y1 = x[g + 1] == -INFINITY ? 0.0f : y1;
                }
                uint32_t c[3];
                e5m2_terms(__floats2half2_rn(y0, y1), c);
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    pb[(k * HG + g) * 16] = (uint8_t)(c[k] >> 8);
                    pb[(k * HG + g + 1) * 16] = (uint8_t)(c[k] >> 24);
                }
            }
            // O^T of the group's rows moves to the new reference once the previous
            // tile's PV has completed, before this tile's PV is issued
            if (j > 0 && rose) {
                if (!tc::mbar_wait(&o_full[(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag, wlim)) bad = true;
                tc::tc_fence_after();
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    uint32_t ov[HG];
                    tc::tmem_ld<HG>(t_o + k * HG, ov);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int g = 0; g < HG; ++g)
                        ov[g] = __float_as_uint(__uint_as_float(ov[g]) * __shfl_sync(0xffffffffu, corr_l, g));
                    tc::tmem_st_n<HG>(t_o + k * HG, ov);
                }
                tc::tmem_wait_st();
            }
            // Value columns of tokens that no row sees are zeroed: their bytes may be anything (a NaN code
            // among them), and 0 times NaN is NaN.  One channel per thread of group 0.
            if (!full && grp == 0) {
                const uint4 vm = *reinterpret_cast<const uint4*>(vmask + (buf * C::NSG + grp) * 4);
                const int s = j % C::NSV;
                if (!tc::mbar_wait(&vfull[s], (j / C::NSV) & 1, abort_flag, wlim)) bad = true;
                const uint32_t w[4] = {vm.x, vm.y, vm.z, vm.w};
                if (chan < D) {
                    uint8_t* const vc = smem + C::SM_V + s * C::TILE + (chan >> 3) * 512 + (chan & 7) * 16;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const uint32_t m = (w[c >> 1] >> (16 * (c & 1))) & 0xffffu;
                        if (m == 0xffffu) continue;
                        uint4* const at = reinterpret_cast<uint4*>(vc + (c >> 2) * C::PAGE + (c & 3) * 128);
                        uint4 v = *at;
                        v.x &= byte_mask(m);
                        v.y &= byte_mask(m >> 4);
                        v.z &= byte_mask(m >> 8);
                        v.w &= byte_mask(m >> 12);
                        *at = v;
                    }
                }
            }
            tc::tc_fence_before();
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&p_ready[buf]);
            return true;
        };

        for (int j = 0; j < n; ++j) {
            const int t0 = tl.tile(tile0 + j) * kTileTokens;
            if (!tc::mbar_wait(&s_full[j & 1], (j >> 1) & 1, abort_flag, wlim)) bad = true;
            if (HOOK && a.stall == kStallWarp && j == 0 && warp == 0) bad = true;
            tc::tc_fence_after();
            const int good = pok[j % C::NSC];
            if (good == 3 && t0 + kTileTokens <= all_end && (t0 >= all_lo || t0 + kTileTokens <= a.sinks))
                grp_abort = !tile(std::true_type{}, j, t0, good);
            else
                grp_abort = !tile(std::false_type{}, j, t0, good);
            if (grp_abort) break;
        }
        // ------------------------------------------------------------ epilogue (thread = channel)
        uint32_t o1[HG], o2[HG], o3[HG];
        if (!grp_abort) {
            if (!tc::mbar_wait(&o_full[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag, wlim)) bad = true;
            tc::tc_fence_after();
            tc::tmem_ld<HG>(t_o, o1);
            tc::tmem_ld<HG>(t_o + HG, o2);
            tc::tmem_ld<HG>(t_o + 2 * HG, o3);
            tc::tmem_wait_ld();
        }
        grp_abort = tc::named_bar_or(bar_id, 128, grp_abort || bad || *abort_flag);
        if (grp_abort) *abort_flag = 1;
        if (!grp_abort) {
            float* const rl = red;   // [4][RED_Q] partial sums (the maxima are no longer read)
            const float l_l = rows_reduce<HG, true>(l_part, lane);
            if (lane < HG) rl[qd * ROWS + gb + lane] = l_l;
            tc::named_bar_sync(bar_id, 128);
            const float unit = pow2i(-kTopExp);
#pragma unroll
            for (int g = 0; g < HG; ++g) {
                const int r = gb + g;
                const float m_g = __shfl_sync(0xffffffffu, m_l, g);
                if (r >= nrows || chan >= D) continue;
                const float l = (rl[r] + rl[ROWS + r]) + (rl[2 * ROWS + r] + rl[3 * ROWS + r]);
                const float o = ((__uint_as_float(o3[g]) + __uint_as_float(o2[g])) + __uint_as_float(o1[g])) * unit;
                const int64_t row = rows[r];
                if (nspl == 1) {
                    a.out[row * D + chan] = __float2bfloat16(l == 0.0f ? 0.0f : o / l);
                } else {
                    a.ws_o[(row * a.max_splits + split) * D + chan] = o;
                    if (chan == 0) reinterpret_cast<float2*>(a.ws_ml)[row * a.max_splits + split] = make_float2(m_g, l);
                }
            }
        }
    }

    tc::tc_fence_before();
    __syncthreads();
    if (*abort_flag && tid == 0) set_status(a.dev_status, BDFP4_DEV_TIMEOUT);
    if (warp == C::MMA_WARP) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tbase, C::T_ALLOC);
    }
    // Splits that are a cluster merge here: behind its barrier each takes a share of the outputs (blocks without a
    // tile have left; they do not count at the barrier).  The partial sums pass through the workspace, which asks for
    // one barrier; through each other's shared memory it would be two (1400 cycles each).
    if (a.cluster && nspl > 1) {
        cluster_sync();
        for (int i = split * C::THREADS + tid; i < nrows * D; i += nspl * C::THREADS) {
            const int64_t row = rows[i / D], at0 = row * a.max_splits;
            float2 ml[kMaxCluster];
            float o[kMaxCluster], M = -INFINITY;
#pragma unroll
            for (int s = 0; s < kMaxCluster; ++s) {
                ml[s] = make_float2(-INFINITY, 0.0f);
                o[s] = 0.0f;
                if (s < nspl) {
                    ml[s] = __ldcg(reinterpret_cast<const float2*>(a.ws_ml) + at0 + s);
                    o[s] = __ldcg(a.ws_o + (at0 + s) * D + i % D);
                }
            }
#pragma unroll
            for (int s = 0; s < kMaxCluster; ++s) M = fmaxf(M, ml[s].x);
            if (M == -INFINITY) M = 0.0f;
            float L = 0.0f, acc = 0.0f;
#pragma unroll
            for (int s = 0; s < kMaxCluster; ++s) {
                const float w = ex2_down(ml[s].x - M);
                L = fmaf(ml[s].y, w, L);
                acc = fmaf(o[s], w, acc);
            }
            a.out[row * D + i % D] = __float2bfloat16(L == 0.0f ? 0.0f : acc * (1.0f / L));
        }
    }
}

// Log-sum-exp merge of the splits, WARPS warps per output row (64 or 128 channels):
//   out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,  M = max_s m_s.
// A split whose tokens a row does not see has m = -inf, l = 0 and weight 0; a NaN among the
// sums reaches the output.  The warps of a row take every WARPS-th split and join their sums in shared memory in
// the order of the warps.  What bounds it is the latency of a warp's chain of splits (0.36 us each with one warp a
// row), so a row gets a block while all rows' blocks run at once; with more rows the grid has warps enough, and the
// joining only costs.  Measured, decode and merge, us, a warp against a block per row: 32 rows, 131072 tokens in 32
// splits 55.3 / 47.9, 8 rows in 64 splits 34.6 / 22.0; 512 rows in 8 splits 24.8 / 24.0; 2048 rows in 2 splits 53.7 /
// 56.8, 8192 rows in 2 splits 71.4 / 87.3.
constexpr int kMergeThreads = 256, kMergeBlocks = 2048 / kMergeThreads;   // blocks that an SM holds at once

template <int D, int WARPS>
__global__ void __launch_bounds__(kMergeThreads) merge_fp8_kernel(const Args a, int rows_per_cta) {
    follow_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned row32 = WARPS == 1 ? blockIdx.x * (kMergeThreads / 32) + warp : blockIdx.x;
    if (row32 >= (unsigned)(a.B * a.T_q * a.H_q)) return;
    const int64_t row = row32;
    const unsigned bt = row32 / (unsigned)a.H_q;
    const int h = row32 % (unsigned)a.H_q, b = bt / (unsigned)a.T_q, i = bt % (unsigned)a.T_q;
    const int r = i * a.G + h % a.G, r0 = r / rows_per_cta * rows_per_cta;
    const Tiles tl = tiles_of(checked_len(a, b), a.T_q, a.G, r0, min(r0 + rows_per_cta, a.G * a.T_q) - 1, a.window, a.sinks);
    const int ns = splits_of(tl, a.chunk_tiles);
    if (ns <= 1) return;   // written by the decode kernel
    const float2* ml = reinterpret_cast<const float2*>(a.ws_ml) + row * a.max_splits;
    float M = -INFINITY;
    for (int s = lane; s < ns; s += 32) M = fmaxf(M, ml[s].x);
    M = tc::redux_max_f32(M, 0xffffffffu);
    if (M == -INFINITY) M = 0.0f;
    constexpr int E = D / 32;
    float acc[E], L = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    const float* o = a.ws_o + row * a.max_splits * D + lane * E;
#pragma unroll 8
    for (int s = WARPS == 1 ? 0 : warp; s < ns; s += WARPS) {
        const float2 w2 = ml[s];
        const float w = exp2f(w2.x - M);
        L = fmaf(w2.y, w, L);
        float v[E];
        if constexpr (E == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(o + (int64_t)s * D);
        else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(o + (int64_t)s * D);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(v[e], w, acc[e]);
    }
    if constexpr (WARPS > 1) {
        __shared__ float part[WARPS][D], part_l[WARPS];
#pragma unroll
        for (int e = 0; e < E; ++e) part[warp][lane * E + e] = acc[e];
        if (lane == 0) part_l[warp] = L;
        __syncthreads();
        if (warp) return;
#pragma unroll
        for (int w = 1; w < WARPS; ++w) {
            L += part_l[w];
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += part[w][lane * E + e];
        }
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(a.out + row * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
}

// ------------------------------------------------------------------ host
inline int rows_for(int G, int64_t T_q) {
    const int64_t rows = G * T_q;
    return rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 ? 16 : kWideRows;
}
inline int ctas_per_sm(int rows) { return rows <= 8 ? 3 : rows == 16 ? 2 : 1; }

// Most tiles that a row group of a sequence of at most N tokens can see.
inline int64_t most_tiles(int64_t N, int T_q, int G, int rows, int window, int sinks) {
    const int64_t all = (N + kTileTokens - 1) / kTileTokens;
    if (window <= 0) return all;
    // the group's query tokens: their windows span window + span - 1 tokens from any slot on
    const int64_t span = std::min<int64_t>(T_q, (rows - 1) / G + 2);
    const int64_t win = (window + span - 1 + kTileTokens - 2) / kTileTokens + 1;
    return std::min(all, win + ((int64_t)sinks + kTileTokens - 1) / kTileTokens);
}

template <int D>
static int launch_merge8(const Args& a, int rows_per_cta, cudaStream_t st) {
    if (a.max_splits <= 1) return BDFP4_OK;
    const int64_t rows = (int64_t)a.B * a.T_q * a.H_q;
    constexpr int kWarps = kMergeThreads / 32;
    const cudaError_t e =
        a.merge_rows ? launch_following(merge_fp8_kernel<D, 1>, (unsigned)((rows + kWarps - 1) / kWarps), kMergeThreads, 0, 1, st,
                                        a, rows_per_cta)
                     : launch_following(merge_fp8_kernel<D, kWarps>, (unsigned)rows, kMergeThreads, 0, 1, st, a, rows_per_cta);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return BDFP4_ERR_CUDA;
    }
    return launch_status();
}

template <int FMT, int D, int ROWS, bool MT, bool HOOK = false>
static int launch(const Args& a, int64_t ctas, cudaStream_t st) {
    using C = Cfg<FMT, D, ROWS, MT>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(decode_fp8_kernel<FMT, D, ROWS, MT, HOOK>, C::SMEM, done);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return BDFP4_ERR_CUDA;
    }
    e = launch_following(decode_fp8_kernel<FMT, D, ROWS, MT, HOOK>, (unsigned)ctas, C::THREADS, C::SMEM,
                         a.cluster ? (unsigned)a.max_splits : 1u, st, a);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return BDFP4_ERR_CUDA;
    }
    const int rc = launch_status();
    if (a.cluster) return rc;
    return rc != BDFP4_OK ? rc : launch_merge8<D>(a, ROWS, st);
}

template <int FMT, int D>
static int dispatch(const Args& a, int rows, int64_t ctas, cudaStream_t st) {
    if (a.wait_limit != kWaitLimit || a.stall) {   // bdfp8_debug_decode_wait_test: E4M3, d = 128
        if constexpr (FMT != BDFP8_E4M3 || D != 128) return BDFP4_ERR_UNSUPPORTED;
        else if (rows == 8 && a.T_q == 1) return launch<FMT, D, 8, false, true>(a, ctas, st);
        else if (rows != kWideRows) return BDFP4_ERR_UNSUPPORTED;
    }
    if (rows == kWideRows) {
        const int rc = launch_wide(a, FMT, D, ctas, st);
        return rc != BDFP4_OK ? rc : launch_merge8<D>(a, kWideRows, st);
    }
    if (a.T_q > 1)
        return rows == 4   ? launch<FMT, D, 4, true>(a, ctas, st)
               : rows == 8 ? launch<FMT, D, 8, true>(a, ctas, st)
                           : launch<FMT, D, 16, true>(a, ctas, st);
    return rows == 4   ? launch<FMT, D, 4, false>(a, ctas, st)
           : rows == 8 ? launch<FMT, D, 8, false>(a, ctas, st)
                       : launch<FMT, D, 16, false>(a, ctas, st);
}

// What every entry point asks of the shape.
static int check_shape(int B, int T_q, int H_q, int H_kv, int d, int window, int sinks) {
    if (B < 0 || T_q <= 0 || H_q <= 0 || H_kv <= 0 || window < 0 || sinks < 0) return BDFP4_ERR_ARG;
    if (H_q % H_kv) return BDFP4_ERR_SHAPE;
    if (d != 64 && d != 128) return BDFP4_ERR_UNSUPPORTED;
    // stacked rows, and grids of at most 2^31 - 1 blocks
    if ((int64_t)T_q * (H_q / H_kv) > (1 << 24) || (int64_t)B * T_q * H_q > INT_MAX) return BDFP4_ERR_UNSUPPORTED;
    return BDFP4_OK;
}

struct Shape {
    int rows, groups, max_splits;
};

static Shape shape_of(int T_q, int H_q, int H_kv, int max_pages, int window, int sinks, int chunk) {
    Shape s;
    const int G = H_q / H_kv;
    s.rows = rows_for(G, T_q);
    s.groups = (int)(((int64_t)G * T_q + s.rows - 1) / s.rows);
    const int64_t tiles = most_tiles((int64_t)max_pages * kPageSlots, T_q, G, s.rows, window, sinks);
    s.max_splits = (int)std::max<int64_t>(1, (tiles + chunk - 1) / chunk);
    return s;
}

// Where the splits of a launch merge: in a cluster when they fit one and all blocks run at once (a cluster's blocks
// hold their SMs until the last is done, which costs nothing only then), else through the workspace.
static bool merges_in_cluster(int rows, int max_splits, int64_t ctas, int sms) {
    return rows <= 16 && max_splits > 1 && max_splits <= kMaxCluster && ctas <= (int64_t)ctas_per_sm(rows) * sms;
}

// Tiles per split.  The model, in ns: the memory gives a tile (256 D bytes at 6.5 TB/s) to one block after another,
// and a block takes at least alone[k] for a tile of its own with k + 1 blocks on its SM; the two overlap but for an
// eighth.  A grid runs in waves of ctas_per_sm blocks an SM, each with a start and an end of 2.65 us and 0.82 us for
// every further block of an SM (6.2 us where the blocks are bound by their own work); with lengths that differ the
// last blocks run on alone; more than one split adds the merge: in a cluster 1.35 us and more for each block on
// an SM and each split, else 2.8 us, 20 ns a split and the partial sums' traffic.  The constants are fitted to 957
// measured calls (1 to 128 sequences of 512 to 131072 tokens, 1 to 8 KV heads, 4 to 128 rows, windows, differing
// lengths), up to 21 splits each: the split count of least modelled time, which is the plan, takes 1% more than
// the fastest split on average and 23% at worst.  Measured, us, by tiles a split: 131072 tokens, 8 KV heads, 4 rows
// 128: 112, 64: 61, 32: 48, 16: 56; one KV head 128: 115, 64: 61, 32: 34, 16: 22; 4 x 4096 tokens 32: 30, 8: 12, 4:
// 13, 1: 19; 64 x 1000 ragged tokens 8: 22, 4: 27, 2: 35.  The block times are the fit's: 16 rows have come
// down since, and the one for 128-row groups stands for a few live rows as for all (1210 and 1480 ns a tile fed
// from L2, start left out).  tiles_of(b): the tiles that a row group of sequence
// b sees at most.
template <class TilesOf>
static int plan(int B, const TilesOf& tiles_of, int64_t items, int sms, int rows, int d) {
    static const float alone4[3] = {900, 910, 1330}, alone8[3] = {920, 1090, 1600}, alone16[2] = {980, 1060},
                       alone128[1] = {1280};
    const float* alone = rows == 4 ? alone4 : rows == 8 ? alone8 : rows == 16 ? alone16 : alone128;
    const int ctas = ctas_per_sm(rows);
    sms = std::max(1, sms);
    int64_t most = 1, all = 0;
    for (int b = 0; b < B; ++b) {
        most = std::max<int64_t>(most, tiles_of(b));
        all += tiles_of(b);
    }
    const double slots = (double)sms * ctas, tile = 256.0 * d / 6500.0, work = (double)all * items * tile;
    // more than a few waves gain nothing
    const int64_t s_max = std::min<int64_t>(most, 8 + (int64_t)(4 * slots * most / std::max<double>(1.0, (double)all * items)));
    double best_cost = -1;
    int64_t best = most, last = 0;
    for (int64_t s = 1; s <= s_max; ++s) {
        const int64_t c = (most + s - 1) / s;
        if (c == last) continue;
        last = c;
        int64_t n = 0, top = 1;
        for (int b = 0; b < B; ++b) n += (tiles_of(b) + c - 1) / c;
        n = std::max<int64_t>(1, n * items);
        top = (most + c - 1) / c;
        const auto wave = [&](double blocks) {   // blocks at once, at most `slots`
            const int k = std::min(ctas, std::max(1, (int)((blocks + sms - 1) / sms)));
            const double mem = work * blocks / n, own = c * (double)alone[k - 1];
            return std::max(mem, own) + 0.12 * std::min(mem, own) + (rows <= 8 ? 2650.0 : 6200.0) + 820.0 * (k - 1);
        };
        const int64_t full = n / (int64_t)slots, rest = n % (int64_t)slots;
        double cost = full * wave(slots) + (rest ? wave((double)rest) : 0.0);
        if (full) cost += 0.5 * (1.0 - (double)all / ((double)B * most)) * c * alone[0];
        if (top > 1)
            cost += merges_in_cluster(rows, (int)top, (int64_t)B * items * top, sms)
                        ? 1350.0 + 650.0 * std::min<double>(n, slots) / sms + 55.0 * top
                        : 2800.0 + 20.0 * top + 0.002 * n * rows * d;
        if (best_cost < 0 || cost < best_cost) {
            best_cost = cost;
            best = c;
        }
    }
    return (int)std::min<int64_t>(best, INT_MAX);
}

static int sm_count(int* sms) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return BDFP4_ERR_CUDA;
    static std::atomic<int> known[64];   // per device, as the attribute query costs about a microsecond
    if (dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return BDFP4_OK;
    if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return BDFP4_ERR_CUDA;
    if (dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
    return BDFP4_OK;
}

}  // namespace fp8
}  // namespace bdfp4

using namespace bdfp4;
using namespace bdfp4::fp8;

extern "C" int bdfp8_decode_plan(const int32_t* host_seq_lens, int B, int T_q, int H_q, int H_kv, int d, int window,
                                 int sinks, int num_sms) {
    const int rc = check_shape(B, T_q, H_q, H_kv, d, window, sinks);
    if (rc != BDFP4_OK) return rc;
    if (num_sms <= 0 || (B > 0 && !host_seq_lens)) return BDFP4_ERR_ARG;
    const Shape s = shape_of(T_q, H_q, H_kv, 1, window, sinks, 1);
    return plan(
        B,
        [&](int b) { return most_tiles(std::max(0, host_seq_lens[b]), T_q, H_q / H_kv, s.rows, window, sinks); },
        (int64_t)H_kv * s.groups, num_sms, s.rows, d);
}

static size_t partial_bytes(int64_t rows, int max_splits, int d) {
    const size_t o = (size_t)rows * max_splits * d * sizeof(float);
    return (o + 255) / 256 * 256;
}

extern "C" size_t bdfp8_decode_workspace_size(int B, int T_q, int H_q, int H_kv, int d, int max_pages_per_seq,
                                              int window, int sinks, int chunk_tiles) {
    if (check_shape(B, T_q, H_q, H_kv, d, window, sinks) != BDFP4_OK || max_pages_per_seq <= 0 || chunk_tiles <= 0)
        return 0;
    const Shape s = shape_of(T_q, H_q, H_kv, max_pages_per_seq, window, sinks, chunk_tiles);
    if (s.max_splits <= 1) return 0;
    const int64_t rows = (int64_t)B * T_q * H_q;
    return partial_bytes(rows, s.max_splits, d) + (size_t)rows * s.max_splits * 2 * sizeof(float);
}

static int run_decode8(const void* q, const void* k_pages, const void* v_pages, const float* kv_scales,
                       const int32_t* block_table, const int32_t* seq_lens, int B, int T_q, int H_q, int H_kv, int d,
                       int max_pages_per_seq, int64_t num_pages, bdfp8_fmt fmt, int window, int sinks, float sm_scale,
                       int chunk_tiles, void* workspace, size_t workspace_bytes, void* out, int32_t* dev_status,
                       void* stream, long long wait_limit, int stall) {
    int rc = check_shape(B, T_q, H_q, H_kv, d, window, sinks);
    if (rc != BDFP4_OK) return rc;
    if (max_pages_per_seq <= 0 || num_pages < 0 || (fmt != BDFP8_E4M3 && fmt != BDFP8_E5M2)) return BDFP4_ERR_ARG;
    // token indexes are 32-bit, with room for a window beyond them
    if (max_pages_per_seq > (1 << 24) || num_pages > INT_MAX) return BDFP4_ERR_UNSUPPORTED;
    if (B == 0) return BDFP4_OK;
    if (!q || !k_pages || !v_pages || !kv_scales || !block_table || !seq_lens || !out) return BDFP4_ERR_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_pages, 128) || !aligned(v_pages, 128) ||
        !aligned(kv_scales, 32) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
        return BDFP4_ERR_ALIGN;
    Args a{};
    a.G = H_q / H_kv;
    a.window = std::min(window, max_pages_per_seq * kPageSlots);
    a.sinks = window > 0 ? std::min(sinks, max_pages_per_seq * kPageSlots) : 0;
    int sms = 0;
    if (chunk_tiles <= 0) {
        if ((rc = sm_count(&sms)) != BDFP4_OK) return rc;
        const Shape s = shape_of(T_q, H_q, H_kv, max_pages_per_seq, a.window, a.sinks, 1);
        const int64_t tiles = s.max_splits;   // at one tile per split
        chunk_tiles = plan(1, [&](int) { return tiles; }, (int64_t)B * H_kv * s.groups, sms, s.rows, d);
    }
    chunk_tiles = std::min(chunk_tiles, 1 << 24);   // more than any sequence's tiles
    const Shape s = shape_of(T_q, H_q, H_kv, max_pages_per_seq, a.window, a.sinks, chunk_tiles);
    a.groups = s.groups;
    a.max_splits = s.max_splits;
    const int64_t ctas = (int64_t)B * H_kv * s.groups * s.max_splits;
    if (ctas > INT_MAX) return BDFP4_ERR_UNSUPPORTED;
    if (s.max_splits > 1) {
        const int64_t rows = (int64_t)B * T_q * H_q;
        const size_t o = partial_bytes(rows, s.max_splits, d);
        if (!workspace || workspace_bytes < o + (size_t)rows * s.max_splits * 2 * sizeof(float))
            return BDFP4_ERR_WORKSPACE;
        if (!aligned(workspace, 128)) return BDFP4_ERR_ALIGN;
        a.ws_o = (float*)workspace;
        a.ws_ml = (float*)((char*)workspace + o);
    }
    if (!sms && (rc = sm_count(&sms)) != BDFP4_OK) return rc;
    a.cluster = merges_in_cluster(s.rows, s.max_splits, ctas, sms);
    a.merge_rows = (int64_t)B * T_q * H_q > (int64_t)kMergeBlocks * sms;
    a.q = (const __nv_bfloat16*)q;
    a.k_pages = (const uint8_t*)k_pages;
    a.v_pages = (const uint8_t*)v_pages;
    a.kv_scales = kv_scales;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.out = (__nv_bfloat16*)out;
    a.dev_status = dev_status;
    a.B = B;
    a.T_q = T_q;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    a.chunk_tiles = chunk_tiles;
    a.sm_scale = sm_scale;
    a.wait_limit = wait_limit;
    a.stall = stall;
    cudaStream_t st = (cudaStream_t)stream;
    if (fmt == BDFP8_E4M3)
        return d == 128 ? dispatch<BDFP8_E4M3, 128>(a, s.rows, ctas, st) : dispatch<BDFP8_E4M3, 64>(a, s.rows, ctas, st);
    return d == 128 ? dispatch<BDFP8_E5M2, 128>(a, s.rows, ctas, st) : dispatch<BDFP8_E5M2, 64>(a, s.rows, ctas, st);
}

extern "C" int bdfp8_decode(const void* q, const void* k_pages, const void* v_pages, const float* kv_scales,
                            const int32_t* block_table, const int32_t* seq_lens, int B, int T_q, int H_q, int H_kv,
                            int d, int max_pages_per_seq, int64_t num_pages, bdfp8_fmt fmt, int window, int sinks,
                            float sm_scale, int chunk_tiles, void* workspace, size_t workspace_bytes, void* out,
                            int32_t* dev_status, void* stream) {
    return run_decode8(q, k_pages, v_pages, kv_scales, block_table, seq_lens, B, T_q, H_q, H_kv, d, max_pages_per_seq,
                       num_pages, fmt, window, sinks, sm_scale, chunk_tiles, workspace, workspace_bytes, out, dev_status,
                       stream, kWaitLimit, 0);
}

extern "C" int bdfp8_debug_decode_wait_test(const void* q, const void* k_pages, const void* v_pages,
                                            const float* kv_scales, const int32_t* block_table,
                                            const int32_t* seq_lens, int B, int T_q, int H_q, int H_kv, int d,
                                            int max_pages_per_seq, int64_t num_pages, bdfp8_fmt fmt, int window,
                                            int sinks, float sm_scale, int chunk_tiles, void* workspace,
                                            size_t workspace_bytes, void* out, int32_t* dev_status,
                                            long long wait_limit_cycles, int stall, void* stream) {
    if (wait_limit_cycles <= 0 || stall < 0 || stall > BDFP8_STALL_WARP) return BDFP4_ERR_ARG;
    return run_decode8(q, k_pages, v_pages, kv_scales, block_table, seq_lens, B, T_q, H_q, H_kv, d, max_pages_per_seq,
                       num_pages, fmt, window, sinks, sm_scale, chunk_tiles, workspace, workspace_bytes, out, dev_status,
                       stream, std::min(wait_limit_cycles, kWaitLimit - 1), stall);
}
