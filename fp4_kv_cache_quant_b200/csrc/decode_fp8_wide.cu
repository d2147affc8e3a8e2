// decode_fp8_wide.cu -- the decode over the 8-bit cache for more than 16 stacked
// query rows per KV head: several query tokens, wide head groups, prompt chunks.
//
// The mathematics is decode_fp8.cu's with rows and tokens exchanged: S = q K^T with
// M = 128 query rows and N = 128 tokens, O = P V with N = D channels, so a TMEM lane
// and its threads own a whole row: sums need no exchange between threads, a maximum
// one between two, and a row's probabilities go back into TMEM, where the value
// product reads them as its A operand.  Its time for a tile fed from L2 hardly depends on
// the rows (1210 ns at 17 and 32, 1480 at 64 and 128; 1240 and 1380 at d = 64); the
// transposed form pays by the row (381, 449 and 580 ns at 4, 8 and 16 rows; 1380 at 32 in an
// earlier state of both).
// Both q terms add into one S (q2 at q1's scale: an absolute error of 2^-17 of the
// row's largest element at the most), the three E5M2 terms of p c into one O.
//
// One CTA per (sequence, KV head, 128 rows, split), alone on its SM.  Two streams take
// the even and the odd tiles of the same rows, each with a maximum, a sum and an O of
// its own, joined at the end like two splits: while one works on its logits the tensor
// cores work for the other.  A stream is two warpgroups, one for each half of a
// tile's tokens, which exchange a row's maximum through shared memory.  TMEM: two S
// (the probabilities over them: 32 tokens' logits read free 32 columns, their terms
// take 24) and two O, 512 columns at D = 128.  (With the probabilities in shared memory
// a stream's next logits need not wait for its value product, but the stores wait
// behind the operand reads: 1830 ns a tile against 1315.)  What bounds it: the chain of a
// stream (logits, maximum, exponentials, terms, value product), which the other stream
// covers in part, and the thread that issues the MMAs: a tile is 20 of them at 67 cycles
// (two terms of q, three of p c), beside seven waits and commits of 100 to 200 cycles
// each.  Up to 32 rows all live warps stand on one scheduler, so that every instruction of
// the chain counts: 16 x 32768 tokens, 32 / 4 heads: 172 us at 17 and 32 rows (82 at the
// copy rate), 214 at 128.

#include "decode_fp8.cuh"

namespace bdfp4 {
namespace fp8 {

template <int FMT, int D>
struct WideCfg {
    static constexpr int ROWS = kWideRows;
    static constexpr int KS = D / 32;
    static constexpr int NSW = 16;
    static constexpr int PRODUCER = NSW, MMA_WARP = NSW + 1;
    static constexpr int THREADS = 32 * (NSW + 2);
    static constexpr int NSK = 3, NSV = 4, NSC = 8;
    static constexpr int PAGE = kPageSlots * D;
    static constexpr int TILE = 2 * PAGE;
    static constexpr int Q_TERM = ROWS * D;                 // [row/8][elem/16][row%8][16]
    static constexpr int SM_K = 0;
    static constexpr int SM_V = SM_K + NSK * TILE;
    static constexpr int SM_Q = SM_V + NSV * TILE;
    static constexpr int SM_SC = SM_Q + 2 * Q_TERM;         // [NSC][2 pages][8] scales
    static constexpr int SM_LSC = SM_SC + NSC * 2 * kScalePage * 4;   // [ROWS] logit factors
    static constexpr int SM_MAX = SM_LSC + ROWS * 4;                  // [2][2][ROWS] a tile's maxima, by stream and half
    static constexpr int SM_ML = SM_MAX + 4 * ROWS * 4;               // [2][3][ROWS] a stream's maxima and its halves' sums
    static constexpr int SM_PART = SM_ML + 6 * ROWS * 4;              // [NSW][4][4] a warp's factors of its four blocks
    static constexpr int SM_POK = SM_PART + NSW * 64;                 // [NSC] page flags
    static constexpr int SM_BARS = SM_POK + NSC * 4;
    static constexpr int NBARS = 2 * NSK + 2 * NSV + 11;
    static constexpr int SM_MISC = SM_BARS + NBARS * 8;
    static constexpr int SMEM = SM_MISC + 16;
    static_assert(SM_PART % 16 == 0 && SM_BARS % 8 == 0 && SMEM <= 232448, "shared memory");
    static_assert(NSC >= NSK + 3, "scale slots: the streams' tiles finish a tile apart");
    // at the end the rings hold each stream's half of O for the other
    static_assert(ROWS * D * 4 <= SM_Q, "exchange buffer");
    static constexpr int T_S = 0, T_O = 256, T_ALLOC = 512;
    static_assert(T_O + 2 * D <= T_ALLOC, "tensor memory");
};

// Two fp32 values in one register pair, for the packed fp32 instructions.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Column, from its S on, of the terms of tokens 32 c .. 32 c + 31 (each half of the tokens within its own logits).
__device__ __forceinline__ constexpr int p_col(int c) { return 64 * (c >> 1) + 24 * (c & 1); }

// Bits of the tokens base .. base + 31 that lie in [lo, hi).
__device__ __forceinline__ uint32_t bits_in(int lo, int hi, int base) {
    const int l = min(max(lo - base, 0), 32), h = min(max(hi - base, 0), 32);
    return h > l ? (0xffffffffu >> (32 - (h - l))) << l : 0u;
}

// Tokens [base, base + 32) that [lo, end) or, in a window, the first `sinks` (below end) hold.
__device__ __forceinline__ uint32_t seen_bits(int lo, int end, int window, int sinks, int base) {
    uint32_t m = bits_in(lo, end, base);
    if (window > 0) m |= bits_in(0, min(sinks, end), base);
    return m;
}

// HOOK: the unwind test's instantiation (bdfp8_debug.h).
template <int FMT, int D, bool HOOK>
__global__ void __launch_bounds__(WideCfg<FMT, D>::THREADS, 1) decode_fp8_wide_kernel(const Args a) {
    using C = WideCfg<FMT, D>;
    const long long wlim = HOOK ? a.wait_limit : kWaitLimit;
    follow_grid();
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* const q_op = smem + C::SM_Q;
    float* const sc_ring = reinterpret_cast<float*>(smem + C::SM_SC);
    float* const lsc = reinterpret_cast<float*>(smem + C::SM_LSC);
    float* const mx = reinterpret_cast<float*>(smem + C::SM_MAX);
    float* const ml = reinterpret_cast<float*>(smem + C::SM_ML);
    int* const pok = reinterpret_cast<int*>(smem + C::SM_POK);
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + C::SM_BARS);
    uint64_t* const kfull = bars;
    uint64_t* const kempty = kfull + C::NSK;
    uint64_t* const vfull = kempty + C::NSK;
    uint64_t* const vempty = vfull + C::NSV;
    uint64_t* const k_seen = vempty + C::NSV;   // [2] the tile's keys, scales and page flags are there -> softmax
    uint64_t* const s_full = k_seen + 2;        // [2] QK done -> softmax
    uint64_t* const p_ready = s_full + 2;       // [2][2] a half's first, second 32 tokens of P written -> MMA
    uint64_t* const o_full = p_ready + 4;       // [2] PV done -> MMA lane, epilogue
    uint64_t* const q_ready = o_full + 2;
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SM_MISC);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + C::SM_MISC + 4);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Place at = place_of(a);
    const int b = at.b, hk = at.hk, split = at.split, rg = at.rg;
    int early[2] = {-1, -1};
    if (warp == C::PRODUCER) early_pages(a, at, lane, early);
    const int r0 = rg * C::ROWS, nrows = min(C::ROWS, a.G * a.T_q - r0);

    const int N = checked_len(a, b);
    const Tiles tl = tiles_of(N, a.T_q, a.G, r0, r0 + nrows - 1, a.window, a.sinks);
    const int nspl = splits_of(tl, a.chunk_tiles);
    if (tid == 0 && split == 0 && rg == 0 && hk == 0 && (N != a.seq_lens[b] || (N > 0 && N < a.T_q)))
        set_status(a.dev_status, BDFP4_DEV_BAD_SEQLEN);
    // row of the [B][T_q][H_q] arrays of stacked row r
    auto row_of = [&](int r) -> int64_t {
        return ((int64_t)b * a.T_q + r / a.G) * a.H_q + (int64_t)hk * a.G + r % a.G;
    };
    if (split > 0 && split >= nspl) return;
    if (tl.total == 0) {
        for (int i = tid; i < nrows * D; i += C::THREADS) a.out[row_of(r0 + i / D) * D + i % D] = __float2bfloat16(0.0f);
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
            tc::mbar_init(&k_seen[i], 1);
            tc::mbar_init(&s_full[i], 1);
            tc::mbar_init(&p_ready[2 * i], C::NSW / 2);
            tc::mbar_init(&p_ready[2 * i + 1], C::NSW / 2);
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
        // (a warp for each stream, issuing side by side, took 1810 ns a tile)
        if (lane == 0) {
            constexpr uint32_t idesc_qk = idesc_f8(Fmt8<BDFP8_E4M3>::mma, Fmt8<FMT>::mma, kTileTokens);
            constexpr uint32_t idesc_pv = idesc_f8(Fmt8<BDFP8_E5M2>::mma, Fmt8<FMT>::mma, D);
            // queries and keys: 8-row groups 8 D bytes apart, 16-element chunks 128 bytes apart; values: 8-channel
            // groups 512 bytes apart, 16-slot chunks 128
            constexpr uint32_t qk_hi = desc_hi(8 * D), v_hi = desc_hi(512);
            const uint32_t q_lo = desc_lo(tc::smem_u32(q_op), 128);
            const uint32_t k_lo = desc_lo(tc::smem_u32(smem + C::SM_K), 128);
            const uint32_t v_lo = desc_lo(tc::smem_u32(smem + C::SM_V), 128);
            // the last commit: its phase completes once every tcgen05 operation issued before it has
            uint64_t* last_bar = nullptr;
            uint32_t last_par = 0;
            auto issue_qk = [&](int j) -> bool {
                const int s = j % C::NSK, wg = j & 1;
                if (!tc::mbar_wait(&kfull[s], (j / C::NSK) & 1, abort_flag, wlim)) return false;
                // passes on this thread's view of the copied scales and the page flags
                tc::mbar_arrive(&k_seen[wg]);
                tc::tc_fence_after();
                const uint32_t kt = k_lo + s * (C::TILE / 16), d = tbase + C::T_S + wg * 128;
                mma_f8<false>(d, q_lo, qk_hi, kt, qk_hi, idesc_qk);
#pragma unroll
                for (int i = 1; i < 2 * C::KS; ++i)
                    mma_f8<true>(d, q_lo + (i / C::KS) * (C::Q_TERM / 16) + (i % C::KS) * 16, qk_hi, kt + (i % C::KS) * 16, qk_hi,
                                 idesc_qk);
                tc::mma_commit(&s_full[wg]);
                tc::mma_commit(&kempty[s]);
                last_bar = &kempty[s];
                last_par = (uint32_t)(j / C::NSK) & 1u;
                return true;
            };
            bool ok = tc::mbar_wait(q_ready, 0, abort_flag, wlim);
            if (ok) tc::tc_fence_after();
            ok = ok && issue_qk(0) && (n < 2 || issue_qk(1));
            for (int j = 0; ok && j < n; ++j) {
                const int s = j % C::NSV, wg = j & 1;
                const uint32_t vt = v_lo + s * (C::TILE / 16), d = tbase + C::T_O + wg * D, p = tbase + C::T_S + wg * 128;
                // 32 tokens a step: both halves' first ones, while the softmax is at the second
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (!(ok = tc::mbar_wait(&p_ready[2 * wg + i], (j >> 1) & 1, abort_flag, wlim))) break;
                    if (i == 0 && !(ok = tc::mbar_wait(&vfull[s], (j / C::NSV) & 1, abort_flag, wlim))) break;
                    tc::tc_fence_after();
#pragma unroll
                    for (int c = i; c < 4; c += 2) {
#pragma unroll
                        for (int k = 0; k < 3; ++k)
                            mma_f8_ts(d, p + p_col(c) + 8 * k, vt + (c >> 1) * (C::PAGE / 16) + (c & 1) * 16, v_hi, idesc_pv,
                                      c + k > 0 ? 1u : (uint32_t)(j > 1));
                    }
                }
                if (!ok) break;
                tc::mma_commit(&o_full[wg]);
                tc::mma_commit(&vempty[s]);
                last_bar = &vempty[s];
                last_par = (uint32_t)(j / C::NSV) & 1u;
                if (j + 2 < n) {
                    // the stream's next logits overwrite the probabilities
                    if (!(ok = tc::mbar_wait(&o_full[wg], (j >> 1) & 1, abort_flag, wlim))) break;
                    ok = issue_qk(j + 2);
                }
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
        const int wg = warp >> 3, half = (warp >> 2) & 1, qd = warp & 3;   // stream, its half of a tile's tokens
        const uint32_t tq = tbase + ((uint32_t)(32 * qd) << 16);
        const uint32_t ts = tq + C::T_S + wg * 128 + 64 * half, to = tq + C::T_O + wg * D;
        bool bad = false;

        // the query terms; a negative sm_scale changes their sign, so that logit factors are not negative
#pragma unroll 4
        for (int r = warp; r < C::ROWS; r += C::NSW) {
            uint32_t w1, w2;
            float x[D / 32];
            load_query<D>(r < nrows ? a.q + row_of(r0 + r) * D : nullptr, lane, x);
            const float f = split_query<D, 0>(x, a.sm_scale, w1, w2);
            const uint32_t flip = a.sm_scale < 0.0f ? 0x80808080u : 0u;
            put_query<D>(q_op, r, lane, w1 ^ flip);
            put_query<D>(q_op + C::Q_TERM, r, lane, w2 ^ flip);
            if (lane == 0) lsc[r] = fabsf(f);
        }
        tc::fence_proxy_async_smem();
        tc::named_bar_sync(1, 32 * C::NSW);
        if (lane == 0) tc::mbar_arrive(q_ready);

        const int r = 32 * qd + lane;                 // this thread's row
        const bool live = 32 * qd < nrows;            // warps of no row only keep the order
        const int live_threads = (nrows + 31) / 32 * 64;   // of a stream
        const float lr = lsc[r];
        const int pos = N - a.T_q + (r0 + r) / a.G;   // its token; it sees [lo_r, pos] and the first tokens up to pos
        const int lo_r = a.window > 0 ? pos - a.window + 1 : 0;
        // tiles all of whose tokens all rows see need no masks
        const int all_end = N - a.T_q + r0 / a.G + 1;
        const int all_lo = a.window > 0 ? N - a.T_q + (r0 + nrows - 1) / a.G - a.window + 1 : 0;
        float m = -INFINITY;
        uint64_t l2 = pair(0.0f, 0.0f);
        float4* const my_part = reinterpret_cast<float4*>(smem + C::SM_PART) + warp * 4;
        float* const my_max = mx + (2 * wg + half) * C::ROWS + r;
        const float* const other_max = mx + (2 * wg + 1 - half) * C::ROWS + r;

        auto arrive = [&](int i) {
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&p_ready[2 * wg + i]);
        };
        // What the rows need of this half's four blocks in a tile is worked out once for the warp, block lane % 4 in each
        // lane, while its logits are still being computed (per row, behind them, it cost 10 % at 32 rows): the key scale, e and
        // 2^(-e - kLift) of the value scale, r in units of 2^(-kTopExp - kLift); blocks that no row sees get those of scales
        // of 0.  Returns the blocks whose value scale is kZeroScale.
        auto put_part = [&](int j, int t0, int good, bool full) -> uint32_t {
            const float* const sc = sc_ring + ((j % C::NSC) * 2 + half) * kScalePage;   // the half's page: keys 0-3, values 4-7
            float k = sc[lane & 3], v = sc[kBlocksPerPage + (lane & 3)];
            if (!full && !((good >> half) & 1 && seen_bits(tl.lo, tl.end, a.window, a.sinks, t0 + 64 * half + 16 * (lane & 3)) & 0xffffu))
                k = v = 0.0f;
            float ve, v_down;
            scale_parts(v, ve, v_down);
            if (lane < 4) my_part[lane] = make_float4(k, ve, v_down, v * v_down * (float)(1 << kTopExp));
            __syncwarp();
            return __ballot_sync(0xffffffffu, v == kZeroScale) & 15u;
        };
        // One tile's logits to probabilities, this half's 64 tokens; FULL: every row sees every token of the tile.
        // False: a warp of the stream gave up.
        auto tile = [&](auto full_c, int j, int t0, int good, uint32_t zeros) -> bool {
            constexpr bool full = decltype(full_c)::value;
            uint32_t see[2] = {0xffffffffu, 0xffffffffu};
            if constexpr (!full) {
                const bool page = (good >> half) & 1;
#pragma unroll
                for (int c = 0; c < 2; ++c) see[c] = page ? seen_bits(lo_r, pos + 1, a.window, a.sinks, t0 + 64 * half + 32 * c) : 0u;
            }
            auto hide = [&](int blk, uint32_t* x) {   // 16 logits of block blk
                const uint32_t w = see[blk >> 1] >> (16 * (blk & 1));
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = (w >> i) & 1 ? x[i] : 0xff800000u;
            };
            // the row's maximum over this half, then over both
            float bm[4];   // a block's largest logit
            {
                uint32_t s[2][32];
                tc::tmem_ld<32>(ts, s[0]);
                tc::tmem_ld<32>(ts + 32, s[1]);
                tc::tmem_wait_ld();
#pragma unroll
                for (int blk = 0; blk < 4; ++blk) {
                    uint32_t* const x = s[blk >> 1] + 16 * (blk & 1);
                    if constexpr (!full) hide(blk, x);
                    float v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(x[i]);
#pragma unroll
                    for (int i = 4; i < 16; ++i) v[i & 3] = fmaxf(v[i & 3], __uint_as_float(x[i]));
                    bm[blk] = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
                }
            }
            auto maximum = [&] {
                float t = -INFINITY;
#pragma unroll
                for (int blk = 0; blk < 4; ++blk) {
                    // a block with nothing to see has no maximum, whatever its factor (0 among them)
                    const float2 f = *reinterpret_cast<const float2*>(my_part + blk);
                    t = fmaxf(t, bm[blk] == -INFINITY ? bm[blk] : fmaf(bm[blk], f.x * lr, f.y));
                }
                return t;
            };
            float mt = maximum();
            // blocks of zeros (see kZeroScale), each warp for its own rows
            if (zeros && __any_sync(0xffffffffu, mt > m + kRise)) {
                const int s = j % C::NSV;
                if (!tc::mbar_wait(&vfull[s], (j / C::NSV) & 1, abort_flag, wlim)) bad = true;
                const uint8_t* const vb = smem + C::SM_V + s * C::TILE + half * C::PAGE;
#pragma unroll 1
                for (int blk = 0; blk < 4; ++blk) {
                    if (!((zeros >> blk) & 1)) continue;
                    const uint32_t any = full ? 0xffffu : seen_bits(tl.lo, tl.end, a.window, a.sinks, t0 + 64 * half + 16 * blk);
                    bool some = false;
#pragma unroll 1
                    for (int c = lane; c < D; c += 32)
                        some |= any_value(*reinterpret_cast<const uint4*>(vb + (c >> 3) * 512 + blk * 128 + (c & 7) * 16), any);
                    if (!__any_sync(0xffffffffu, some) && lane == 0) {
                        float ve, v_down;
                        scale_parts(0.0f, ve, v_down);
                        my_part[blk] = make_float4(my_part[blk].x, ve, v_down, 0.0f);
                    }
                }
                __syncwarp();
                mt = maximum();
            }
            *my_max = mt;
            if (tc::named_bar_or(2 + wg, live_threads, bad)) return false;
            mt = fmaxf(mt, *other_max);
            float4 fn = my_part[0];
            uint32_t s[2][16];
            tc::tmem_ld<16>(ts, s[0]);
            // a new reference, where the maximum has left the old one
            const bool rise = mt > m + kRise;
            if (__any_sync(0xffffffffu, rise)) {
                const float corr = rise ? ex2_down(m - mt) : 1.0f;   // 0 before the first visible token
                l2 = mul2(l2, pair(corr, corr));
                if (j > 1) {   // the stream's previous PV completed before its logits here were computed
#pragma unroll 1
                    for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
                        uint32_t o[32];
                        tc::tmem_ld<32>(to + c, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
                        tc::tmem_st16(to + c, o);
                        tc::tmem_st16(to + c + 16, o + 16);
                    }
                    tc::tmem_wait_st();
                }
                m = rise ? mt : m;
            }
            const float mz = (m == -INFINITY ? 0.0f : m) - (float)kLift;
            tc::tmem_wait_ld();
            // probabilities times value scales as three E5M2 terms
#pragma unroll
            for (int blk = 0; blk < 4; ++blk) {
                uint32_t* const x = s[blk & 1];
                if (blk < 3) tc::tmem_ld<16>(ts + 16 * (blk + 1), s[(blk + 1) & 1]);
                if constexpr (!full) hide(blk, x);
                const float4 f = fn;
                if (blk < 3) fn = my_part[blk + 1];
                const float kf = f.x * lr, ref = f.y - mz;   // e - m + kLift
                const uint64_t k2 = pair(kf, kf), v2 = pair(f.w, f.w), ref2 = pair(ref, ref), down2 = pair(f.z, f.z);
                uint32_t w[3][4];
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    uint32_t codes[2][3];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x0 = __uint_as_float(x[i + 2 * e]), x1 = __uint_as_float(x[i + 2 * e + 1]);
                        float2 z = unpair(fma2(pair(x0, x1), k2, ref2));
                        if constexpr (!full) {   // -inf times a factor of 0 is no number
                            z.x = x0 == -INFINITY ? x0 : z.x;
                            z.y = x1 == -INFINITY ? x1 : z.y;
                        }
                        const uint64_t p = pair(tc::ex2_approx(z.x), tc::ex2_approx(z.y));
                        l2 = fma2(p, down2, l2);
                        float2 y = unpair(mul2(p, v2));
                        if constexpr (!full) {   // nor is 0 times a scale that is none
                            y.x = x0 == -INFINITY ? 0.0f : y.x;
                            y.y = x1 == -INFINITY ? 0.0f : y.y;
                        }
                        e5m2_terms(__floats2half2_rn(y.x, y.y), codes[e]);
                    }
#pragma unroll
                    for (int k = 0; k < 3; ++k) w[k][i / 4] = __byte_perm(codes[0][k], codes[1][k], 0x7531);
                }
                if (blk < 3) tc::tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 3; ++k) tc::tmem_st4(ts + p_col(blk >> 1) + 8 * k + 4 * (blk & 1), w[k][0], w[k][1], w[k][2], w[k][3]);
                if (blk & 1) {
                    tc::tmem_wait_st();
                    arrive(blk >> 1);
                }
            }
            return true;
        };

        for (int j = wg; j < n; j += 2) {
            const int t0 = tl.tile(tile0 + j) * kTileTokens;
            // (a warp that gives up stays until the stream's vote: the others may have seen the tile arrive)
            bad = !tc::mbar_wait(&k_seen[wg], (j >> 1) & 1, abort_flag, wlim);
            const int good = pok[j % C::NSC];
            const bool full = good == 3 && t0 + kTileTokens <= all_end && (t0 >= all_lo || t0 + kTileTokens <= a.sinks);
            const uint32_t zeros = live ? put_part(j, t0, good, full) : 0u;
            if (!tc::mbar_wait(&s_full[wg], (j >> 1) & 1, abort_flag, wlim) || (HOOK && a.stall == kStallWarp && j == 0 && warp == 0)) bad = true;
            tc::tc_fence_after();
            // Value columns of tokens that no row sees are zeroed: their bytes may be anything (a NaN code
            // among them), and 0 times NaN is NaN.  One channel per thread of the stream's first half.
            if (!full && half == 0) {
                const int chan = tid & 127, s = j % C::NSV;
                if (tc::mbar_wait(&vfull[s], (j / C::NSV) & 1, abort_flag, wlim) && chan < D) {
                    uint8_t* const vc = smem + C::SM_V + s * C::TILE + (chan >> 3) * 512 + (chan & 7) * 16;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const uint32_t word = (good >> (c >> 2)) & 1 ? seen_bits(tl.lo, tl.end, a.window, a.sinks, t0 + 32 * (c >> 1)) : 0u;
                        const uint32_t mk = (word >> (16 * (c & 1))) & 0xffffu;
                        if (mk == 0xffffu) continue;
                        uint4* const at = reinterpret_cast<uint4*>(vc + (c >> 2) * C::PAGE + (c & 3) * 128);
                        uint4 v = *at;
                        v.x &= byte_mask(mk);
                        v.y &= byte_mask(mk >> 4);
                        v.z &= byte_mask(mk >> 8);
                        v.w &= byte_mask(mk >> 12);
                        *at = v;
                    }
                }
                tc::fence_proxy_async_smem();
            }
            if (live) {
                bad = full ? !tile(std::true_type{}, j, t0, good, zeros) : !tile(std::false_type{}, j, t0, good, zeros);
            } else if (!bad) {
                arrive(0);
                arrive(1);
            }
            if (bad) break;
        }
        // ------------------------------------------------------------ joining the streams
        const int last = n - 1 - ((n - 1 - wg) & 1);   // this stream's last tile (-1: none)
        const bool some = last >= wg;
        if (some && !bad && !tc::mbar_wait(&o_full[wg], (last >> 1) & 1, abort_flag, wlim)) bad = true;
        tc::tc_fence_after();
        const float2 l = unpair(l2);
        if (half == 0) ml[(3 * wg) * C::ROWS + r] = m;
        ml[(3 * wg + 1 + half) * C::ROWS + r] = l.x + l.y;
        // all tiles are done behind this barrier: the rings are free
        if (tc::named_bar_or(1, 32 * C::NSW, bad || *abort_flag)) {
            *abort_flag = 1;
        } else {
            const float m_o = ml[3 * (1 - wg) * C::ROWS + r];
            const float M = fmaxf(m, m_o), Mz = M == -INFINITY ? 0.0f : M;
            const float m0 = wg == 0 ? m : m_o, m1 = wg == 0 ? m_o : m;
            const float L = (ml[C::ROWS + r] + ml[2 * C::ROWS + r]) * ex2_down(m0 - Mz) +
                            (ml[4 * C::ROWS + r] + ml[5 * C::ROWS + r]) * ex2_down(m1 - Mz);
            const float f = some ? ex2_down(m - Mz) * pow2i(-kTopExp) : 0.0f;
            float* const xch = reinterpret_cast<float*>(smem);   // [D][ROWS]
            constexpr int Q = D / 4;                             // channels that a warpgroup writes out
            const int keep = (2 * wg + half) * Q, give = (2 * (1 - wg) + half) * Q;
            uint32_t o[Q];
            tc::tmem_ld<Q>(to + give, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < Q; ++i) xch[(give + i) * C::ROWS + r] = some ? __uint_as_float(o[i]) * f : 0.0f;
            tc::named_bar_sync(1, 32 * C::NSW);
            const int64_t row = row_of(r0 + min(r, nrows - 1));
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
            tc::tmem_ld<Q>(to + keep, o);
            tc::tmem_wait_ld();
            float v[Q];
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const float mine = some ? __uint_as_float(o[i]) * f : 0.0f;
                v[i] = mine + xch[(keep + i) * C::ROWS + r];
            }
            if (r < nrows) {
                if (nspl == 1) {
                    uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + keep);
#pragma unroll
                    for (int i = 0; i < Q; i += 8) {
                        uint32_t pk[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __nv_bfloat162 p = __floats2bfloat162_rn(v[i + 2 * e] * inv, v[i + 2 * e + 1] * inv);
                            pk[e] = *reinterpret_cast<const uint32_t*>(&p);
                        }
                        dst[i / 8] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                } else {
                    float4* dst = reinterpret_cast<float4*>(a.ws_o + (row * a.max_splits + split) * D + keep);
#pragma unroll
                    for (int i = 0; i < Q; i += 4) dst[i / 4] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    if (keep == 0) {
                        a.ws_ml[(row * a.max_splits + split) * 2] = M;
                        a.ws_ml[(row * a.max_splits + split) * 2 + 1] = L;
                    }
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
}

template <int FMT, int D, bool HOOK = false>
static int launch_w(const Args& a, int64_t ctas, cudaStream_t st) {
    using C = WideCfg<FMT, D>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(decode_fp8_wide_kernel<FMT, D, HOOK>, C::SMEM, done);
    if (e == cudaSuccess)
        e = launch_following(decode_fp8_wide_kernel<FMT, D, HOOK>, (unsigned)ctas, C::THREADS, C::SMEM, 1, st, a);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return BDFP4_ERR_CUDA;
    }
    return launch_status();
}

int launch_wide(const Args& a, int fmt, int d, int64_t ctas, cudaStream_t st) {
    if (a.wait_limit != kWaitLimit || a.stall) return launch_w<BDFP8_E4M3, 128, true>(a, ctas, st);
    if (fmt == BDFP8_E4M3)
        return d == 128 ? launch_w<BDFP8_E4M3, 128>(a, ctas, st) : launch_w<BDFP8_E4M3, 64>(a, ctas, st);
    return d == 128 ? launch_w<BDFP8_E5M2, 128>(a, ctas, st) : launch_w<BDFP8_E5M2, 64>(a, ctas, st);
}

}  // namespace fp8
}  // namespace bdfp4
