// decode_fp8.cuh -- what the two decode kernels over the 8-bit cache share: arguments,
// the tiles that a group of query rows sees, query terms and the producer warp.
#pragma once

#include "../../include/bdfp8_debug.h"
#include "decode_common.cuh"
#include "fp8_device.cuh"
#include "host_common.h"

namespace bdfp4 {
namespace fp8 {

struct Args {
    const __nv_bfloat16* q;
    const uint8_t* k_pages;
    const uint8_t* v_pages;
    const float* kv_scales;
    const int32_t* block_table;
    const int32_t* seq_lens;
    float* ws_o;    // [B T_q H_q][max_splits][d] unnormalised partial outputs
    float* ws_ml;   // [B T_q H_q][max_splits][2] (m in log2 units, l)
    __nv_bfloat16* out;
    int32_t* dev_status;
    int B, T_q, H_q, H_kv, G, max_pages, window, sinks, chunk_tiles, max_splits, groups;
    int cluster;   // 1: the splits of a (sequence, KV head) are a thread block cluster and merge behind its barrier
    int merge_rows;   // 1: the merge kernel takes a warp per output row, 0: a block
    int64_t num_pages;
    float sm_scale;
    // the unwind test's instantiations (bdfp8_debug.h): the bound of every wait in clock cycles, and what goes wrong
    long long wait_limit;
    int stall;
};

// The tiles that rows r0 .. r1 of a KV head's stacked rows see (row r is query token r / G).
struct Tiles {
    int end;      // tokens from here on are seen by none of the rows
    int lo;       // first token of the oldest window (0 without a window)
    int front;    // tiles of the first tokens, before the window's tiles
    int first;    // first tile of the window
    int total;
    __device__ __forceinline__ int tile(int v) const { return v < front ? v : first + v - front; }
};

__device__ __forceinline__ Tiles tiles_of(int N, int T_q, int G, int r0, int r1, int window, int sinks) {
    Tiles t;
    t.end = max(0, N - T_q + r1 / G + 1);
    t.lo = window > 0 ? max(0, N - T_q + r0 / G - window + 1) : 0;
    t.lo = min(t.lo, t.end);
    const int last = (t.end + kTileTokens - 1) / kTileTokens;
    t.first = t.lo / kTileTokens;
    t.front = window > 0 ? min((min(sinks, t.end) + kTileTokens - 1) / kTileTokens, t.first) : 0;
    t.total = t.front + last - t.first;
    return t;
}

__device__ __forceinline__ int splits_of(const Tiles& t, int chunk) { return (t.total + chunk - 1) / chunk; }

// A length out of range counts as an empty sequence.
__device__ __forceinline__ int checked_len(const Args& a, int b) {
    const int N = a.seq_lens[b];
    return N < 0 || N > a.max_pages * kPageSlots ? 0 : N;
}

// The lane's D / 32 elements of a query row (zeros for row = null).
template <int D>
__device__ __forceinline__ void load_query(const __nv_bfloat16* row, int lane, float (&x)[D / 32]) {
    constexpr int E = D / 32;
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = 0.0f;
    if (row) {
        const __nv_bfloat162* src = reinterpret_cast<const __nv_bfloat162*>(row) + lane * (E / 2);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const float2 f = __bfloat1622float2(src[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

// A query row as two E4M3 terms, by a warp: q 2^(7-e) in [128, 256) for the row's largest element, and
// the rest times 2^SHIFT.  Returns the factor of the logits (log2 units) that the terms' products carry; a row with
// an infinity or a NaN gets a NaN.  x: the lane's elements, whose codes are c1 and c2.
template <int D, int SHIFT>
__device__ __forceinline__ float split_query(const float (&x)[D / 32], float sm_scale, uint32_t& c1, uint32_t& c2) {
    constexpr int E = D / 32;
    // the largest exponent field of the row (255: an infinity or a NaN)
    uint32_t ex = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) ex = max(ex, (__float_as_uint(x[i]) >> 23) & 0xffu);
    ex = __reduce_max_sync(0xffffffffu, ex);
    const int e = min(max((int)ex - 127, -119), 127);
    const float up = pow2i(7 - e);
    c1 = c2 = 0;
#pragma unroll
    for (int i = 0; i < E; i += 2) {
        const float y0 = x[i] * up, y1 = x[i + 1] * up;
        const uint32_t c = f8x2<BDFP8_E4M3>(y0, y1);
        const float2 v = tc::e4m3x2_value(c);
        c1 |= c << (8 * i);
        c2 |= f8x2<BDFP8_E4M3>((y0 - v.x) * (float)(1 << SHIFT), (y1 - v.y) * (float)(1 << SHIFT)) << (8 * i);
    }
    return ex == 255u ? __uint_as_float(0x7fc00000u) : sm_scale * kLog2e * pow2i(e - 7);
}

// The lane's codes into row `row` of a K-major operand [row/8][elem/16][row%8][16].
template <int D>
__device__ __forceinline__ void put_query(uint8_t* op, int row, int lane, uint32_t codes) {
    constexpr int E = D / 32;
    const int e0 = lane * E;
    uint8_t* const dst = op + (row >> 3) * (8 * D) + (e0 >> 4) * 128 + (row & 7) * 16 + (e0 & 15);
    if constexpr (E == 4) *reinterpret_cast<uint32_t*>(dst) = codes;
    else *reinterpret_cast<uint16_t*>(dst) = (uint16_t)codes;
}

// What goes into the value product is p c, a probability times its value block's scale c = 2^e r, 1/2 < r <= 1: so a
// row's reference m is the maximum over the tokens that it sees of x + e (x the logit in log2 units), and with w =
// 2^(x + e - m) the product takes w r and the sum of probabilities w 2^-e, both in units of 2^m.  Every row has its own
// bound, however scales differ, and tokens that it does not see have no part in it.  (One bound on the scales for all rows of
// a block cost rows with small values their bits beside a large block that only others saw, or that had no weight.)
// The reference follows its maximum only when that has risen by more than kRise: rescaling O waits for the value
// product before, and exact maxima rise in four of ten tiles of a split of 32 (four rows a thread).  So w <= 2^kRise;
// the terms of w r, below 2^15, are in units of 2^-kTopExp, which puts their floor at 2^-28 of the row's largest p c.
// w is computed as 2^kLift w: the exponential flushes below 2^-126, and a token whose p c is that far below the
// largest may still have the larger p.
constexpr float kRise = 4.0f;
constexpr int kTopExp = 11, kLift = 22;

// e and 2^(-e - kLift) of a scale (of its amount: -0 is 0).  e >= -92, as sums of w 2^-e over 2^30 tokens have to stay finite (a scale below, 0
// among them, gives r < 1/2); the other is down to 2^-149, which fp32 holds.  A scale that is no number gets finite
// ones: its r is none.
__device__ __forceinline__ void scale_parts(float c, float& e, float& down) {
    const uint32_t u = min(max((__float_as_uint(fabsf(c)) + 0x7fffffu) >> 23, 127u - 92u), 254u);
    e = __uint_as_float(0x4b000000u + u) - (8388608.0f + 127.0f);
    down = __uint_as_float(max((254u - u) << 23, 0x400000u)) * (1.0f / (float)(1 << kLift));
}

// bdfp8_append gives a block of zeros scale 1, which says nothing of its values (those around it may have scales of
// 2^-20) and must not become a reference: before a block of scale 1 moves one, its codes are looked at, and where all of
// those that some row sees are zeros it counts as a block of scale 0.  That is rare (blocks of zeros beside others of scale
// 1 or more move nothing), so tiles pay for a comparison only.
constexpr float kZeroScale = 1.0f;

// The bytes of four slots (bits 0-3 of m4) as a mask.
__device__ __forceinline__ uint32_t byte_mask(uint32_t m4) { return (((m4 & 15u) * 0x00204081u) & 0x01010101u) * 0xffu; }

// Whether any of 16 value codes of a channel (those in the mask) is not a zero of either sign.
__device__ __forceinline__ bool any_value(const uint4& v, uint32_t mask16) {
    return ((v.x & byte_mask(mask16)) | (v.y & byte_mask(mask16 >> 4)) | (v.z & byte_mask(mask16 >> 8)) |
            (v.w & byte_mask(mask16 >> 12))) & 0x7f7f7f7fu;
}

// 2^x for x <= 0, down to fp32's smallest (references of very different scales meet).
__device__ __forceinline__ float ex2_down(float x) {
    const float h = tc::ex2_approx(0.5f * x);
    return h * h;
}

constexpr long long kWaitLimit = 1LL << 32;   // clock cycles (about 2 s)

// What the unwind test does to a block: its first key tile is never announced; or one softmax warp gives up on its
// first tile, which the others see arrive.
constexpr int kStallTile = BDFP8_STALL_TILE, kStallWarp = BDFP8_STALL_WARP;

// The block's place in a grid of B x H_kv x max_splits x groups: row groups of one split stand next to each
// other (they read the same tiles), then the splits.
struct Place {
    int b, hk, split, rg;
};
__device__ __forceinline__ Place place_of(const Args& a) {
    Place p;
    unsigned x = blockIdx.x;
    p.rg = x % (unsigned)a.groups;
    x /= (unsigned)a.groups;
    p.split = x % (unsigned)a.max_splits;
    x /= (unsigned)a.max_splits;
    p.hk = x % (unsigned)a.H_kv;
    p.b = x / (unsigned)a.H_kv;
    return p;
}

// Without a window a split's pages do not depend on the sequence's length: the producer warp loads the entries of
// its first 32 tiles while the length is on its way (those within the table; produce uses what the length allows).
__device__ __forceinline__ void early_pages(const Args& a, const Place& p, int lane, int (&early)[2]) {
    const int64_t pi = ((int64_t)p.split * a.chunk_tiles + lane) * 2;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        early[i] = a.window == 0 && pi + i < a.max_pages ? a.block_table[(int64_t)p.b * a.max_pages + pi + i] : -1;
}

// The producer warp.  Step k issues the keys and scales of tile k and the values of tile k - 1, so keys run a
// tile ahead.  Lanes read the page ids of 32 tiles at once; one lane per copy issues.
// Scales go to slot k % NSC with the keys' byte count.  A key stage is refilled once its QK
// has completed, and the MMA lane issues QK of tile t only after p_ready of tile t - 2: when
// tile k's keys are issued, the softmax is done with the scales of tile k - NSK - 2, and
// with NSC >= NSK + 2 slot k % NSC is free.
// HOOK: the unwind test's instantiation.
template <class C, bool HOOK>
__device__ __forceinline__ void produce(const Args& a, const Tiles& tl, int tile0, int n, int b, int hk, int lane, uint8_t* smem,
                                        float* sc_ring, int* pok, uint64_t* kfull, uint64_t* kempty, uint64_t* vfull,
                                        uint64_t* vempty, volatile int* abort_flag, const int (&early)[2]) {
    const long long wlim = HOOK ? a.wait_limit : kWaitLimit;
    bool ok = true;
    int pv0 = -1, pv1 = -1;
    int k_last = -1, v_last = -1;
    for (int j0 = 0; ok && j0 <= n; j0 += 32) {
        int pg_l[2] = {-1, -1};
        if (j0 + lane < n) {
            const int tile = tl.tile(tile0 + j0 + lane);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int pi = tile * 2 + p, t0 = pi * kPageSlots;
                // pages that no row sees are not looked up
                if (t0 < tl.end && (t0 + kPageSlots > tl.lo || t0 < a.sinks)) {
                    const int v = a.window == 0 && j0 == 0 ? early[p] : a.block_table[(int64_t)b * a.max_pages + pi];
                    if (v >= 0 && v < a.num_pages) pg_l[p] = v;
                    else set_status(a.dev_status, BDFP4_DEV_BAD_PAGE);
                }
            }
        }
        const int kmax = min(32, n + 1 - j0);
        for (int kk = 0; kk < kmax; ++kk) {
            const int k = j0 + kk, v = k - 1;
            const int pk0 = __shfl_sync(0xffffffffu, pg_l[0], kk), pk1 = __shfl_sync(0xffffffffu, pg_l[1], kk);
            if (k < n && !(HOOK && k == 0 && a.stall == kStallTile)) {
                const int s = k % C::NSK;
                if (lane == 0) {
                    if (k >= C::NSK && !tc::mbar_wait(&kempty[s], ((k / C::NSK) - 1) & 1, abort_flag, wlim)) {
                        ok = false;
                    } else {
                        pok[k % C::NSC] = (pk0 >= 0 ? 1 : 0) | (pk1 >= 0 ? 2 : 0);
                        tc::mbar_arrive_expect_tx(&kfull[s], ((pk0 >= 0) + (pk1 >= 0)) * (C::PAGE + kScalePage * 4));
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                if (lane < 4) {
                    const int p = lane & 1, pg = p ? pk1 : pk0;
                    const int64_t ph = (int64_t)pg * a.H_kv + hk;
                    if (pg >= 0) {
                        if (lane < 2)
                            tc::bulk_g2s(smem + C::SM_K + s * C::TILE + p * C::PAGE, a.k_pages + ph * C::PAGE, C::PAGE,
                                         &kfull[s]);
                        else
                            tc::bulk_g2s(sc_ring + ((k % C::NSC) * 2 + p) * kScalePage, a.kv_scales + ph * kScalePage,
                                         kScalePage * 4, &kfull[s]);
                    }
                }
                k_last = k;
            }
            if (v >= 0) {
                const int s = v % C::NSV;
                if (lane == 0) {
                    if (v >= C::NSV && !tc::mbar_wait(&vempty[s], ((v / C::NSV) - 1) & 1, abort_flag, wlim))
                        ok = false;
                    else
                        tc::mbar_arrive_expect_tx(&vfull[s], ((pv0 >= 0) + (pv1 >= 0)) * C::PAGE);
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                const int pg = lane ? pv1 : pv0;
                if (lane < 2 && pg >= 0)
                    tc::bulk_g2s(smem + C::SM_V + s * C::TILE + lane * C::PAGE,
                                 a.v_pages + ((int64_t)pg * a.H_kv + hk) * C::PAGE, C::PAGE, &vfull[s]);
                v_last = v;
            }
            pv0 = pk0;
            pv1 = pk1;
        }
    }
    if (!ok && lane == 0) *abort_flag = 1;
    // unwinding: every copy this warp started lands before the CTA can exit
    if ((!ok || *abort_flag) && lane == 0) {
        for (int s = 0; s < C::NSK; ++s)
            if (k_last >= s)
                tc::mbar_wait_drain(&kfull[s], ((k_last - (k_last - s) % C::NSK) / C::NSK) & 1, wlim);
        for (int s = 0; s < C::NSV; ++s)
            if (v_last >= s)
                tc::mbar_wait_drain(&vfull[s], ((v_last - (v_last - s) % C::NSV) / C::NSV) & 1, wlim);
    }
    __syncwarp();
}

// The kernel for more than 16 stacked rows (decode_fp8_wide.cu); launches on `st`, returns a host status.
constexpr int kWideRows = 128;
int launch_wide(const Args& a, int fmt, int d, int64_t ctas, cudaStream_t st);

}  // namespace fp8
}  // namespace bdfp4
