// append_fp8.cu -- appending keys and values to the 8-bit paged cache (bdfp8.h)
// with the position rotation of keys and queries on the way.
//
// One CTA per (block of 16 tokens that the call touches, KV head): D threads for
// the keys (16 elements of a row each), D for the values (two channels of eight
// rows each), and all of them for the rotation of the group's queries.  The work is moving bytes
// (2 B in, 1 B out per key and value element, 2 + 2 per query element); a block's
// scale needs its maximum first, so its elements wait in registers.  A thread keeps its
// token's cosines and sines for its key and half of the group's query heads (loaded for
// each of them the kernel ran 143 M warp instructions for 32768 tokens at 32 / 8 heads,
// 184 us).  Measured: those tokens 140 us, 5200 GB/s or 79 % of the copy rate, bound by
// issue and loads in flight; 16 tokens 5.2 us a call (4.8 in a captured graph).
//
// Which sequence a CTA serves: sequence b gets the item numbers f(b) .. f(b+1) - 1,
// f(b) = cu[b] / 16 + 2 b.  n tokens from any offset touch at most n / 16 + 2 blocks
// (rounded down), which that leaves room for, so f needs no prefix sum: a warp
// finds b by a 32-way search of cu_tokens.

#include <algorithm>
#include <climits>

#include "decode_common.cuh"
#include "fp8_device.cuh"
#include "host_common.h"

namespace bdfp4 {
namespace fp8 {

struct AppendArgs {
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    const __nv_bfloat16* q;
    __nv_bfloat16* q_out;
    int64_t k_stride, v_stride, q_stride;
    const int32_t* cu;
    const int32_t* seq_lens;
    const int32_t* positions;
    const float* cos_sin;
    float* k_open;
    __nv_bfloat16* v_open;
    const int32_t* block_table;
    uint8_t* k_pages;
    uint8_t* v_pages;
    float* kv_scales;
    int32_t* dev_status;
    int64_t num_pages;
    int B, T, H_q, H_kv, G, rot, max_pos, max_pages, heads_per_cta;
};

// x cos - y sin to the nearest fp32 but for the last step's rounding: both products' and the
// difference's errors are kept, so that a code does not depend on how fp32 happened to round.
__device__ __forceinline__ float turn(float x, float c, float y, float s) {
    const float p = __fmul_rn(x, c), ep = __fmaf_rn(x, c, -p);
    const float q = __fmul_rn(y, s), eq = __fmaf_rn(y, s, -q);
    const float t = __fsub_rn(p, q);
    const float bb = __fsub_rn(t, p);
    const float e = __fadd_rn(__fsub_rn(p, __fsub_rn(t, bb)), -__fadd_rn(q, bb));
    return __fadd_rn(t, __fadd_rn(e, __fsub_rn(ep, eq)));
}

__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
    uint4 o;
    uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return o;
}

__device__ __forceinline__ void load8(const float* p, float* x) {
    const float4* v = reinterpret_cast<const float4*>(p);
    *reinterpret_cast<float4*>(x) = v[0];
    *reinterpret_cast<float4*>(x + 4) = v[1];
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    float4* v = reinterpret_cast<float4*>(p);
    v[0] = *reinterpret_cast<const float4*>(x);
    v[1] = *reinterpret_cast<const float4*>(x + 4);
}

// max(|a|, |b|), a NaN if one is.
__device__ __forceinline__ float absmax(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

// A row is handled in units of 16 elements, 8 from ea and 8 from eb, that hold both sides of
// their rotated pairs and share 8 cosines and sines: with halves paired, elements 8 u.. and 8 u + rot / 2..;
// else, and behind rot, 16 u.. and 16 u + 8...
struct Unit {
    int u, ea, eb;
    __device__ __forceinline__ Unit(int u_, int rot, bool adjacent) : u(u_) {
        const bool halves = !adjacent && 16 * u < rot;
        ea = halves ? 8 * u : 16 * u;
        eb = halves ? 8 * u + (rot >> 1) : 16 * u + 8;
    }
};

// A unit's cosines and sines, of row `cs` of the table (rot / 2 cosines, then as many sines).
struct Turn {
    float c[8], s[8];
    __device__ __forceinline__ void load(const float* cs, int u, int rot) {
        load8(cs + 8 * u, c);
        load8(cs + (rot >> 1) + 8 * u, s);
    }
    // the unit's elements a[8], b[8]
    template <bool EXACT, bool ADJ>
    __device__ __forceinline__ void apply(float* a, float* b) const {
        auto comb = [](float x, float cc, float y, float ss) { return EXACT ? turn(x, cc, y, ss) : fmaf(x, cc, -(y * ss)); };
        if constexpr (!ADJ) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = a[i], y = b[i];
                a[i] = comb(x, c[i], y, s[i]);
                b[i] = comb(y, c[i], x, -s[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float* const p = (i < 4 ? a : b) + 2 * (i & 3);
                const float x = p[0], y = p[1];
                p[0] = comb(x, c[i], y, s[i]);
                p[1] = comb(y, c[i], x, -s[i]);
            }
        }
    }
};

// The smallest power of two s >= 2^-126 with amax <= top s, as its exponent; top = 1.75 2^L.
template <int FMT>
__device__ __forceinline__ int scale_exp(uint32_t amax_bits) {
    constexpr int L = FMT == BDFP8_E4M3 ? 8 : 15;
    const int e = (int)(amax_bits >> 23) - 127 - L + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return amax_bits == 0 ? 0 : max(e, -126);
}

template <int FMT, int D, bool ADJ>
__global__ void __launch_bounds__(2 * D, 384 / D) append_fp8_kernel(const AppendArgs a) {
    constexpr int WK = D / 32;             // warps of the keys, and of the values
    constexpr int UNITS = D / 16;          // units of a row
    constexpr int PAGE = kPageSlots * D;
    follow_grid();
    __shared__ uint32_t red[2][2][WK];     // by turns, so that one barrier a block does
    int turn_of = 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned head_ctas = (a.H_kv + a.heads_per_cta - 1) / a.heads_per_cta;
    const int item = blockIdx.x / head_ctas, hk0 = blockIdx.x % head_ctas * a.heads_per_cta;

    if (blockIdx.x == 0)   // the sequences that are left out
        for (int b = tid; b < a.B; b += 2 * D) {
            const int c0 = a.cu[b], c1 = a.cu[b + 1], N = a.seq_lens[b];
            if (c0 < 0 || c1 < c0 || c1 > a.T || N < c1 - c0 || N > a.max_pages * kPageSlots)
                set_status(a.dev_status, BDFP4_DEV_BAD_SEQLEN);
        }

    // The last b with cu[b] / 16 + 2 b <= item: down to 31 candidates, whose entries and lengths the lanes
    // then hold (one round of loads for up to 31 sequences).
    int lo = 0, hi = a.B;
    while (hi - lo > 31) {
        const int step = (hi - lo + 31) >> 5;
        const int at = lo + lane * step;
        const bool le = at < hi && (lane == 0 || (a.cu[at] >> 4) + 2 * at <= item);
        const int k = __popc(__ballot_sync(0xffffffffu, le)) - 1;
        lo += k * step;
        hi = min(hi, lo + step);
    }
    const int mine_b = lo + lane;
    const int cu_l = mine_b <= hi ? a.cu[mine_b] : 0;
    const int len_l = mine_b < hi ? a.seq_lens[mine_b] : 0;
    const int at_l = __popc(__ballot_sync(0xffffffffu, mine_b < hi && (lane == 0 || (cu_l >> 4) + 2 * mine_b <= item))) - 1;
    const int b = lo + at_l;
    const int c0 = __shfl_sync(0xffffffffu, cu_l, at_l), n = __shfl_sync(0xffffffffu, cu_l, at_l + 1) - c0;
    const int end = __shfl_sync(0xffffffffu, len_l, at_l);
    if (n <= 0 || c0 < 0 || c0 > a.T - n || end < n || end > a.max_pages * kPageSlots) return;
    const int start = end - n;
    const int blk0 = start / kBlockTokens, last = (end - 1) / kBlockTokens;
    const int mine = blk0 + item - ((c0 >> 4) + 2 * b);
    if (mine < blk0 || mine > last) return;

    // table row of token t's position (null: none; the token stays as it is, infinities and signs of zeros too)
    auto angles = [&](int t, int index) -> const float* {
        const int pos = a.positions ? a.positions[t] : index;
        if (pos < 0 || pos >= a.max_pos) {
            set_status(a.dev_status, BDFP8_DEV_BAD_POSITION);
            return nullptr;
        }
        return a.cos_sin + (int64_t)pos * a.rot;
    };

    // A thread's token of a block and its unit: the first D threads take it of the keys, and both halves of the block
    // of every other query head of the group, so cosines and sines are loaded once per thread.
    const int tok = tid / UNITS % kBlockTokens, side = tid / D;
    const Unit un(tid % UNITS, a.rot, ADJ);
    const int my = mine * kBlockTokens + tok;                    // its index in the sequence
    const bool live = my >= start && my < end;
    Turn tn;
    bool turns = false;
    if (16 * un.u < a.rot && live)
        if (const float* const cs = angles(c0 + my - start, my)) {
            turns = true;
            tn.load(cs, un.u, a.rot);
        }

    const bool reads_open = start % kBlockTokens != 0;
    const bool chained = reads_open && last != blk0;
    for (int hk = hk0; hk < min(hk0 + a.heads_per_cta, a.H_kv); ++hk) {
        // The queries' first loads go out before the keys and values are worked on.
        const int64_t t64 = c0 + my - start;
        const __nv_bfloat16* const q_row = a.q + t64 * a.q_stride + hk * a.G * D;
        __nv_bfloat16* const q_dst = a.q_out + (t64 * a.H_q + hk * a.G) * D;
        const int heads = a.q && live ? a.G : 0;
        auto q_load = [&](int h, uint4* w) {
            w[0] = *reinterpret_cast<const uint4*>(q_row + h * D + un.ea);
            w[1] = *reinterpret_cast<const uint4*>(q_row + h * D + un.eb);
        };
        auto q_store = [&](int h, const uint4* w) {
            float f[8], g[8];
            unpack8(w[0], f);
            unpack8(w[1], g);
            if (turns) tn.apply<false, ADJ>(f, g);
            *reinterpret_cast<uint4*>(q_dst + h * D + un.ea) = pack8(f);
            *reinterpret_cast<uint4*>(q_dst + h * D + un.eb) = pack8(g);
        };
        uint4 qw[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (side + 2 * i < heads) q_load(side + 2 * i, qw[i]);

        // Blocks of this CTA: its own; and, where the sequence's first block has open rows and is not its last,
        // the first block's CTA does the last one too, after it has read the open rows that the last one replaces.
        for (int blk = mine;;) {
            if (!(chained && mine == last)) {
                const int i0 = blk * kBlockTokens;                 // first token index of the block
                const bool whole = i0 >= start && i0 + kBlockTokens <= end;   // all its tokens are new
                const int page = a.block_table[(int64_t)b * a.max_pages + i0 / kPageSlots];
                const bool page_ok = page >= 0 && page < a.num_pages;
                if (!page_ok && tid == 0) set_status(a.dev_status, BDFP4_DEV_BAD_PAGE);
                const int64_t ph = (int64_t)page * a.H_kv + hk;
                const int slot0 = i0 % kPageSlots;
                // values: channels 2 c and 2 c + 1 of eight rows
                const int vc = tid % (D / 2) * 2, vr = (tid - D) / (D / 2) * 8;
                float x[16];
                if (side == 0) {
                    const int i = i0 + tok;
                    float* const open = a.k_open + (((int64_t)b * kBlockTokens + tok) * a.H_kv + hk) * D;
                    if (i >= start && i < end) {
                        const int t = c0 + i - start;
                        const __nv_bfloat16* row = a.k + t * a.k_stride + hk * D;
                        const uint4 w0 = *reinterpret_cast<const uint4*>(row + un.ea);
                        const uint4 w1 = *reinterpret_cast<const uint4*>(row + un.eb);
                        unpack8(w0, x);
                        unpack8(w1, x + 8);
                        if (blk == mine) {
                            if (turns) tn.apply<true, ADJ>(x, x + 8);
                        } else if (const float* const cs = 16 * un.u < a.rot ? angles(t, i) : nullptr) {
                            Turn other;
                            other.load(cs, un.u, a.rot);
                            other.apply<true, ADJ>(x, x + 8);
                        }
                        if (blk == last) {
                            store8(open + un.ea, x);
                            store8(open + un.eb, x + 8);
                        }
                    } else if (i < start) {
                        load8(open + un.ea, x);
                        load8(open + un.eb, x + 8);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) x[e] = 0.0f;
                    }
                } else {
                    uint32_t w[8];
                    __nv_bfloat16* const open = a.v_open + (((int64_t)b * kBlockTokens + vr) * a.H_kv + hk) * D + vc;
                    const int64_t open_step = (int64_t)a.H_kv * D;
                    const __nv_bfloat16* const row = a.v + (int64_t)(c0 + i0 + vr - start) * a.v_stride + hk * D + vc;
                    if (whole) {
#pragma unroll
                        for (int r = 0; r < 8; ++r) w[r] = *reinterpret_cast<const uint32_t*>(row + r * a.v_stride);
                    } else {
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            const int i = i0 + vr + r;
                            w[r] = 0;
                            if (i < end) w[r] = *reinterpret_cast<const uint32_t*>(i < start ? open + r * open_step : row + r * a.v_stride);
                        }
                    }
                    if (blk == last) {
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            const int i = i0 + vr + r;
                            if (i >= start && i < end) *reinterpret_cast<uint32_t*>(open + r * open_step) = w[r];
                        }
                    }
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        x[r] = __uint_as_float(w[r] << 16);
                        x[8 + r] = __uint_as_float(w[r] & 0xffff0000u);
                    }
                }
                // as bits, a NaN is above an infinity and that above every number
                float am = absmax(x[0], x[1]);
#pragma unroll
                for (int e = 2; e < 16; ++e) am = absmax(am, x[e]);
                uint32_t mx = __reduce_max_sync(0xffffffffu, __float_as_uint(am));
                if (lane == 0) red[turn_of][side][warp % WK] = mx;
                __syncthreads();
                mx = red[turn_of][side][0];
#pragma unroll
                for (int w = 1; w < WK; ++w) mx = max(mx, red[turn_of][side][w]);
                turn_of ^= 1;
                // a block with an infinity or a NaN says so by its scale; its codes are 0, which no product spreads to
                // rows that do not see the block
                const bool finite = mx < 0x7f800000u;
                const int e = scale_exp<FMT>(mx);
                const float inv = pow2i(-e);
                uint2 w[2] = {};
                if (finite) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float* y = x + 8 * i;
                        w[i].x = f8x2<FMT>(y[0] * inv, y[1] * inv) | (f8x2<FMT>(y[2] * inv, y[3] * inv) << 16);
                        w[i].y = f8x2<FMT>(y[4] * inv, y[5] * inv) | (f8x2<FMT>(y[6] * inv, y[7] * inv) << 16);
                    }
                }
                if (page_ok) {
                    if (side == 0) {
                        const int s = slot0 + tok;
                        uint8_t* const dst = a.k_pages + ph * PAGE + (s >> 3) * (8 * D) + (s & 7) * 16;
                        *reinterpret_cast<uint2*>(dst + (un.ea >> 4) * 128 + (un.ea & 15)) = w[0];
                        *reinterpret_cast<uint2*>(dst + (un.eb >> 4) * 128 + (un.eb & 15)) = w[1];
                    } else {
                        uint8_t* const dst = a.v_pages + ph * PAGE + (vc >> 3) * 512 + (slot0 / kBlockTokens) * 128 + (vc & 7) * 16 + vr;
                        *reinterpret_cast<uint2*>(dst) = w[0];
                        *reinterpret_cast<uint2*>(dst + 16) = w[1];
                    }
                    if (tid == 0 || tid == D)
                        a.kv_scales[ph * kScalePage + side * kBlocksPerPage + slot0 / kBlockTokens] =
                            finite ? pow2i(e) : __uint_as_float(0x7fc00000u);
                }
            }
            if (!(chained && blk == blk0)) break;
            blk = last;
            __syncthreads();   // the open rows of the first block are read, its maxima too
        }

#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (side + 2 * i < heads) q_store(side + 2 * i, qw[i]);
        for (int h = side + 4; h < heads; h += 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (h + 2 * i < heads) q_load(h + 2 * i, qw[i]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (h + 2 * i < heads) q_store(h + 2 * i, qw[i]);
        }
    }
}

template <int FMT, int D>
static int launch_append(const AppendArgs& a, bool adjacent, unsigned grid, cudaStream_t st) {
    const cudaError_t e = launch_following(adjacent ? append_fp8_kernel<FMT, D, true> : append_fp8_kernel<FMT, D, false>, grid,
                                           2 * D, 0, 1, st, a);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return BDFP4_ERR_CUDA;
    }
    return launch_status();
}

}  // namespace fp8
}  // namespace bdfp4

using namespace bdfp4;
using namespace bdfp4::fp8;

extern "C" int bdfp8_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const void* q,
                            int64_t q_stride, void* q_out, const int32_t* cu_tokens, const int32_t* seq_lens,
                            const int32_t* positions, const float* cos_sin, int rot_dim, int max_pos, int pairing,
                            float* k_open, void* v_open, const int32_t* block_table, int B, int T, int H_q, int H_kv,
                            int d, int max_pages_per_seq, int64_t num_pages, bdfp8_fmt fmt, void* k_pages,
                            void* v_pages, float* kv_scales, int32_t* dev_status, void* stream) {
    if (B < 0 || T < 0 || H_q <= 0 || H_kv <= 0 || max_pages_per_seq <= 0 || num_pages < 0 || max_pos < 0 || rot_dim < 0 ||
        (fmt != BDFP8_E4M3 && fmt != BDFP8_E5M2) || (pairing != BDFP8_ROTATE_HALVES && pairing != BDFP8_ROTATE_ADJACENT) ||
        !q != !q_out)
        return BDFP4_ERR_ARG;
    if (H_q % H_kv || rot_dim > d || rot_dim % 16 || k_stride < (int64_t)H_kv * d || v_stride < (int64_t)H_kv * d ||
        (q && q_stride < (int64_t)H_q * d))
        return BDFP4_ERR_SHAPE;
    if (d != 64 && d != 128) return BDFP4_ERR_UNSUPPORTED;
    const int64_t ctas = ((int64_t)T / kBlockTokens + 2 * (int64_t)B) * H_kv;
    if (max_pages_per_seq > (1 << 24) || num_pages > INT_MAX || ctas > INT_MAX || (int64_t)T + 32LL * B > INT_MAX)
        return BDFP4_ERR_UNSUPPORTED;
    if (B == 0 || T == 0) return BDFP4_OK;
    if (!k || !v || !cu_tokens || !seq_lens || !k_open || !v_open || !block_table || !k_pages || !v_pages || !kv_scales ||
        (rot_dim > 0 && !cos_sin))
        return BDFP4_ERR_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(cos_sin, 16) ||
        !aligned(k_open, 128) || !aligned(v_open, 128) || !aligned(k_pages, 128) || !aligned(v_pages, 128) ||
        !aligned(kv_scales, 32) || !aligned(cu_tokens, 4) || !aligned(seq_lens, 4) ||
        !aligned(positions, 4) || !aligned(block_table, 4) || k_stride % 8 || v_stride % 8 || (q && q_stride % 8))
        return BDFP4_ERR_ALIGN;
    AppendArgs a{};
    a.k = (const __nv_bfloat16*)k;
    a.v = (const __nv_bfloat16*)v;
    a.q = (const __nv_bfloat16*)q;
    a.q_out = (__nv_bfloat16*)q_out;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_stride = q_stride;
    a.cu = cu_tokens;
    a.seq_lens = seq_lens;
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.k_open = k_open;
    a.v_open = (__nv_bfloat16*)v_open;
    a.block_table = block_table;
    a.k_pages = (uint8_t*)k_pages;
    a.v_pages = (uint8_t*)v_pages;
    a.kv_scales = kv_scales;
    a.dev_status = dev_status;
    a.num_pages = num_pages;
    a.B = B;
    a.T = T;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.G = H_q / H_kv;
    a.rot = rot_dim;
    a.max_pos = max_pos;
    a.max_pages = max_pages_per_seq;
    cudaStream_t st = (cudaStream_t)stream;
    // Many blocks: a CTA takes several KV heads of its tokens, which share the search and the table's rows (the second
    // and third waves of CTAs pay for neither); few: one, for the shortest call.
    const int64_t items = ctas / H_kv;
    a.heads_per_cta = ctas >= 4096 ? std::min(4, H_kv) : 1;
    const unsigned grid = (unsigned)(items * ((H_kv + a.heads_per_cta - 1) / a.heads_per_cta));
    const bool adj = pairing == BDFP8_ROTATE_ADJACENT;
    if (fmt == BDFP8_E4M3)
        return d == 128 ? launch_append<BDFP8_E4M3, 128>(a, adj, grid, st) : launch_append<BDFP8_E4M3, 64>(a, adj, grid, st);
    return d == 128 ? launch_append<BDFP8_E5M2, 128>(a, adj, grid, st) : launch_append<BDFP8_E5M2, 64>(a, adj, grid, st);
}
