"""Operators of the 8-bit paged KV cache: their cases, their plain forms and their exact values.

Three operators belong together: a serving loop appends the new tokens' keys and
values to the cache (rotating queries and keys by position on the way), then
attends over it, to the whole context or through a sliding window with a few
first tokens that stay visible.

The cache holds pages of 64 tokens per KV head in 8-bit floats (E4M3 or E5M2) with
one fp32 scale per block of 16 tokens and head, for keys and for values:

  k_pages    [pages][H_kv][slot/8][elem/16][slot%8][16]       bytes
  v_pages    [pages][H_kv][chan/8][slot/16][chan%8][16]       bytes (tokens contiguous)
  kv_scales  [pages][H_kv][2][4] fp32                         (keys, values; 4 blocks a page)

Everything here is seeded: lengths and page tables follow from the case alone,
values from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

_DEV = "cuda" if torch.cuda.is_available() else "cpu"
_PAGE, _BLOCK = 64, 16
_FMTS = {"e4m3": (0, torch.float8_e4m3fn, 448.0), "e5m2": (1, torch.float8_e5m2, 57344.0)}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one generated token per sequence, Qwen3-4B head layout, 16 sequences: a decode step's append
        dict(name="append_step_b16", op="append", kind="step", seqs=16, new=1, lo=1000, hi=32768, hq=32, hkv=8, d=128,
             rot=128, pairs="halves", fmt="e4m3", lens=1),
        # four drafted tokens per sequence (speculative verification), Qwen3-30B-A3B head layout
        dict(name="append_verify_b64", op="append", kind="verify", seqs=64, new=4, lo=8192, hi=131072, hq=32, hkv=4,
             d=128, rot=128, pairs="halves", fmt="e4m3", lens=2),
        # eight prompts of ragged lengths, about 32 thousand tokens: a prefill batch
        dict(name="append_prefill", op="append", kind="prefill", seqs=8, new=4096, lo=0, hi=0, hq=32, hkv=8, d=128,
             rot=128, pairs="halves", fmt="e4m3", lens=3),
        # three prompts' next chunks behind cached context, head dim 64, half of it rotated in adjacent pairs
        dict(name="append_chunk_d64", op="append", kind="prefill", seqs=3, new=517, lo=16, hi=4096, hq=16, hkv=2, d=64,
             rot=32, pairs="adjacent", fmt="e5m2", lens=4),
        # one short conversation: the smallest call, where latency counts
        dict(name="decode_b1_1k", op="decode", seqs=1, tq=1, lo=1024, hi=1024, hq=4, hkv=1, d=128, fmt="e4m3",
             window=0, sinks=0, lens=5),
        # Qwen3-4B serving batch at 32768 tokens each
        dict(name="decode_b16_32k", op="decode", seqs=16, tq=1, lo=32768, hi=32768, hq=32, hkv=8, d=128, fmt="e4m3",
             window=0, sinks=0, lens=6),
        # Qwen3-30B-A3B serving batch, ragged contexts of 8 to 131 thousand tokens: the largest
        dict(name="decode_ragged_b64", op="decode", seqs=64, tq=1, lo=8192, hi=131072, hq=32, hkv=4, d=128, fmt="e4m3",
             window=0, sinks=0, lens=7),
        # verification of four drafted tokens on the Qwen3-4B batch
        dict(name="decode_verify_t4", op="decode", seqs=16, tq=4, lo=20000, hi=32768, hq=32, hkv=8, d=128, fmt="e4m3",
             window=0, sinks=0, lens=8),
        # four documents of 131 thousand tokens in the wider-range type
        dict(name="decode_131k_e5m2", op="decode", seqs=4, tq=1, lo=131072, hi=131072, hq=32, hkv=8, d=128, fmt="e5m2",
             window=0, sinks=0, lens=9),
        # a streaming batch: 4096-token window, four first tokens kept, the pages between evicted
        dict(name="window_b64", op="decode", seqs=64, tq=1, lo=8192, hi=131072, hq=32, hkv=4, d=128, fmt="e4m3",
             window=4096, sinks=4, lens=10),
        # one long stream through a window of odd length: latency
        dict(name="window_b1_131k", op="decode", seqs=1, tq=1, lo=131000, hi=131072, hq=32, hkv=8, d=128, fmt="e4m3",
             window=1000, sinks=4, lens=11),
        # the next 256 prompt tokens of two sequences through a window: chunked prefill, bound by arithmetic
        dict(name="window_chunk_t256", op="decode", seqs=2, tq=256, lo=9000, hi=20000, hq=32, hkv=8, d=128, fmt="e4m3",
             window=8192, sinks=16, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    lens = rng.randrange(1 << 30)
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8, 16])
    fmt = rng.choice(["e4m3", "e4m3", "e5m2"])
    if rng.random() < 0.35:
        kind = rng.choice(["step", "verify", "prefill"])
        rot = rng.choice([d, d, d // 2, 16])
        case = dict(op="append", kind=kind, hq=hq, hkv=hkv, d=d, rot=rot, pairs=rng.choice(["halves", "adjacent"]),
                    fmt=fmt, lens=lens)
        if kind == "prefill":
            seqs = _log(rng, 1, 12)
            new = _log(rng, 3, 20000 // seqs)
            return dict(case, seqs=seqs, new=new, lo=0, hi=rng.choice([0, 8192]))
        hi = _log(rng, 40, 131072)
        return dict(case, seqs=_log(rng, 1, 256), new=1 if kind == "step" else rng.randrange(2, 9), lo=hi // 3, hi=hi)
    window, sinks = 0, 0
    if rng.random() < 0.45:
        window, sinks = _log(rng, 17, 9000), rng.choice([0, 1, 4, 37, 130])
    hi = _log(rng, 20, 131072)
    tq = rng.choice([1, 1, 1, 2, 3, 5, 8, 33, 150])
    tq = min(tq, max(1, hi // 4))
    # no more than the largest listed case reads, nor than its chunk multiplies
    most = min(4.0e9 / (hi * hkv * 2 * d), 1.2e11 / (4.0 * tq * hi * hq * d), 3.0e9 / (hi * hq * tq * 4.0))
    seqs = _log(rng, 1, max(1, min(96, int(most)))) if most > 1 else 1
    return dict(op="decode", seqs=seqs, tq=tq, lo=max(tq, hi // 4), hi=hi, hq=hq, hkv=hkv, d=d, fmt=fmt,
                window=window, sinks=sinks, lens=lens)


# ----------------------------------------------------------------------------- lengths and pages
def _decode_lens(case):
    r = random.Random(case["lens"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]


def _append_lens(case):
    """[(cached tokens before the call, new tokens)] of each sequence."""
    r = random.Random(case["lens"])
    got = []
    for _ in range(case["seqs"]):
        start = r.randint(case["lo"], case["hi"])
        new = case["new"]
        if case["kind"] == "prefill":      # chunks begin at whole blocks
            start -= start % _BLOCK
            new = r.randint(max(1, new // 2), new + new // 2)
        elif start % _BLOCK + new > _BLOCK:  # drafted tokens within the open block
            start -= start % _BLOCK + new - _BLOCK
            start = max(start, 0)
        got.append((start, new))
    return got


def _pages_of(n):
    return (n + _PAGE - 1) // _PAGE


def _gen(seed, k):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed * 1009 + k)
    return g


def _randn(shape, seed, k):
    return torch.randn(shape, generator=_gen(seed, k), device=_DEV, dtype=torch.float32)


def _outliers(hkv, d, seed):
    """Per-channel factors of the keys: N(0, 1) but for a few channels 10 to 30 times as wide."""
    f = np.ones((hkv, d), np.float32)
    r = np.random.RandomState(seed % (1 << 31))
    for h in range(hkv):
        c = r.choice(d, 3, replace=False)
        f[h, c] = r.uniform(10, 30, 3)
    return torch.from_numpy(f).to(_DEV)


def _pow2_scale(amax, top):
    """The smallest power of two s with amax <= top s; 1 for a block of zeros (all in fp32, exact)."""
    m, e = torch.frexp(amax / top)                       # a correctly rounded quotient of at most a half ulp
    s = torch.ldexp(torch.ones_like(amax), torch.where(m == 0.5, e - 1, e).clamp(min=-126))
    s = torch.where(amax > top * s, s * 2, s)
    return torch.where(amax == 0, torch.ones_like(s), s)


# ----------------------------------------------------------------------------- inputs
def prepare(case, seed):
    return _prepare_append(case, seed) if case["op"] == "append" else _prepare_decode(case, seed)


def _prepare_append(case, seed):
    fmt, _, _ = _FMTS[case["fmt"]]
    hq, hkv, d, B = case["hq"], case["hkv"], case["d"], case["seqs"]
    lens = _append_lens(case)
    cu = np.concatenate([[0], np.cumsum([n for _, n in lens])]).astype(np.int32)
    T = int(cu[-1])
    ends = np.array([s + n for s, n in lens], np.int32)
    # the pool holds the pages that the call can write; earlier pages' entries point into it too, unread
    first = [s // _PAGE for s, _ in lens]
    need = [_pages_of(int(e)) - f for e, f in zip(ends, first)]
    P = sum(need)
    r = np.random.RandomState(case["lens"] % (1 << 31))
    perm = r.permutation(P).astype(np.int32)
    table = r.randint(0, P, size=(B, max(_pages_of(int(e)) for e in ends))).astype(np.int32)
    at = 0
    for b in range(B):
        table[b, first[b]: first[b] + need[b]] = perm[at: at + need[b]]
        at += need[b]
    # q, k and v are column ranges of one projection's output, as a model has them
    qkv = _randn((T, (hq + 2 * hkv) * d), seed, 1).to(torch.bfloat16)
    k = qkv[:, hq * d: (hq + hkv) * d].unflatten(1, (hkv, d))
    k.mul_(_outliers(hkv, d, seed).to(torch.bfloat16))
    pos = torch.arange(int(ends.max()), device=_DEV, dtype=torch.float64)
    freq = 1e6 ** (-torch.arange(0, case["rot"], 2, device=_DEV, dtype=torch.float64) / case["rot"])
    ang = pos[:, None] * freq[None, :]
    st = dict(
        case=case, q=qkv[:, : hq * d].unflatten(1, (hq, d)), k=k,
        v=qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)),
        cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float(),
        cu=torch.from_numpy(cu).to(_DEV), seq_lens=torch.from_numpy(ends).to(_DEV), table=torch.from_numpy(table).to(_DEV),
        k_open=_randn((B, _BLOCK, hkv, d), seed, 2) * _outliers(hkv, d, seed),
        v_open=_randn((B, _BLOCK, hkv, d), seed, 3).to(torch.bfloat16),
        k_pages=torch.zeros((P, hkv, _PAGE * d), dtype=torch.uint8, device=_DEV),
        v_pages=torch.zeros((P, hkv, _PAGE * d), dtype=torch.uint8, device=_DEV),
        kv_scales=torch.ones((P, hkv, 2, 4), dtype=torch.float32, device=_DEV),
        q_out=torch.zeros((T, hq, d), dtype=torch.bfloat16, device=_DEV))
    if own:
        from fp4_kv_cache_quant_b200 import bdfp8
        st["cache"] = bdfp8.FP8Cache(st["k_pages"], st["v_pages"], st["kv_scales"], P, hkv, d, fmt)
        st["open"] = bdfp8.OpenBlocks(st["k_open"], st["v_open"])
    return st


def _prepare_decode(case, seed):
    fmt, f8, top = _FMTS[case["fmt"]]
    hq, hkv, d, B, tq = case["hq"], case["hkv"], case["d"], case["seqs"], case["tq"]
    lens = _decode_lens(case)
    mp = max(_pages_of(n) for n in lens)
    table = np.full((B, mp), -1, np.int32)
    live = []
    for b, n in enumerate(lens):        # a streaming cache has given back the pages that no query sees
        lo = max(0, n - tq - case["window"] + 1) if case["window"] else 0
        live += [(b, p) for p in range(_pages_of(n)) if p * _PAGE + _PAGE > lo or p * _PAGE < case["sinks"]]
    P = len(live)
    perm = np.random.RandomState(case["lens"] % (1 << 31)).permutation(P).astype(np.int32)
    ij = np.array(live)
    table[ij[:, 0], ij[:, 1]] = perm

    def pages(k, width):
        x = _randn((P, hkv, 4, _BLOCK, d), seed, k)
        if width is not None:
            x.mul_(width[None, :, None, None, :])
        s = _pow2_scale(x.abs().amax((3, 4)), top)
        codes = x.div_(s[..., None, None]).to(f8).view(torch.uint8).view(P, hkv, _PAGE, d)
        return codes, s

    kc, ks = pages(1, _outliers(hkv, d, seed))
    vc, vs = pages(2, None)
    # slots behind a sequence's end were never written: NaN codes, whatever the allocator left
    ends = torch.tensor([n % _PAGE for n in lens if n % _PAGE], device=_DEV)
    last = torch.tensor([int(table[b, _pages_of(n) - 1]) for b, n in enumerate(lens) if n % _PAGE], device=_DEV,
                        dtype=torch.int64)
    dead = torch.arange(_PAGE, device=_DEV)[None, :] >= ends[:, None]
    for c in (kc, vc):
        tail = c[last]
        c[last] = torch.where(dead[:, None, :, None], torch.full_like(tail, 0x7F), tail)
    k_pages = kc.view(P, hkv, 8, 8, d // 16, 16).transpose(3, 4).reshape(P, hkv, _PAGE * d)
    v_pages = vc.view(P, hkv, 4, 16, d // 8, 8).permute(0, 1, 4, 2, 5, 3).reshape(P, hkv, _PAGE * d)
    st = dict(case=case, k_pages=k_pages, v_pages=v_pages, kv_scales=torch.stack([ks, vs], 2).contiguous(),
              q=_randn((B, tq, hq, d), seed, 3).to(torch.bfloat16),
              table=torch.from_numpy(table).to(_DEV), seq_lens=torch.tensor(lens, dtype=torch.int32, device=_DEV))
    if own:
        from fp4_kv_cache_quant_b200 import bdfp8
        st["cache"] = bdfp8.FP8Cache(k_pages, v_pages, st["kv_scales"], P, hkv, d, fmt)
        st["chunk"] = bdfp8.bdfp8_decode_plan(lens, tq, hq, hkv, d, torch.cuda.get_device_properties(0).multi_processor_count,
                                              window=case["window"], sinks=case["sinks"])
        st["workspace"] = bdfp8.workspace_for(B, tq, hq, hkv, d, mp, st["chunk"], window=case["window"], sinks=case["sinks"])
        st["out"] = torch.empty_like(st["q"])
    return st


# ----------------------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    if case["op"] == "append":
        if own:
            from fp4_kv_cache_quant_b200 import bdfp8
            bdfp8.bdfp8_append(st["k"], st["v"], st["cu"], st["seq_lens"], st["table"], st["cos_sin"], st["cache"],
                               st["open"], q=st["q"], q_out=st["q_out"], interleaved=case["pairs"] == "adjacent")
        else:
            _plain_append(st)
        f8 = _FMTS[case["fmt"]][1]
        return dict(k_pages=st["k_pages"].view(f8), v_pages=st["v_pages"].view(f8), kv_scales=st["kv_scales"],
                    k_open=st["k_open"], v_open=st["v_open"], q_out=st["q_out"])
    if own:
        from fp4_kv_cache_quant_b200 import bdfp8
        return bdfp8.bdfp8_decode(st["q"], st["cache"], st["table"], st["seq_lens"], 1.0 / math.sqrt(case["d"]),
                                  st["chunk"], st["workspace"], st["out"], window=case["window"], sinks=case["sinks"])
    return _plain_decode(st)


def _rotate(x, cos, sin, rot, pairs):
    """x [T, H, d] in 64 bits (values next to a border of the 8-bit type), its first `rot` elements turned by pairs."""
    x = x.double()
    y = x.clone()
    c, s = cos[:, None, :], sin[:, None, :]
    if pairs == "halves":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2] = a * c - b * s
        y[..., rot // 2: rot] = b * c + a * s
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * c - b * s
        y[..., 1:rot:2] = b * c + a * s
    return y


def _plain_append(st):
    case = st["case"]
    _, f8, top = _FMTS[case["fmt"]]
    hkv, d, rot = case["hkv"], case["d"], case["rot"]
    cu, ends, table = st["cu"].long(), st["seq_lens"].long(), st["table"].long()
    T, B, P = st["k"].shape[0], table.shape[0], st["k_pages"].shape[0]
    t = torch.arange(T, device=_DEV)
    b = torch.searchsorted(cu, t, right=True) - 1
    start = ends - (cu[1:] - cu[:-1])                     # cached tokens before the call
    at = start[b] + t - cu[b]                             # index in the sequence = position
    cs = st["cos_sin"].double()[at]
    cos, sin = cs[:, : rot // 2], cs[:, rot // 2:]
    kr = _rotate(st["k"], cos, sin, rot, case["pairs"]).float()
    st["q_out"].copy_(_rotate(st["q"], cos, sin, rot, case["pairs"]).float())
    # the open block's earlier tokens are quantized again with the new ones; rows of none go to a spare block
    row = torch.arange(_BLOCK, device=_DEV)
    old = row[None, :] < (start % _BLOCK)[:, None]        # [B, 16]
    at_old = (start - start % _BLOCK)[:, None] + row[None, :]
    blk_old = torch.where(old, table.gather(1, (at_old // _PAGE).clamp(max=table.shape[1] - 1)) * 4 + at_old % _PAGE // _BLOCK, 4 * P)
    slot = torch.cat([at % _BLOCK, row.repeat(B)])
    blk = torch.cat([table[b, at // _PAGE] * 4 + at % _PAGE // _BLOCK, blk_old.reshape(-1)])
    for x, which, pages in ((torch.cat([kr, st["k_open"].flatten(0, 1)]), 0, "k_pages"),
                            (torch.cat([st["v"].float(), st["v_open"].float().flatten(0, 1)]), 1, "v_pages")):
        amax = torch.zeros((4 * P + 1, hkv), device=_DEV)
        amax.scatter_reduce_(0, blk[:, None].expand(-1, hkv), x.abs().amax(2), "amax")
        s = _pow2_scale(amax, top)
        codes = torch.zeros((4 * P + 1, _BLOCK, hkv, d), dtype=torch.uint8, device=_DEV)
        codes[blk, slot] = (x / s[blk][:, :, None]).to(f8).view(torch.uint8)
        hit = torch.zeros(4 * P + 1, dtype=torch.bool, device=_DEV)
        hit[blk] = True
        codes = codes[:-1].view(P, 4, _BLOCK, hkv, d).permute(0, 3, 1, 2, 4)      # [P, H, 4, 16, d]
        hit = hit[:-1].view(P, 1, 4)
        if which == 0:
            to = st[pages].view(P, hkv, 4, 2, d // 16, 8, 16)
            new = codes.reshape(P, hkv, 4, 2, 8, d // 16, 16).transpose(4, 5)
        else:
            to = st[pages].view(P, hkv, d // 8, 4, 8, 16).transpose(2, 3)
            new = codes.reshape(P, hkv, 4, _BLOCK, d // 8, 8).permute(0, 1, 2, 4, 5, 3)
        to.copy_(torch.where(hit.view(P, 1, 4, *[1] * (to.dim() - 3)), new, to))
        sc = st["kv_scales"][:, :, which]
        sc.copy_(torch.where(hit, s[:-1].view(P, 4, hkv).transpose(1, 2), sc))
    # the last block's new tokens, for the next call
    last = at // _BLOCK == (ends[b] - 1) // _BLOCK
    o = torch.where(last, b * _BLOCK + at % _BLOCK, B * _BLOCK)
    for buf, x in (("k_open", kr), ("v_open", st["v"])):
        flat = torch.cat([st[buf].flatten(0, 1), st[buf].new_zeros((1, hkv, d))])
        flat[o] = x.to(flat.dtype)
        st[buf].copy_(flat[:-1].view_as(st[buf]))


def _plain_decode(st):
    case = st["case"]
    _, f8, _ = _FMTS[case["fmt"]]
    hq, hkv, d, tq, W, S = (case[k] for k in ("hq", "hkv", "d", "tq", "window", "sinks"))
    q, table, N = st["q"], st["table"].long(), st["seq_lens"].long()
    B, mp = table.shape
    g = hq // hkv
    # the pages that a query can see: the first ones, and the window's (all, without a window)
    if W:
        first = (N - tq - W + 1).clamp(min=0) // _PAGE
        front = min(_pages_of(S), mp)
        n = min(_pages_of(W + tq) + 1, mp)
        idx = torch.cat([torch.arange(front, device=_DEV).expand(B, front), first[:, None] + torch.arange(n, device=_DEV)], 1)
        again = torch.arange(front + n, device=_DEV)[None, :] >= front
        again = again & (idx < front)                     # a page of both lists counts once
    else:
        idx = torch.arange(mp, device=_DEV).expand(B, mp)
        again = torch.zeros_like(idx, dtype=torch.bool)
    page = table.gather(1, idx.clamp(max=mp - 1))
    pos = (idx[:, :, None] * _PAGE + torch.arange(_PAGE, device=_DEV)).reshape(B, -1)     # [B, n]
    held = ((page >= 0) & ~again)[:, :, None].expand(-1, -1, _PAGE).reshape(B, -1) & (pos < N[:, None])
    p0 = page.clamp(min=0)
    n = pos.shape[1]

    def values(which):
        if which == 0:
            c = st["k_pages"][p0].view(B, -1, hkv, 8, d // 16, 8, 16).permute(0, 2, 1, 3, 5, 4, 6).reshape(B, hkv, n, d)
        else:
            c = st["v_pages"][p0].view(B, -1, hkv, d // 8, 4, 8, 16).permute(0, 2, 1, 4, 6, 3, 5).reshape(B, hkv, n, d)
        x = c.view(f8).float()
        s = st["kv_scales"][:, :, which][p0].transpose(1, 2).reshape(B, hkv, n // _BLOCK)
        x.view(B, hkv, n // _BLOCK, _BLOCK, d).mul_(s[..., None, None])
        return x.masked_fill_(~held[:, None, :, None], 0.0)

    rows = q.view(B, tq, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, tq * g, d).float()
    at = N[:, None] - tq + torch.arange(tq, device=_DEV)                                  # position of each query
    see = held[:, None, :] & (pos[:, None, :] <= at[:, :, None])
    if W:
        see = see & ((pos[:, None, :] > at[:, :, None] - W) | (pos[:, None, :] < S))
    x = rows @ values(0).transpose(2, 3)
    x.mul_(1.0 / math.sqrt(d))
    x.view(B, hkv, tq, g, n).masked_fill_(~see[:, None, :, None, :], -math.inf)
    m = x.amax(3, keepdim=True)
    x.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = x.sum(3, keepdim=True)
    o = (x @ values(1)) / torch.where(total == 0, torch.ones_like(total), total)
    return o.view(B, hkv, tq, g, d).permute(0, 2, 1, 3, 4).reshape(B, tq, hq, d).to(torch.bfloat16)


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    if case["op"] == "append":
        lens = _append_lens(case)
        T = sum(n for _, n in lens)
        old = sum(s % _BLOCK for s, _ in lens)                                   # rows of the open blocks
        last = sum(min(n, s + n - (s + n - 1) // _BLOCK * _BLOCK) for s, n in lens)
        blocks = sum((s + n - 1) // _BLOCK - s // _BLOCK + 1 for s, n in lens)
        return {"bytes": 2.0 * T * d * (2 * hkv + 2 * hq) + 4.0 * T * case["rot"] + (4 + 2) * (old + last) * hkv * d
                + 2.0 * blocks * hkv * (_BLOCK * d + 4),
                "flops": 3.0 * T * (hq + hkv) * case["rot"] + 4.0 * T * hkv * d}
    tq, W, S = case["tq"], case["window"], case["sinks"]
    read, pairs = 0, 0
    for n in _decode_lens(case):
        lo = max(0, n - tq - W + 1) if W else 0
        read += n - lo + min(S if W else 0, lo)
        for i in range(tq):
            at = n - tq + i
            low = max(0, at - W + 1) if W else 0
            pairs += at + 1 - low + min(S if W else 0, low)
    return {"bytes": read * hkv * (2.0 * d + 0.5) + 4.0 * case["seqs"] * tq * hq * d, "flops": 4.0 * pairs * hq * d}


# ----------------------------------------------------------------------------- exact values
def _offsets(d):
    """Byte of (slot, element) in a key page and in a value page of one head."""
    s, e = np.arange(_PAGE)[:, None], np.arange(d)[None, :]
    k = s // 8 * 8 * d + e // 16 * 128 + s % 8 * 16 + e % 16
    v = e // 8 * 512 + s // 16 * 128 + e % 8 * 16 + s % 16
    return k, v


def _code_values(fmt):
    """The 256 values of an 8-bit float type, from its definition."""
    ebits, mbits, bias = (4, 3, 7) if fmt == "e4m3" else (5, 2, 15)
    got = np.zeros(256)
    for c in range(256):
        e, m = c >> mbits & (1 << ebits) - 1, c & (1 << mbits) - 1
        v = m * 2.0 ** (1 - bias - mbits) if e == 0 else (1 + m * 2.0 ** -mbits) * 2.0 ** (e - bias)
        if (fmt == "e4m3" and c & 127 == 127) or (fmt == "e5m2" and e == 31):
            v = np.nan if fmt == "e4m3" or m else np.inf
        got[c] = -v if c & 128 else v
    return got


def exact(case, seed):
    return _exact_append(case, seed) if case["op"] == "append" else _exact_decode(case, seed)


def _round8(x, fmt):
    """64-bit values to the nearest of the type, ties to even, saturating."""
    mbits, low, top = (3, -6, 448.0) if fmt == "e4m3" else (2, -14, 57344.0)
    e = torch.frexp(x.abs())[1] - 1
    step = torch.ldexp(torch.ones_like(x), e.clamp(min=low) - mbits)
    return (torch.round(x / step) * step).clamp(-top, top)


def _exact_append(case, seed):
    st = _prepare_append(case, seed)
    fmt, d, hkv, rot = case["fmt"], case["d"], case["hkv"], case["rot"]
    top = _FMTS[fmt][2]
    ko, vo = (torch.from_numpy(o).to(_DEV) for o in _offsets(d))
    kp, vp, sc = (torch.zeros_like(st[n], dtype=torch.float64) for n in ("k_pages", "v_pages", "kv_scales"))
    sc += 1.0
    k_open, v_open = st["k_open"].double(), st["v_open"].double()
    q_out = torch.zeros(st["q"].shape, dtype=torch.float64, device=_DEV)
    half = torch.arange(rot // 2, device=_DEV)
    i, j = (half, half + rot // 2) if case["pairs"] == "halves" else (2 * half, 2 * half + 1)
    table, t = st["table"].tolist(), 0
    for b, (start, new) in enumerate(_append_lens(case)):
        cs = st["cos_sin"][start: start + new].double()[:, None, :]
        c, s = cs[..., : rot // 2], cs[..., rot // 2:]
        turned = []
        for name in ("q", "k"):
            x = st[name][t: t + new].double()
            y = x.clone()
            y[..., i] = x[..., i] * c - x[..., j] * s
            y[..., j] = x[..., j] * c + x[..., i] * s
            turned.append(y)
        q_out[t: t + new] = turned[0]
        v = st["v"][t: t + new].double()
        t += new
        head = start % _BLOCK
        first, end = start - head, start + new
        pad = -end % _BLOCK
        for x, buf, off, pages, which in ((turned[1], k_open, ko, kp, 0), (v, v_open, vo, vp, 1)):
            z = torch.zeros((pad, hkv, d), dtype=torch.float64, device=_DEV)
            rows = torch.cat([buf[b, :head], x, z]).view(-1, _BLOCK, hkv, d)
            amax = rows.abs().amax((1, 3))
            s2 = torch.ones_like(amax)
            nz = amax > 0
            s2[nz] = torch.ldexp(torch.ones_like(amax[nz]), torch.ceil(torch.log2(amax[nz] / top)).long())
            s2 = torch.where(amax > top * s2, 2 * s2, torch.where((amax <= top * s2 / 2) & nz, s2 / 2, s2))
            r = _round8(rows / s2[:, None, :, None], fmt)
            n = torch.arange(first, end + pad, device=_DEV)
            pg = torch.tensor(table[b], device=_DEV)[n // _PAGE]
            flat = r.view(-1, hkv, d)
            h = torch.arange(hkv, device=_DEV)[None, :, None]
            pages[pg[:, None, None], h, off[n % _PAGE][:, None, :]] = flat
            k0 = n[::_BLOCK]
            sc[pg[::_BLOCK][:, None], h[:, :, 0], which, (k0 % _PAGE // _BLOCK)[:, None]] = s2
            keep = (end - 1) // _BLOCK * _BLOCK
            a = max(keep, start)
            buf[b, a - keep: end - keep] = x[a - start:]
    return dict(k_pages=kp, v_pages=vp, kv_scales=sc, k_open=k_open, v_open=v_open, q_out=q_out)


def _exact_decode(case, seed):
    st = _prepare_decode(case, seed)
    hq, hkv, d, tq, W, S = (case[k] for k in ("hq", "hkv", "d", "tq", "window", "sinks"))
    ko, vo = (torch.from_numpy(o).to(_DEV) for o in _offsets(d))
    value = torch.from_numpy(_code_values(case["fmt"])).to(_DEV)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=_DEV)
    for b, n in enumerate(_decode_lens(case)):
        t = torch.arange(n, device=_DEV)
        if W:
            t = t[(t > n - tq - W) | (t < S)]
        pg = st["table"][b].long()[t // _PAGE]
        at = n - tq + torch.arange(tq, device=_DEV)
        see = t[None, :] <= at[:, None]
        if W:
            see &= (t[None, :] > at[:, None] - W) | (t[None, :] < S)
        for h in range(hkv):
            k = value[st["k_pages"][pg, h].gather(1, ko[t % _PAGE]).long()]
            k *= st["kv_scales"][pg, h, 0, t % _PAGE // _BLOCK].double()[:, None]
            v = value[st["v_pages"][pg, h].gather(1, vo[t % _PAGE]).long()]
            v *= st["kv_scales"][pg, h, 1, t % _PAGE // _BLOCK].double()[:, None]
            for r in range(h * hq // hkv, (h + 1) * hq // hkv):
                x = st["q"][b, :, r].double() @ k.T / math.sqrt(d)
                x = torch.where(see, x, torch.full_like(x, -math.inf))
                out[b, :, r] = torch.softmax(x, 1) @ v
    return out
