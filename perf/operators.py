"""Cases of the serving and training operators around the attention kernels, with plain forms of each.

Three operators, reached through the package's entry points:

  append   paged_kv_append_rope, paged_kv_append_rope_fp8: new tokens' queries and keys are rotated
           to their positions, keys and values go into the pages of the cache.
  shared   paged_attn_decode_shared, paged_attn_decode_shared_fp8: one query per sequence over the
           paged cache, for groups of sequences whose first pages are the same pages.
  scoremod attn_fwd_scoremod, attn_bwd_scoremod, paged_attn_decode_scoremod(_fp8): attention whose
           scores are capped by a tanh, get a bias that falls with distance, and see an interval
           of keys per query (documents packed into a row, a prefix that all see, a window).

``own = False`` computes a case with elementary torch operations in 32 bits; ``own = True`` makes
the framework's calls.  ``exact`` computes the same in 64 bits, written apart from both.
"""
import random

import numpy as np
import torch

own = False
DEV = "cuda"
PAGE = 16
HEADS = ((12, 12), (16, 16), (32, 32), (32, 8), (32, 4), (14, 2), (6, 2), (8, 1))
DIMS = (32, 64, 80, 96, 128)
NEG = float("-inf")


def listed():
    return [
        # one decode step of a GPT-2-small-sized model for four users: the append is all latency
        dict(name="append_step_b4", op="append", B=4, N=1, H=12, Hkv=12, d=64, rope=64, inter=False, fp8=False,
             start=700, ragged=False, lseed=1),
        # one decode step of a full serving batch over an e4m3 cache, rotation of half the dims
        dict(name="append_step_b128_fp8", op="append", B=128, N=1, H=32, Hkv=8, d=128, rope=64, inter=True, fp8=True,
             start=1500, ragged=False, lseed=2),
        # chunked prefill: up to 1024 new tokens of eight sequences at once, padded to the longest
        dict(name="append_chunk_b8", op="append", B=8, N=1024, H=32, Hkv=8, d=128, rope=128, inter=False, fp8=False,
             start=2000, ragged=True, lseed=3),
        # four samples drawn from one short prompt by a GPT-2-small-sized model
        dict(name="shared_samples_b4", op="shared", B=4, S=4, H=12, Hkv=12, d=64, pages=32, suffix=64, fp8=False,
             pad=0, lseed=4),
        # a chat batch behind one long system prompt of 8192 tokens
        dict(name="shared_prompt_b32", op="shared", B=32, S=32, H=32, Hkv=8, d=128, pages=512, suffix=500, fp8=False,
             pad=1, lseed=5),
        # two long documents asked by 64 users each, e4m3 cache, some places of the batch unused
        dict(name="shared_documents_b128_fp8", op="shared", B=128, S=64, H=32, Hkv=8, d=128, pages=1024, suffix=1000,
             fp8=True, pad=5, lseed=6),
        # a short odd batch: distance bias both ways, the first tokens seen by all, padded keys
        dict(name="fwd_prefix_bias_n333", op="fwd", B=2, H=12, Hkv=12, Nq=333, Nkv=333, d=80, causal=False, cap=0.0,
             bias=True, mask="prefix", padded=True, lseed=7),
        # pretraining on documents packed into rows of 8192 tokens, capped scores
        dict(name="fwd_documents_cap_n8192", op="fwd", B=1, H=16, Hkv=4, Nq=8192, Nkv=8192, d=128, causal=True,
             cap=50.0, bias=False, mask="docs", padded=False, lseed=8),
        # fine-tuning step of a small model: distance bias under a causal mask, grouped heads, odd length
        dict(name="bwd_bias_n1000", op="bwd", B=2, H=16, Hkv=4, Nq=1000, Nkv=1000, d=64, causal=True, cap=0.0,
             bias=True, mask="none", padded=True, lseed=9),
        # the backward pass of capped scores under a causal mask with a window of 4096 keys
        dict(name="bwd_window_cap_n8192", op="bwd", B=1, H=16, Hkv=16, Nq=8192, Nkv=8192, d=128, causal=True,
             cap=30.0, bias=False, mask="window", padded=False, lseed=10),
        # two users of a small model with a distance bias
        dict(name="decode_bias_b2", op="decode", B=2, H=12, Hkv=12, d=64, ctx=900, cap=0.0, bias=True, window=0,
             fp8=False, lseed=11),
        # a serving batch of a capped model with grouped heads, long contexts, a window on the oldest keys
        dict(name="decode_cap_b32_fp8", op="decode", B=32, H=32, Hkv=8, d=128, ctx=8192, cap=50.0, bias=False,
             window=6000, fp8=True, lseed=12),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(min(hi, max(lo, round(float(np.exp(rng.uniform(np.log(lo), np.log(hi + 1)) - 1e-9))))))


def draw(rng):
    op = rng.choice(("append", "shared", "fwd", "bwd", "decode"))
    H, Hkv = rng.choice(HEADS)
    d = rng.choice(DIMS)
    case = dict(op=op, H=H, Hkv=Hkv, d=d, lseed=rng.randrange(1 << 30))
    if op == "append":
        N = 1 if rng.random() < 0.5 else _log(rng, 2, 1024)
        B = _log(rng, 1, max(1, min(256, 8192 // N)))
        case |= dict(B=B, N=N, rope=rng.choice((d, d, d // 2)), inter=rng.random() < 0.5, fp8=rng.random() < 0.5,
                     start=_log(rng, 1, 2000), ragged=rng.random() < 0.5)
        if case["rope"] % 16:
            case["rope"] = d
    elif op == "shared":
        S = _log(rng, 1, 64)
        G = _log(rng, 1, max(1, 128 // S))
        case |= dict(B=G * S, S=S, pages=_log(rng, 1, max(1, 1024 // max(1, G // 2))), suffix=_log(rng, 1, 1000),
                     fp8=rng.random() < 0.5, pad=rng.choice((0, 0, 1)) if S > 1 else 0)
    elif op in ("fwd", "bwd"):
        # one query and key have a gradient of zero, and its rounding error is no value to compare
        N = _log(rng, 1 if op == "fwd" else 32, 4096)
        B = _log(rng, 1, max(1, min(8, int(5e8 / (H * N * N)))))
        more = 0 if op == "bwd" or rng.random() < 0.6 else _log(rng, 1, 1000)
        mask = rng.choice(("none", "docs", "prefix", "window"))
        case |= dict(B=B, Nq=N, Nkv=N + more, causal=mask != "prefix" and rng.random() < 0.7,
                     cap=rng.choice((0.0, 20.0, 30.0, 50.0)), bias=rng.random() < 0.5, mask=mask,
                     padded=rng.random() < 0.4)
    else:
        ctx = _log(rng, 1, 8192)
        B = _log(rng, 1, max(1, min(64, 120_000_000 // (Hkv * ctx * d))))
        case |= dict(B=B, ctx=ctx, cap=rng.choice((0.0, 30.0, 50.0)), bias=rng.random() < 0.5,
                     window=rng.choice((0, 0, max(1, ctx // 2))), fp8=rng.random() < 0.5)
    return case


# ---------------------------------------------------------------- lengths and masks of a case (seed-free)
def _lens(case, lo, hi, n, salt=0):
    r = random.Random(case["lseed"] * 7 + salt)
    return np.array([r.randint(lo, max(lo, hi)) for _ in range(n)], dtype=np.int64)


def _starts(case):
    return _lens(case, 0, case["start"], case["B"])


def _new(case):
    N = case["N"]
    return _lens(case, 0, N, case["B"], 1) if case["ragged"] else np.full(case["B"], N, dtype=np.int64)


def _shared_pages(case):
    G, P = case["B"] // case["S"], case["pages"]
    p = _lens(case, max(1, P // 2), P, G, 2)
    p[0] = P
    return p


def _shared_ctx(case):
    """Tokens of each sequence: its group's shared pages and 1 to `suffix` of its own; 0 for unused places."""
    ctx = np.repeat(_shared_pages(case), case["S"]) * PAGE + _lens(case, 1, case["suffix"], case["B"], 3)
    if case["pad"]:
        ctx[-case["pad"]:] = 0
    return ctx


def _decode_ctx(case):
    return _lens(case, max(1, case["ctx"] // 16), case["ctx"], case["B"], 4)


def _interval(case):
    """(key_begin, key_end, kv_lens) of a training case: int64 [B, Nq], [B, Nq], [B], None where there is none."""
    B, Nq, Nkv = case["B"], case["Nq"], case["Nkv"]
    pos = np.arange(Nq)[None, :] + (Nkv - Nq) + np.zeros((B, 1), dtype=np.int64)
    kv_lens = _lens(case, max(1, Nkv - Nkv // 4), Nkv, B, 5) if case["padded"] else None
    begin = end = None
    if case["mask"] == "docs":
        begin, end = np.zeros((B, Nq), np.int64), np.zeros((B, Nq), np.int64)
        for b in range(B):
            r = random.Random(case["lseed"] * 11 + b)
            edges = [0]
            while edges[-1] < Nkv:
                edges.append(min(Nkv, edges[-1] + r.randint(max(1, Nkv // 64), max(1, Nkv // 4))))
            e = np.array(edges)
            at = np.searchsorted(e, pos[b], side="right") - 1
            begin[b], end[b] = e[at], e[at + 1]
    elif case["mask"] == "prefix":
        end = np.maximum(pos + 1, _lens(case, 0, Nkv // 2, B, 6)[:, None])
    elif case["mask"] == "window":
        begin = pos - max(1, Nkv // 2) + 1
    return begin, end, kv_lens


def _bounds(case):
    """First and one-past-last key that each query sees: int64 [B, Nq]."""
    B, Nq, Nkv = case["B"], case["Nq"], case["Nkv"]
    begin, end, kv_lens = _interval(case)
    lo = np.zeros((B, Nq), np.int64) if begin is None else np.maximum(begin, 0)
    hi = np.full((B, Nq), Nkv, np.int64) if end is None else np.minimum(end, Nkv)
    if kv_lens is not None:
        hi = np.minimum(hi, kv_lens[:, None])
    if case["causal"]:
        hi = np.minimum(hi, np.arange(Nq)[None, :] + (Nkv - Nq) + 1)
    return lo, hi


def work(case):
    H, Hkv, d, B = case["H"], case["Hkv"], case["d"], case["B"]
    e = 1 if case.get("fp8") else 2
    if case["op"] == "append":
        t = int(_new(case).sum())
        return {"bytes": t * (4 * H * d + 2 * Hkv * d * (2 + e) + 4 * case["rope"]), "flops": 3 * t * (H + Hkv) * case["rope"]}
    if case["op"] == "shared":
        pre, ctx = _shared_pages(case) * PAGE, _shared_ctx(case)
        own_tokens = int((ctx - np.repeat(pre, case["S"])).clip(0).sum())
        return {"bytes": (int(pre.sum()) + own_tokens) * 2 * Hkv * d * e + 4 * B * H * d + 4 * B * H,
                "flops": 4 * H * d * int(ctx.sum())}
    if case["op"] == "decode":
        ctx = _decode_ctx(case)
        seen = int((np.minimum(ctx, case["window"]) if case["window"] else ctx).sum())
        return {"bytes": seen * 2 * Hkv * d * e + 4 * B * H * d + 4 * B * H, "flops": 4 * H * d * seen}
    lo, hi = _bounds(case)
    pairs = int((hi - lo).clip(0).sum()) * H
    q, kv, row = B * H * case["Nq"] * d * 2, B * Hkv * case["Nkv"] * d * 2, 4 * B * H * case["Nq"]
    if case["op"] == "fwd":
        return {"bytes": 2 * q + 2 * kv + row, "flops": 4 * d * pairs}
    return {"bytes": 4 * q + 4 * kv + row, "flops": 10 * d * pairs}


# ---------------------------------------------------------------- inputs
def _i32(a):
    return None if a is None else torch.tensor(np.ascontiguousarray(a), dtype=torch.int32, device=DEV)


def _slopes(case):
    H = case["H"]
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device=DEV)


def _pool(case, g, pages):
    """K and V pages with normal values: bf16, or e4m3 codes of values / scale."""
    shape = (pages, case["Hkv"], PAGE, case["d"])
    x = [torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    if case["fp8"]:
        x = [(t.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for t, s in zip(x, (0.02, 0.015))]
    return x


def _table(g, per_seq):
    """Page tables of sequences with pages of their own, in an order of the pool that the seed gives."""
    per_seq = np.asarray(per_seq)
    total, width = int(per_seq.sum()), max(1, int(per_seq.max()))
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor(np.concatenate([[0], np.cumsum(per_seq)[:-1]]), device=DEV)
    col = torch.arange(width, device=DEV)
    ok = col[None, :] < torch.tensor(per_seq, device=DEV)[:, None]
    at = (first[:, None] + col[None, :]).clamp(max=max(0, total - 1))
    return torch.where(ok, perm[at], torch.zeros_like(perm[at])).contiguous(), total


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    H, Hkv, d, B = case["H"], case["Hkv"], case["d"], case["B"]
    s = dict(case=case, scale=d ** -0.5, k_scale=0.02, v_scale=0.015)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)

    if case["op"] == "append":
        N, r = case["N"], case["rope"]
        start, new = _starts(case), _new(case)
        table, total = _table(g, np.maximum(1, -(-(start + N) // PAGE)))
        s["k_pages"], s["v_pages"] = _pool(case, g, total)
        # the projection's output, [B, N, (H + 2 Hkv) d]; queries, keys and values are views of it
        qkv = normal(B, N, (H + 2 * Hkv), d).transpose(1, 2)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        s["q_out"] = torch.zeros(B, H, N, d, dtype=torch.bfloat16, device=DEV)
        angle = torch.arange(int((start + N).max()), dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, r, 2, dtype=torch.float64) / r)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().to(DEV)
        s["table"], s["start"], s["new"] = table, _i32(start), _i32(new) if case["ragged"] else None
    elif case["op"] == "shared":
        pre, ctx = _shared_pages(case), _shared_ctx(case)
        own_pages = np.maximum(0, -(-ctx // PAGE) - np.repeat(pre, case["S"]))
        table, total = _table(g, np.concatenate([pre, own_pages]))
        G, width = len(pre), int((np.repeat(pre, case["S"]) + own_pages).max())
        col = torch.arange(width, device=DEV)[None, :]
        pre_b = torch.tensor(np.repeat(pre, case["S"]), device=DEV)[:, None]
        head = table[:G].repeat_interleave(case["S"], 0)
        tail = table[G:]
        s["table"] = torch.where(col < pre_b, head.gather(1, col.clamp(max=table.shape[1] - 1).expand(B, -1)),
                                 tail.gather(1, (col - pre_b).clamp(0, table.shape[1] - 1))).contiguous()
        s["k_pages"], s["v_pages"] = _pool(case, g, total)
        s["q"] = normal(B, H, d)
        s["ctx"], s["shared"] = _i32(ctx), _i32(pre)
        s["pre_max"], s["own_max"] = int(pre.max()), max(1, int(own_pages.max()))
    elif case["op"] == "decode":
        ctx = _decode_ctx(case)
        s["table"], total = _table(g, -(-ctx // PAGE))
        s["k_pages"], s["v_pages"] = _pool(case, g, total)
        s["q"] = normal(B, H, d)
        s["ctx"] = _i32(ctx)
        s["slopes"] = _slopes(case) if case["bias"] else None
        s["begin"] = _i32(ctx - case["window"]) if case["window"] else None
    else:
        Nq, Nkv = case["Nq"], case["Nkv"]
        s["q"], s["k"], s["v"] = normal(B, H, Nq, d), normal(B, Hkv, Nkv, d), normal(B, Hkv, Nkv, d)
        begin, end, kv_lens = _interval(case)
        s["begin"], s["end"], s["kv_lens"] = _i32(begin), _i32(end), _i32(kv_lens)
        s["slopes"] = _slopes(case) if case["bias"] else None
        if case["op"] == "bwd":  # what the forward pass left, and the gradient that comes in
            s["o"], s["lse"] = _fwd(s)
            s["dout"] = normal(B, H, Nq, d)
    return s


# ---------------------------------------------------------------- plain forms, 32 bits
def _append(s):
    c, q, k = s["case"], s["q"].float(), s["k_new"].float()
    N, r, fp8 = c["N"], c["rope"], c["fp8"]
    pos = s["start"].long()[:, None] + torch.arange(N, device=DEV)
    cs = s["cos_sin"][pos][:, None]  # [B, 1, N, rope]
    cos, sin = cs[..., :r // 2], cs[..., r // 2:]

    def rotate(x):
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["inter"] else (x[..., :r // 2], x[..., r // 2:r])
        u, w = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack([u, w], -1).flatten(-2) if c["inter"] else torch.cat([u, w], -1)
        return torch.cat([turned, x[..., r:]], -1)

    def coded(x, scale):
        if not fp8:
            return x.to(torch.bfloat16)
        return (x * (1.0 / torch.tensor(scale, dtype=torch.float32, device=DEV))).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    valid = torch.ones_like(pos, dtype=torch.bool) if s["new"] is None else torch.arange(N, device=DEV) < s["new"][:, None]
    b, t = valid.nonzero(as_tuple=True)
    at = pos[b, t]
    page, slot = s["table"][b, at // PAGE].long(), at % PAGE
    s["k_pages"][page, :, slot] = coded(rotate(k), s["k_scale"])[b, :, t]
    s["v_pages"][page, :, slot] = coded(s["v_new"].float(), s["v_scale"])[b, :, t]
    s["q_out"].copy_(torch.where(valid[:, None, :, None], rotate(q).to(torch.bfloat16), s["q_out"]))


def _values(codes, scale, fp8):
    return codes.view(torch.float8_e4m3fn).float() * scale if fp8 else codes.float()


def _pages(s, ids):
    """Keys and values of tables of pages ids [n, p], as [n, Hkv, p * 16, d] in 32 bits."""
    n, p = ids.shape
    fp8 = s["case"]["fp8"]

    def of(pool, scale):
        return _values(pool[ids.long()], scale, fp8).permute(0, 2, 1, 3, 4).reshape(n, pool.shape[1], p * PAGE, -1)

    return of(s["k_pages"], s["k_scale"]), of(s["v_pages"], s["v_scale"])


def _softmax(x):
    """Weights over the last axis and the log of their sum; rows that see nothing have weights 0 and -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == NEG, torch.zeros_like(m), m)
    e = (x - m).exp()
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total)), (m + total.log()).squeeze(-1)


def _shared(s):
    c = s["case"]
    B, S, H, Hkv, d = c["B"], c["S"], c["H"], c["Hkv"], c["d"]
    G, gp = B // S, H // Hkv
    pre = s["shared"].long()
    kp, vp = _pages(s, s["table"][::S, :s["pre_max"]])  # the shared pages, once for a group
    col = (pre.repeat_interleave(S)[:, None] + torch.arange(s["own_max"], device=DEV)).clamp(max=s["table"].shape[1] - 1)
    ks, vs = _pages(s, s["table"].gather(1, col))  # each sequence's own
    q = s["q"].float() * s["scale"]
    xp = torch.matmul(q.view(G, S, Hkv, gp, d).transpose(1, 2).reshape(G, Hkv, S * gp, d), kp.transpose(2, 3))
    xp = xp.view(G, Hkv, S, gp, -1).transpose(1, 2).reshape(B, Hkv, gp, -1)
    xs = torch.matmul(q.view(B, Hkv, gp, d), ks.transpose(2, 3))
    pt = pre.repeat_interleave(S)[:, None] * PAGE
    ctx = s["ctx"].long()[:, None]
    jp, js = torch.arange(xp.shape[-1], device=DEV), torch.arange(xs.shape[-1], device=DEV)
    xp = xp.masked_fill(~((jp < pt) & (jp < ctx))[:, None, None], NEG)
    xs = xs.masked_fill(~(js + pt < ctx)[:, None, None], NEG)
    p, lse = _softmax(torch.cat([xp, xs], -1))
    pp, ps = p[..., :xp.shape[-1]], p[..., xp.shape[-1]:]
    o = torch.matmul(pp.reshape(G, S, Hkv, gp, -1).transpose(1, 2).reshape(G, Hkv, S * gp, -1), vp)
    o = o.view(G, Hkv, S, gp, d).transpose(1, 2).reshape(B, Hkv, gp, d) + torch.matmul(ps, vs)
    return o.reshape(B, H, d).to(torch.bfloat16), lse.reshape(B, H)


def _decode(s):
    c = s["case"]
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    k, v = _pages(s, s["table"])
    x = torch.matmul(s["q"].float().view(B, Hkv, H // Hkv, d), k.transpose(2, 3)) * s["scale"]
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    j, ctx = torch.arange(k.shape[2], device=DEV), s["ctx"].long()[:, None]
    if c["bias"]:
        far = (ctx - 1 - j).float()
        x = x - s["slopes"].view(1, Hkv, H // Hkv, 1) * far[:, None, None]
    see = j < ctx
    if s["begin"] is not None:
        see = see & (j >= s["begin"][:, None])
    p, lse = _softmax(x.masked_fill(~see[:, None, None], NEG))
    return torch.matmul(p, v).reshape(B, H, d).to(torch.bfloat16), lse.reshape(B, H)


def _see(s):
    c = s["case"]
    i = torch.arange(c["Nq"], device=DEV)[:, None] + (c["Nkv"] - c["Nq"])
    j = torch.arange(c["Nkv"], device=DEV)[None, :]
    see = (j <= i if c["causal"] else j >= 0).expand(c["B"], c["Nq"], c["Nkv"])
    if s["begin"] is not None:
        see = see & (j >= s["begin"][:, :, None])
    if s["end"] is not None:
        see = see & (j < s["end"][:, :, None])
    if s["kv_lens"] is not None:
        see = see & (j < s["kv_lens"][:, None, None])
    return see, (i - j).abs().float()


def _grouped(s):
    c = s["case"]
    q = s["q"].float().view(c["B"], c["Hkv"], c["H"] // c["Hkv"], c["Nq"], c["d"])
    return q, s["k"].float()[:, :, None], s["v"].float()[:, :, None]


def _scores(s, q, k):
    """Scores with the cap, the bias and the mask, and the tanh of the cap where there is one."""
    c = s["case"]
    x, t = torch.matmul(q, k.transpose(-1, -2)) * s["scale"], None
    if c["cap"]:
        t = torch.tanh(x / c["cap"])
        x = c["cap"] * t
    see, far = _see(s)
    if c["bias"]:
        x = x - s["slopes"].view(1, c["Hkv"], -1, 1, 1) * far
    return x.masked_fill(~see[:, None, None], NEG), t


def _fwd(s):
    q, k, v = _grouped(s)
    p, lse = _softmax(_scores(s, q, k)[0])
    return torch.matmul(p, v).reshape(s["q"].shape).to(torch.bfloat16), lse.reshape(s["q"].shape[:3])


def _bwd(s):
    q, k, v = _grouped(s)
    x, t = _scores(s, q, k)
    lse = s["lse"].view(q.shape[:4])[..., None]
    p = (x - torch.where(lse == NEG, torch.zeros_like(lse), lse)).exp()
    do, o = s["dout"].float().view(q.shape), s["o"].float().view(q.shape)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True))
    if t is not None:
        ds = ds * (1 - t * t)
    ds = ds * s["scale"]
    dq = torch.matmul(ds, k).reshape(s["q"].shape)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
    return dq.to(torch.bfloat16), dk.to(torch.bfloat16), dv.to(torch.bfloat16)


PLAIN = dict(append=_append, shared=_shared, decode=_decode, fwd=_fwd, bwd=_bwd)


# ---------------------------------------------------------------- the framework's calls
def _calls(s):
    import attn_fwd_02_gb300 as A
    c = s["case"]
    scales = (s["k_scale"], s["v_scale"])
    if c["op"] == "append":
        if c["fp8"]:
            A.paged_kv_append_rope_fp8(s["q"], s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], *scales, s["cos_sin"],
                                       s["table"], s["start"], interleaved=c["inter"], new_lens=s["new"], q_out=s["q_out"])
        else:
            A.paged_kv_append_rope(s["q"], s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["cos_sin"], s["table"],
                                   s["start"], interleaved=c["inter"], new_lens=s["new"], q_out=s["q_out"])
        return None
    if c["op"] == "shared":
        if c["fp8"]:
            return A.paged_attn_decode_shared_fp8(s["q"], s["k_pages"], s["v_pages"], *scales, s["table"], s["ctx"],
                                                  s["shared"], c["S"], s["scale"])
        return A.paged_attn_decode_shared(s["q"], s["k_pages"], s["v_pages"], s["table"], s["ctx"], s["shared"], c["S"],
                                          s["scale"])
    if c["op"] == "decode":
        if c["fp8"]:
            return A.paged_attn_decode_scoremod_fp8(s["q"], s["k_pages"], s["v_pages"], *scales, s["table"], s["ctx"],
                                                    s["scale"], softcap=c["cap"], alibi_slopes=s["slopes"],
                                                    key_begin=s["begin"])
        return A.paged_attn_decode_scoremod(s["q"], s["k_pages"], s["v_pages"], s["table"], s["ctx"], s["scale"],
                                            softcap=c["cap"], alibi_slopes=s["slopes"], key_begin=s["begin"])
    mod = dict(softcap=c["cap"], alibi_slopes=s["slopes"], key_begin=s["begin"], key_end=s["end"], kv_lens=s["kv_lens"])
    if c["op"] == "fwd":
        return A.attn_fwd_scoremod(s["q"], s["k"], s["v"], c["causal"], s["scale"], **mod)
    return A.attn_bwd_scoremod(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dout"], c["causal"], s["scale"], **mod)


def _named(s, out):
    c = s["case"]
    if c["op"] == "append":
        f8 = (lambda t: t.view(torch.float8_e4m3fn)) if c["fp8"] else (lambda t: t)
        return dict(q=s["q_out"], k_pages=f8(s["k_pages"]), v_pages=f8(s["v_pages"]))
    return dict(zip(("dq", "dk", "dv") if c["op"] == "bwd" else ("o", "lse"), out))


def run(s):
    return _named(s, _calls(s) if own else PLAIN[s["case"]["op"]](s))


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The operators from their definitions, one batch entry and one key/value head at a time."""
    s = prepare(case, seed)
    B, H, Hkv, d = case["B"], case["H"], case["Hkv"], case["d"]
    gp = H // Hkv
    f = torch.float64

    if case["op"] == "append":
        r, half = case["rope"], case["rope"] // 2
        start, new = _starts(case), _new(case)
        ks, vs = (s["k_scale"], s["v_scale"]) if case["fp8"] else (1.0, 1.0)
        out = [t.view(torch.float8_e4m3fn).to(f) if case["fp8"] else t.to(f) for t in (s["k_pages"], s["v_pages"])]
        qo = s["q_out"].to(f)
        i = torch.arange(half, device=DEV)
        first, second = (2 * i, 2 * i + 1) if case["inter"] else (i, i + half)
        for b in range(B):
            n = int(new[b])
            pos = torch.arange(int(start[b]), int(start[b]) + n, device=DEV)
            z = torch.complex(s["cos_sin"][pos, :half].to(f), s["cos_sin"][pos, half:].to(f))
            page, slot = s["table"][b][pos // PAGE].long(), pos % PAGE
            for what, src in (("q", s["q"]), ("k", s["k_new"])):
                x = src[b, :, :n].to(f)
                w = torch.complex(x[..., first], x[..., second]) * z
                x[..., first], x[..., second] = w.real, w.imag
                if what == "q":
                    qo[b, :, :n] = x
                else:
                    out[0][page, :, slot] = (x.transpose(0, 1) / ks).clamp(-448, 448) if case["fp8"] else x.transpose(0, 1)
            v = s["v_new"][b, :, :n].to(f).transpose(0, 1)
            out[1][page, :, slot] = (v / vs).clamp(-448, 448) if case["fp8"] else v
        return dict(q=qo, k_pages=out[0], v_pages=out[1])

    def attend(q, k, v, keep, far, slopes, cap):
        """q [g, n, d], k, v [m, d], keep and far [n, m], slopes [g] or None: outputs [g, n, d], logs [g, n], and the weights."""
        x = q @ k.T * s["scale"]
        t = torch.tanh(x / cap) if cap else None
        x = cap * t if cap else x
        if slopes is not None:
            x = x - slopes[:, None, None] * far
        x = torch.where(keep, x, torch.full((), NEG, dtype=f, device=DEV))
        lse = torch.logsumexp(x, -1)
        p = torch.exp(x - lse.nan_to_num(neginf=0.0)[..., None])
        return p @ v, lse, p, t

    if case["op"] in ("shared", "decode"):
        ctx = _shared_ctx(case) if case["op"] == "shared" else _decode_ctx(case)
        o, l = torch.zeros(B, H, d, dtype=f, device=DEV), torch.full((B, H), NEG, dtype=f, device=DEV)
        cap = case.get("cap", 0.0)
        for b in range(B):
            n = int(ctx[b])
            lo = max(0, n - case["window"]) if case.get("window") else 0
            if n == 0:
                continue
            j = torch.arange(lo, n, device=DEV)
            page, slot = s["table"][b][j // PAGE].long(), j % PAGE
            kv = [t[page, :, slot] for t in (s["k_pages"], s["v_pages"])]
            if case["fp8"]:
                kv = [t.view(torch.float8_e4m3fn).to(f) * c for t, c in zip(kv, (s["k_scale"], s["v_scale"]))]
            k, v = (t.to(f).transpose(0, 1) for t in kv)  # [Hkv, n, d]
            x = torch.einsum("hgd,hnd->hgn", s["q"][b].to(f).view(Hkv, gp, d), k) * s["scale"]
            if cap:
                x = cap * torch.tanh(x / cap)
            if case.get("bias"):
                x = x - s["slopes"].to(f).view(Hkv, gp, 1) * (n - 1 - j)
            l[b] = torch.logsumexp(x, -1).view(H)
            o[b] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), v).reshape(H, d)
        return dict(o=o, lse=l)

    Nq, Nkv = case["Nq"], case["Nkv"]
    lo, hi = (torch.tensor(t, device=DEV) for t in _bounds(case))
    j = torch.arange(Nkv, device=DEV)
    far = (torch.arange(Nq, device=DEV)[:, None] + (Nkv - Nq) - j).abs().to(f)
    q = s["q"].to(f).view(B, Hkv, gp, Nq, d)
    names = ("o", "lse") if case["op"] == "fwd" else ("dq", "dk", "dv")
    res = [torch.zeros(B, Hkv, gp, Nq, d, dtype=f, device=DEV), torch.zeros(B, Hkv, gp, Nq, dtype=f, device=DEV)]
    if case["op"] == "bwd":
        res = [res[0], torch.zeros(B, Hkv, Nkv, d, dtype=f, device=DEV), torch.zeros(B, Hkv, Nkv, d, dtype=f, device=DEV)]
        # the gradient is that of the function itself: outputs and weights come from 64 bits too
        dout = s["dout"].to(f).view(B, Hkv, gp, Nq, d)
    for b in range(B):
        keep = (j >= lo[b][:, None]) & (j < hi[b][:, None])
        for h in range(Hkv):
            k, v = s["k"][b, h].to(f), s["v"][b, h].to(f)
            for e in range(gp):
                sl = s["slopes"].to(f)[h * gp + e:h * gp + e + 1] if case["bias"] else None
                o, lse, p, t = attend(q[b, h, e][None], k, v, keep, far, sl, case["cap"])
                if case["op"] == "fwd":
                    res[0][b, h, e], res[1][b, h, e] = o[0], lse[0]
                    continue
                p, g = p[0], dout[b, h, e]
                res[2][b, h] += p.T @ g
                ds = p * (g @ v.T - (g * o[0]).sum(-1, keepdim=True)) * s["scale"]
                if t is not None:
                    ds = ds * (1 - t[0] ** 2)
                res[0][b, h, e] = ds @ k
                res[1][b, h] += ds.T @ q[b, h, e]
    shape = dict(o=(B, H, Nq, d), lse=(B, H, Nq), dq=(B, H, Nq, d), dk=(B, Hkv, Nkv, d), dv=(B, Hkv, Nkv, d))
    return {n: r.reshape(shape[n]) for n, r in zip(names, res)}
