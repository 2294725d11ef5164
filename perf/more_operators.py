"""Cases of the operators around a 4-bit paged cache, with plain forms of each.

Five operators, reached through the package's entry points:

  decode4  paged_attn_decode_fp4: one query per sequence over a cache of e2m1 codes with an e4m3 scale per 16 dims.
  append   paged_kv_append_rope_axes(_fp8), paged_kv_append_fp4: new queries and keys are rotated by positions with
           several axes (time, height, width), keys and values go into the pages; a 4-bit cache's pages are then
           unpacked (paged_kv_unpack_fp4), as a chunked prefill over it reads them.
  rope     attn_rope_axes, attn_rope_axes_bwd: the rotation of a training step's queries and keys, and of their
           gradients.
  branch   paged_kv_fork, paged_kv_reserve, paged_kv_copy_pages: sequences continue others (samples, beams) or end,
           and get pages for their next tokens; a shared last page is copied.
  compact  paged_kv_compact, paged_kv_copy_pages: the pages in use move to the front of the pool.

``own = False`` computes a case with elementary torch operations in 32 bits; ``own = True`` makes the framework's
calls.  ``exact`` computes the same in 64 bits, written apart from both.
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
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # two users of a GPT-2-small-sized model with a distance bias: the call is all latency
        dict(name="decode4_b2", op="decode4", B=2, H=12, Hkv=12, d=64, ctx=900, cap=0.0, bias=True, window=0, lseed=1),
        # a serving batch with grouped heads and long contexts
        dict(name="decode4_b32", op="decode4", B=32, H=32, Hkv=8, d=128, ctx=8192, cap=0.0, bias=False, window=0, lseed=2),
        # one very long context, capped scores, a window that leaves the oldest tokens out
        dict(name="decode4_long_b1", op="decode4", B=1, H=32, Hkv=8, d=128, ctx=131072, cap=50.0, bias=False,
             window=120000, lseed=3),
        # one decode step of a small multimodal model over a 4-bit cache
        dict(name="append4_step_b4", op="append", B=4, N=1, H=12, Hkv=12, d=64, rope=64, inter=False, cache="fp4",
             axes=3, layout="sections", start=60, ragged=False, lseed=4),
        # a prompt with images, up to 1024 new tokens of eight sequences at once, into a 4-bit cache
        dict(name="append4_chunk_b8", op="append", B=8, N=1024, H=32, Hkv=8, d=128, rope=128, inter=False, cache="fp4",
             axes=3, layout="sections", start=500, ragged=True, lseed=5),
        # a decode step of a full batch into an e4m3 cache, the axes' frequencies interleaved
        dict(name="append_step_b128_fp8", op="append", B=128, N=1, H=32, Hkv=8, d=128, rope=128, inter=False, cache="fp8",
             axes=3, layout="cyclic", start=1500, ragged=False, lseed=6),
        # a vision tower: eight images of 32 x 32 patches, height and width, heads of 80
        dict(name="rope_images", op="rope", bwd=False, B=8, N=1024, H=16, Hkv=16, d=80, rope=80, inter=False, axes=2,
             layout="sections", lseed=7),
        # the gradients of a video's queries and keys, back into the fused projection's gradient
        dict(name="rope_video_bwd", op="rope", bwd=True, B=2, N=16384, H=32, Hkv=8, d=128, rope=128, inter=True, axes=3,
             layout="cyclic", lseed=8),
        # beam search, four requests of four beams
        dict(name="branch_beams_b16", op="branch", R=4, S=4, beams=True, Hkv=12, d=64, ctx=500, layers=2, spare=64, width=64,
             lseed=9),
        # sixteen samples of each of eight long prompts, eight layers
        dict(name="branch_samples_b128", op="branch", R=8, S=16, beams=False, Hkv=8, d=128, ctx=8000, layers=8, spare=8000,
             width=1024, lseed=10),
        # a small pool after a few users have left
        dict(name="compact_small", op="compact", B=8, pages=400, live=0.5, Hkv=12, d=64, layers=2, lseed=11),
        # a large pool at low use, before it shrinks
        dict(name="compact_large", op="compact", B=64, pages=16384, live=0.4, Hkv=8, d=128, layers=2, lseed=12),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(min(hi, max(lo, round(float(np.exp(rng.uniform(np.log(lo), np.log(hi + 1)) - 1e-9))))))


def draw(rng):
    op = rng.choice(("decode4", "append", "rope", "branch", "compact"))
    H, Hkv = rng.choice(HEADS)
    d = rng.choice(DIMS)
    case = dict(op=op, Hkv=Hkv, d=d, lseed=rng.randrange(1 << 30))
    if op == "decode4":
        ctx = _log(rng, 1, 65536)
        B = _log(rng, 1, max(1, min(128, 120_000_000 // (Hkv * ctx * d))))
        case |= dict(H=H, B=B, ctx=ctx, cap=rng.choice((0.0, 0.0, 30.0, 50.0)), bias=rng.random() < 0.3,
                     window=rng.choice((0, 0, max(1, ctx // 2))))
    elif op == "append":
        N = 1 if rng.random() < 0.4 else _log(rng, 2, 1024)
        B = _log(rng, 1, max(1, min(128, 8192 // N)))
        rope = rng.choice((d, d, d // 2))
        case |= dict(H=H, B=B, N=N, rope=d if rope % 16 else rope, inter=rng.random() < 0.5,
                     cache=rng.choice(("fp4", "fp4", "fp8", "bf16")), axes=rng.choice((1, 2, 3, 4)),
                     layout=rng.choice(("sections", "cyclic")), start=_log(rng, 1, 500), ragged=rng.random() < 0.5)
    elif op == "rope":
        N = _log(rng, 1, 16384)
        B = _log(rng, 1, max(1, min(64, 16384 // N)))
        rope = rng.choice((d, d, d // 2))
        case |= dict(H=H, bwd=rng.random() < 0.5, B=B, N=N, rope=d if rope % 16 else rope, inter=rng.random() < 0.5,
                     axes=rng.choice((1, 2, 3, 4)), layout=rng.choice(("sections", "cyclic")))
    elif op == "branch":
        S = _log(rng, 1, 32)
        R = _log(rng, 1, max(1, 128 // S))
        ctx = _log(rng, 1, 4000)
        beams = rng.random() < 0.5
        case |= dict(R=R, S=S, beams=beams, ctx=ctx, layers=_log(rng, 1, 4), spare=_log(rng, 1, 1000),
                     width=ctx // PAGE + 2 + _log(rng, 1, 100))
    else:
        B = _log(rng, 1, 64)
        case |= dict(B=B, pages=_log(rng, max(8, B), 8000), live=rng.choice((0.1, 0.4, 0.7, 0.95)), layers=_log(rng, 1, 2))
    return case


# ---------------------------------------------------------------- lengths, positions and tables of a case (seed-free)
def _lens(case, lo, hi, n, salt=0):
    r = random.Random(case["lseed"] * 7 + salt)
    return np.array([r.randint(lo, max(lo, hi)) for _ in range(n)], dtype=np.int64)


def _ctx(case):
    return _lens(case, max(1, case["ctx"] // 2 if case["B"] == 1 else case["ctx"] // 16), case["ctx"], case["B"], 4)


def _starts(case):
    return _lens(case, 0, case["start"], case["B"])


def _new(case):
    N = case["N"]
    return _lens(case, 0, N, case["B"], 1) if case["ragged"] else np.full(case["B"], N, dtype=np.int64)


def _positions(case):
    """Positions [axes, B, N] of text around images or frames: runs of text, whose axes advance together, and grids."""
    B, N, A = case["B"], case["N"], case["axes"]
    pos = np.zeros((A, B, N), dtype=np.int64)
    first = _starts(case) if case["op"] == "append" else np.zeros(B, dtype=np.int64)
    for b in range(B):
        r = random.Random(case["lseed"] * 13 + b)
        at, base = 0, int(first[b])
        while at < N:
            w, h, f = r.randint(4, 48), r.randint(4, 48), r.randint(1, 8)
            n = min(N - at, w * h * f)
            j = np.arange(n)
            grid = (j // (w * h), j // w % h, j % w)
            for a in range(A):
                pos[a, b, at:at + n] = base + (grid[a - A + 3] if 0 <= a - A + 3 < 3 else j * 0)
            at, base = at + n, base + max(w, h, f)
            n = min(N - at, r.randint(1, 100))
            pos[:, b, at:at + n] = base + np.arange(n)
            at, base = at + n, base + n
    return pos


def _pair_axis(case):
    """The axis of each of the rope / 2 pairs: contiguous sections, or one axis after the other."""
    half, A = case["rope"] // 2, case["axes"]
    i = np.arange(half)
    return bytes((i * A // half if case["layout"] == "sections" else i % A).tolist())


def _branch(case):
    """Tables [B, width] of page numbers 0, 1, ... (-1: none), tokens and parents of a branching step, and the pages used."""
    R, S, W = case["R"], case["S"], case["width"]
    r = random.Random(case["lseed"] * 17)
    table, ctx = np.full((R * S, W), -1, dtype=np.int64), np.zeros(R * S, dtype=np.int64)
    parents, used = np.zeros(R * S, dtype=np.int64), 0
    for q in range(R):
        n = r.randint(max(1, case["ctx"] // 2), case["ctx"])
        pages = -(-n // PAGE)
        if case["beams"]:  # the beams share all pages but the last few, which each has of its own
            tail = min(pages, r.randint(1, 4))
            for k in range(S):
                table[q * S + k, :pages - tail] = used + np.arange(pages - tail)
                table[q * S + k, pages - tail:pages] = used + pages - tail + k * tail + np.arange(tail)
                ctx[q * S + k] = n
                parents[q * S + k] = q * S + r.randrange(S)
            used += pages - tail + S * tail
        else:  # the prompt sits in the first row
            table[q * S, :pages] = used + np.arange(pages)
            ctx[q * S], parents[q * S:q * S + S] = n, q * S
            used += pages
    if R * S > 3:
        parents[r.randrange(R * S)] = -1  # one has ended
    return table, ctx, parents, used


def _compact_table(case):
    """Table [B, width] over scattered pages: a part of the pool is live, some of it in several rows."""
    B, P = case["B"], case["pages"]
    r = np.random.RandomState(case["lseed"] % (1 << 31))
    live = r.permutation(P)[:max(1, int(P * case["live"]))]
    rows = np.array_split(live, B)
    shared = rows[0][:len(rows[0]) // 2]
    width = max(len(x) for x in rows) + len(shared) + 3
    table = np.full((B, width), -1, dtype=np.int64)
    for b, x in enumerate(rows):
        x = np.concatenate([shared, x]) if b % 2 else x
        table[b, :len(x)] = x
    return table


def _moves(table, P):
    ref = np.bincount(table[table >= 0], minlength=P)
    live = np.nonzero(ref > 0)[0]
    return int((live >= len(live)).sum())


def work(case):
    Hkv, d = case["Hkv"], case["d"]
    if case["op"] == "decode4":
        ctx, H, B = _ctx(case), case["H"], case["B"]
        seen = int((np.minimum(ctx, case["window"]) if case["window"] else ctx).sum())
        return {"bytes": seen * 2 * Hkv * (9 * d // 16) + 4 * B * H * d + 4 * B * H, "flops": 4 * H * d * seen}
    if case["op"] == "append":
        t, H = int(_new(case).sum()), case["H"]
        e = {"bf16": 2 * d, "fp8": d, "fp4": 9 * d // 16}[case["cache"]]
        b = t * (4 * H * d + 2 * Hkv * (2 * d + e) + 4 * case["axes"])
        if case["cache"] == "fp4":
            pages = int(np.maximum(1, -(-(_starts(case) + case["N"]) // PAGE)).sum())
            b += pages * Hkv * 2 * PAGE * (9 * d // 16 + 2 * d)
        return {"bytes": b, "flops": 3 * t * (H + Hkv) * case["rope"]}
    if case["op"] == "rope":
        t = case["B"] * case["N"]
        return {"bytes": t * (4 * (case["H"] + Hkv) * d + 4 * case["axes"]), "flops": 3 * t * (case["H"] + Hkv) * case["rope"]}
    page = PAGE * Hkv * d * 2 * 2 * case["layers"]  # of all pools
    if case["op"] == "branch":
        table, ctx, parents, used = _branch(case)
        new = np.where(parents >= 0, ctx[parents.clip(0)], 0)
        copies = int(((new % PAGE != 0) & (parents >= 0)).sum()) if case["S"] > 1 else 0
        return {"bytes": 2 * copies * page + 8 * table.size + 8 * (used + case["spare"]), "flops": 0}
    table = _compact_table(case)
    return {"bytes": 2 * _moves(table, case["pages"]) * page + 8 * table.size + 8 * case["pages"], "flops": 0}


# ---------------------------------------------------------------- the 4-bit page format
def _quantise(x, scale):
    """Codes (uint8, one a value) and e4m3 block scales (uint8) of x [..., d] in 32 bits."""
    u = x * (1.0 / torch.tensor(scale, dtype=torch.float32, device=DEV))
    u = u.unflatten(-1, (-1, 16))
    s = (u.abs().amax(-1) * torch.tensor(1.0 / 6.0, dtype=torch.float32, device=DEV)).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float()[..., None]
    y = torch.where(f > 0, u / torch.where(f > 0, f, torch.ones_like(f)), torch.zeros_like(u))
    m = y.abs()
    code = torch.zeros_like(y, dtype=torch.uint8)
    for edge, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (m >= edge) if up else (m > edge)  # ties go to the even code
    return (code | (torch.signbit(y).to(torch.uint8) << 3)).flatten(-2), s.view(torch.uint8)


def _pack(codes, scales, value):
    """Pages [P, Hkv, 9 d] of codes [P, Hkv, 16, d] and scales [P, Hkv, 16, d / 16]; value: the values' form."""
    P, h, _, d = codes.shape
    if value:  # blocks of 16 dims; quads of tokens 2t, 2t + 1, 2t + 8, 2t + 9, a pair of them in a byte
        c = codes.view(P, h, 2, 4, 2, d // 16, 16).permute(0, 1, 5, 3, 2, 6, 4)
        s = scales.view(P, h, 2, 4, 2, d // 16).permute(0, 1, 3, 5, 2, 4)
    else:
        c, s = codes.view(P, h, 16, d // 2, 2), scales
    return torch.cat([(c[..., 0] | (c[..., 1] << 4)).reshape(P, h, 8 * d), s.reshape(P, h, d)], -1)


def _unpack(pages, d, value):
    """Codes and scales of pages, the inverse of _pack."""
    P, h, _ = pages.shape
    b, s = pages[..., :8 * d], pages[..., 8 * d:]
    if value:
        c = torch.stack([b & 15, b >> 4], -1).view(P, h, d // 16, 4, 2, 16, 2).permute(0, 1, 4, 3, 6, 2, 5)
        return c.reshape(P, h, 16, d), s.reshape(P, h, 4, d // 16, 2, 2).permute(0, 1, 4, 2, 5, 3).reshape(P, h, 16, d // 16)
    return torch.stack([b & 15, b >> 4], -1).view(P, h, 16, d), s.reshape(P, h, 16, d // 16)


def _values(codes, scales, scale):
    """The values of codes [..., d] under their scales, in 32 bits."""
    of = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=DEV)
    x = of[codes.int()].unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]
    return x.flatten(-2) * scale


# ---------------------------------------------------------------- inputs
def _i32(a):
    return None if a is None else torch.tensor(np.ascontiguousarray(a), dtype=torch.int32, device=DEV)


def _pool4(case, g, pages):
    shape, r = (pages, case["Hkv"], PAGE, case["d"]), []
    for value, scale in ((False, 0.0113), (True, 0.00871)):
        parts = []
        for p in range(0, pages, 2048):
            x = torch.randn((min(2048, pages - p),) + shape[1:], generator=g, device=DEV)
            parts.append(_pack(*_quantise(x, scale), value))
        r.append(torch.cat(parts))
    return r


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
    Hkv, d = case["Hkv"], case["d"]
    s = dict(case=case, scale=d ** -0.5, k_scale=0.0113, v_scale=0.00871)

    def normal(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=g)

    if case["op"] == "decode4":
        ctx, H = _ctx(case), case["H"]
        s["table"], total = _table(g, -(-ctx // PAGE))
        s["k_pages"], s["v_pages"] = _pool4(case, g, total)
        s["q"], s["ctx"] = normal(case["B"], H, d), _i32(ctx)
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device=DEV) if case["bias"] else None
        s["begin"] = _i32(ctx - case["window"]) if case["window"] else None
        return s
    if case["op"] in ("append", "rope"):
        B, N, H, r = case["B"], case["N"], case["H"], case["rope"]
        pos = _positions(case)
        s["positions"], s["pair_axis"] = _i32(pos), _pair_axis(case)
        s["axis"] = torch.tensor(list(s["pair_axis"]), device=DEV)
        angle = torch.arange(int(pos.max()) + 1, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, r, 2, dtype=torch.float64) / r)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().to(DEV)
    if case["op"] == "append":
        start, new = _starts(case), _new(case)
        s["table"], total = _table(g, np.maximum(1, -(-(start + N) // PAGE)))
        if case["cache"] == "fp4":
            s["k_pages"], s["v_pages"] = _pool4(case, g, total)
            s["ids"] = torch.arange(total, dtype=torch.int32, device=DEV)
            s["bits"] = [torch.empty(total, Hkv, PAGE, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        else:
            x = [normal(total, Hkv, PAGE, d) for _ in range(2)]
            if case["cache"] == "fp8":
                x = [(t.float() / c).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for t, c in zip(x, (0.0113, 0.00871))]
            s["k_pages"], s["v_pages"] = x
        # the projection's output, [B, N, (H + 2 Hkv) d]; queries, keys and values are views of it
        qkv = normal(B, N, H + 2 * Hkv, d).transpose(1, 2)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        s["q_out"] = torch.zeros(B, H, N, d, dtype=torch.bfloat16, device=DEV)
        s["start"], s["new"] = _i32(start), _i32(new) if case["ragged"] else None
    elif case["op"] == "rope":
        qkv = torch.zeros(B, N, H + 2 * Hkv, d, dtype=torch.bfloat16, device=DEV) if case["bwd"] else normal(B, N, H + 2 * Hkv, d)
        qkv = qkv.transpose(1, 2)
        dense = normal(B, H, N, d), normal(B, Hkv, N, d)
        views = qkv[:, :H], qkv[:, H:H + Hkv]
        s["q"], s["k"] = dense if case["bwd"] else views
        s["q_out"], s["k_out"] = views if case["bwd"] else (torch.empty_like(dense[0]), torch.empty_like(dense[1]))
    else:
        if case["op"] == "branch":
            table, ctx, parents, used = _branch(case)
            s["P"] = used + case["spare"]
            s["ctx"], s["parents"] = _i32(ctx), _i32(parents)
            s["new"] = _i32((parents >= 0).astype(np.int64))
            ids = torch.randperm(s["P"], generator=g, device=DEV).to(torch.int32)
        else:
            table, s["P"] = _compact_table(case), case["pages"]
            ids = torch.randperm(s["P"], generator=g, device=DEV).to(torch.int32)
        t = _i32(table)
        s["table"] = torch.where(t >= 0, ids[t.clamp(min=0).long()], t).contiguous()
        s["ref"] = torch.zeros(s["P"] + 1, dtype=torch.int32, device=DEV).index_add_(
            0, torch.where(s["table"] >= 0, s["table"], s["P"]).flatten(), torch.ones(t.numel(), dtype=torch.int32, device=DEV))[:-1].clone()
        s["pools"] = [normal(s["P"], Hkv, PAGE, d) for _ in range(2 * case["layers"])]
    return s


# ---------------------------------------------------------------- plain forms, 32 bits
def _softmax(x):
    """Weights over the last axis and the log of their sum; rows that see nothing have weights 0 and -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == NEG, torch.zeros_like(m), m)
    e = (x - m).exp()
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total)), (m + total.log()).squeeze(-1)


def _decode4(s):
    c = s["case"]
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]

    def pages(pool, scale, value):
        x = _values(*_unpack(pool[s["table"].flatten().long()], d, value), scale)
        return x.view(B, -1, Hkv, PAGE, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)

    k = pages(s["k_pages"], s["k_scale"], False)
    x = torch.matmul(s["q"].float().view(B, Hkv, H // Hkv, d), k.transpose(2, 3)) * s["scale"]
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    j, ctx = torch.arange(k.shape[2], device=DEV), s["ctx"].long()[:, None]
    if c["bias"]:
        x = x - s["slopes"].view(1, Hkv, H // Hkv, 1) * (ctx - 1 - j).float()[:, None, None]
    see = j < ctx
    if s["begin"] is not None:
        see = see & (j >= s["begin"][:, None])
    p, lse = _softmax(x.masked_fill(~see[:, None, None], NEG))
    v = pages(s["v_pages"], s["v_scale"], True)
    return dict(o=torch.matmul(p, v).reshape(B, H, d).to(torch.bfloat16), lse=lse.reshape(B, H))


def _turn(s, x, back=False):
    """x [B, heads, N, d] in 32 bits, its first rope dims turned by their pairs' positions (back: the transpose)."""
    c, half = s["case"], s["case"]["rope"] // 2
    row = s["positions"].long()[s["axis"]]  # [pairs, B, N]
    pair = torch.arange(half, device=DEV)[:, None, None]
    cos, sin = (s["cos_sin"][row, pair + h].permute(1, 2, 0)[:, None] for h in (0, half))
    sin = -sin if back else sin
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if c["inter"] else (x[..., :half], x[..., half:2 * half])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if c["inter"] else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _append(s):
    c = s["case"]
    N, d = c["N"], c["d"]
    at = s["start"].long()[:, None] + torch.arange(N, device=DEV)
    valid = torch.ones_like(at, dtype=torch.bool) if s["new"] is None else torch.arange(N, device=DEV) < s["new"][:, None]
    b, t = valid.nonzero(as_tuple=True)
    page, slot = s["table"][b, at[b, t] // PAGE].long(), at[b, t] % PAGE
    out = {}
    for name, x, scale in (("k_pages", _turn(s, s["k_new"].float()), s["k_scale"]), ("v_pages", s["v_new"].float(), s["v_scale"])):
        rows, pool, value = x[b, :, t], s[name], name == "v_pages"
        if c["cache"] == "fp4":
            codes, scales = _unpack(pool, d, value)
            codes[page, :, slot], scales[page, :, slot] = _quantise(rows, scale)
            pool.copy_(_pack(codes, scales, value))
            out[name] = _values(codes, scales, scale).to(torch.bfloat16)
        elif c["cache"] == "fp8":
            rows = rows * (1.0 / torch.tensor(scale, dtype=torch.float32, device=DEV))
            pool[page, :, slot] = rows.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            out[name] = pool.view(torch.float8_e4m3fn)
        else:
            pool[page, :, slot] = rows.to(torch.bfloat16)
            out[name] = pool
    s["q_out"].copy_(torch.where(valid[:, None, :, None], _turn(s, s["q"].float()).to(torch.bfloat16), s["q_out"]))
    return out | dict(q=s["q_out"])


def _rope(s):
    s["q_out"].copy_(_turn(s, s["q"].float(), s["case"]["bwd"]))
    s["k_out"].copy_(_turn(s, s["k"].float(), s["case"]["bwd"]))
    return dict(q=s["q_out"], k=s["k_out"])


def _count(table, P):
    """How many entries of a table name each page."""
    at = torch.where(table >= 0, table, P).flatten().long()
    return torch.zeros(P + 1, dtype=torch.int32, device=DEV).index_add_(0, at, torch.ones_like(at, dtype=torch.int32))[:-1]


def _copy(pools, src, dst):
    ok = src >= 0
    src, dst = src[ok].long(), dst[ok].long()
    for p in pools:
        p[dst] = p[src]


def _branch_plain(s):
    table, ctx, ref, P = s["table"], s["ctx"], s["ref"], s["P"]
    B, W = table.shape
    col = torch.arange(W, device=DEV)
    # the fork
    own_row, par = s["parents"] == torch.arange(B, device=DEV), s["parents"].clamp(min=0).long()
    n = torch.where(s["parents"] >= 0, ctx[par], torch.zeros_like(ctx))
    forked = torch.where(col < (n[:, None] + PAGE - 1) // PAGE, table[par], -1)
    t2 = torch.where(own_row[:, None], table, forked).int()
    ref2 = ref + _count(t2, P) - _count(table, P)
    # pages for the next tokens: the entries that cover them become the row's own
    to = (n + s["new"] + PAGE - 1) // PAGE
    wanted = (s["new"] > 0) & (to <= W)
    shared = (t2 >= 0) & (ref2[t2.clamp(min=0).long()] > 1)
    alloc = (col >= (n // PAGE)[:, None]) & (col < to[:, None]) & ((t2 < 0) | shared) & wanted[:, None]
    need = alloc.sum(1)
    end = need.cumsum(0)
    free = ref2 <= 0
    ok = wanted & ((need == 0) | (end <= free.sum()))
    rank = torch.where(free, free.cumsum(0) - 1, P)
    ids = torch.zeros(P + 1, dtype=torch.int32, device=DEV).scatter_(0, rank, torch.arange(P, dtype=torch.int32, device=DEV))
    fresh = alloc & ok[:, None]
    t3 = torch.where(fresh, ids[((end - need)[:, None] + alloc.cumsum(1) - 1).clamp(0, P)], t2)
    ref3 = ref2 + _count(t3, P) - _count(t2, P)
    tail = (n // PAGE).clamp(max=W - 1).long()[:, None]
    copied = (n % PAGE != 0) & (fresh & shared).gather(1, tail)[:, 0]
    src = torch.where(copied, t2.gather(1, tail)[:, 0], -1)
    dst = torch.where(copied, t3.gather(1, tail)[:, 0], -1)
    _copy(s["pools"], src, dst)
    return dict(table=t3, ctx=n, ref=ref3, reserved=torch.where(ok, s["new"], 0), src=src, dst=dst, pools=s["pools"])


def _compact_plain(s):
    table, ref, P = s["table"], s["ref"], s["P"]
    live = ref > 0
    L = live.sum()
    i = torch.arange(P, device=DEV)
    hole, mover = ~live & (i < L), live & (i >= L)

    def listing(mask):
        r = torch.where(mask, mask.cumsum(0) - 1, P)
        return torch.full((P + 1,), -1, dtype=torch.int32, device=DEV).scatter_(0, r, torch.where(mask, i, -1).int())[:P]

    src, dst = listing(mover), listing(hole)
    to = torch.where(live & (i < L), i, -1).int()
    to = torch.cat([to, to.new_full((1,), -1)]).scatter_(0, torch.where(src >= 0, src, P).long(), dst)[:P]
    t2 = torch.where(table >= 0, to[table.clamp(min=0).long()], -1)
    ref2 = torch.where(i < L, ref, 0)
    ref2 = torch.cat([ref2, ref2.new_zeros(1)]).scatter_(0, torch.where(dst >= 0, dst, P).long(), ref[src.clamp(min=0).long()])[:P]
    _copy(s["pools"], src, dst)
    return dict(table=t2, ref=ref2, src=src, dst=dst, count=mover.sum().int().reshape(1), pools=s["pools"])


PLAIN = dict(decode4=_decode4, append=_append, rope=_rope, branch=_branch_plain, compact=_compact_plain)


# ---------------------------------------------------------------- the framework's calls
def _calls(s):
    import attn_fwd_02_gb300 as A
    c = s["case"]
    scales = (s["k_scale"], s["v_scale"])
    if c["op"] == "decode4":
        o, lse = A.paged_attn_decode_fp4(s["q"], s["k_pages"], s["v_pages"], *scales, s["table"], s["ctx"], s["scale"],
                                         softcap=c["cap"], alibi_slopes=s["slopes"], key_begin=s["begin"])
        return dict(o=o, lse=lse)
    if c["op"] == "append":
        new = (s["q"], s["k_new"], s["v_new"], s["k_pages"], s["v_pages"])
        if c["cache"] == "fp4":
            A.paged_kv_append_fp4(*new, *scales, s["table"], s["start"], cos_sin=s["cos_sin"], positions=s["positions"],
                                  pair_axis=s["pair_axis"], interleaved=c["inter"], new_lens=s["new"], q_out=s["q_out"])
            k, v = A.paged_kv_unpack_fp4(s["k_pages"], s["v_pages"], *scales, s["ids"], k_out=s["bits"][0], v_out=s["bits"][1])
            return dict(q=s["q_out"], k_pages=k, v_pages=v)
        rest = (s["cos_sin"], s["positions"], s["pair_axis"], s["table"], s["start"])
        more = dict(interleaved=c["inter"], new_lens=s["new"], q_out=s["q_out"])
        if c["cache"] == "fp8":
            A.paged_kv_append_rope_axes_fp8(*new, *scales, *rest, **more)
            return dict(q=s["q_out"], k_pages=s["k_pages"].view(torch.float8_e4m3fn), v_pages=s["v_pages"].view(torch.float8_e4m3fn))
        A.paged_kv_append_rope_axes(*new, *rest, **more)
        return dict(q=s["q_out"], k_pages=s["k_pages"], v_pages=s["v_pages"])
    if c["op"] == "rope":
        f = A.attn_rope_axes_bwd if c["bwd"] else A.attn_rope_axes
        q, k = f(s["q"], s["k"], s["cos_sin"], s["positions"], s["pair_axis"], interleaved=c["inter"], q_out=s["q_out"], k_out=s["k_out"])
        return dict(q=q, k=k)
    if c["op"] == "branch":
        table, ctx, ref = A.paged_kv_fork(s["table"], s["ctx"], s["parents"], s["ref"])
        table, ref, reserved, src, dst = A.paged_kv_reserve(table, ctx, s["new"], ref)
        A.paged_kv_copy_pages(s["pools"], src, dst)
        return dict(table=table, ctx=ctx, ref=ref, reserved=reserved, src=src, dst=dst, pools=s["pools"])
    table, ref, src, dst, count = A.paged_kv_compact(s["table"], s["ref"])
    A.paged_kv_copy_pages(s["pools"], src, dst, count=count)
    return dict(table=table, ref=ref, src=src, dst=dst, count=count, pools=s["pools"])


def run(s):
    return _calls(s) if own else PLAIN[s["case"]["op"]](s)


# ---------------------------------------------------------------- 64 bits
def _round4(u):
    """Values and block scales of u [..., 16] (in units of the tensor's scale) by nearest search, ties to the even code."""
    e4 = torch.arange(127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()

    def nearest(x, grid):  # x >= 0: index of the nearest value of the ascending grid, ties to the even index
        hi = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
        lo = hi - 1
        down, up = x - grid[lo], grid[hi] - x
        return torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)

    sc = e4[nearest(u.abs().amax(-1) / 6, e4)][..., None]
    grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    y = grid[nearest(torch.where(sc > 0, u.abs() / sc, torch.zeros_like(u)), grid)]
    return torch.copysign(y, u) * sc


def exact(case, seed):
    """The operators from their definitions, one sequence at a time."""
    s = prepare(case, seed)
    f, d, Hkv = torch.float64, case["d"], case["Hkv"]

    def read4(pool, value):
        """The pool's values, without the tensor's scale, by the place of each nibble and scale: [P, Hkv, 16, d]."""
        t, x = torch.arange(16, device=DEV)[:, None], torch.arange(d, device=DEV)[None, :]
        quad, half = t % 8 // 2, t // 8
        at = x // 16 * 128 + quad * 32 + half * 16 + x % 16 if value else t * (d // 2) + x // 2
        high = (t if value else x) % 2 * 4
        sc = 8 * d + (quad * (d // 4) + x // 16 * 4 + half * 2 + t % 2 if value else t * (d // 16) + x // 16)
        b = pool.flatten(0, 1)
        code = (b[:, at.expand(16, d).flatten()].view(-1, 16, d) >> high.to(torch.uint8)) & 15
        mag = torch.tensor(E2M1, dtype=f, device=DEV)[(code & 7).int()]
        sf = b[:, sc.expand(16, d).flatten()].view(torch.float8_e4m3fn).view(-1, 16, d).to(f)
        return (torch.where(code >= 8, -mag, mag) * sf).view(*pool.shape[:2], 16, d)

    if case["op"] == "decode4":
        B, H = case["B"], case["H"]
        ctx, gp = _ctx(case), H // Hkv
        o, l = torch.zeros(B, H, d, dtype=f, device=DEV), torch.zeros(B, H, dtype=f, device=DEV)
        for b in range(B):
            n = int(ctx[b])
            lo = max(0, n - case["window"]) if case["window"] else 0
            j = torch.arange(lo, n, device=DEV)
            ids = s["table"][b, :-(-n // PAGE)].long()
            k, v = (read4(s[p][ids], p == "v_pages").transpose(0, 1).reshape(Hkv, -1, d)[:, lo:n] * s[p[0] + "_scale"]
                    for p in ("k_pages", "v_pages"))
            x = torch.einsum("hgd,hnd->hgn", s["q"][b].to(f).view(Hkv, gp, d), k) * s["scale"]
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if case["bias"]:
                x = x - s["slopes"].to(f).view(Hkv, gp, 1) * (n - 1 - j)
            l[b] = torch.logsumexp(x, -1).view(H)
            o[b] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), v).reshape(H, d)
        return dict(o=o, lse=l)

    if case["op"] in ("append", "rope"):
        B, N, half = case["B"], case["N"], case["rope"] // 2
        i = torch.arange(half, device=DEV)
        first, second = (2 * i, 2 * i + 1) if case["inter"] else (i, i + half)

        def turned(x, b, back=False):
            """x [heads, N, d] of sequence b, as complex numbers times those of the angles."""
            x, p = x.to(f), s["positions"][:, b].long()
            z = torch.stack([torch.complex(s["cos_sin"][p[s["pair_axis"][k]], k].to(f), s["cos_sin"][p[s["pair_axis"][k]], half + k].to(f))
                             for k in range(half)], -1)
            w = torch.complex(x[..., first], x[..., second]) * (z.conj() if back else z)
            x[..., first], x[..., second] = w.real, w.imag
            return x

        if case["op"] == "rope":
            return {n: torch.stack([turned(s[n][b], b, case["bwd"]) for b in range(B)]) for n in ("q", "k")}
        start, new, qo, out = _starts(case), _new(case), s["q_out"].to(f), {}
        for name in ("k_pages", "v_pages"):
            if case["cache"] == "fp4":
                out[name] = read4(s[name], name == "v_pages") * s[name[0] + "_scale"]
            else:
                out[name] = (s[name].view(torch.float8_e4m3fn) if case["cache"] == "fp8" else s[name]).to(f)
        for b in range(B):
            n = int(new[b])
            at = torch.arange(int(start[b]), int(start[b]) + n, device=DEV)
            page, slot = s["table"][b][at // PAGE].long(), at % PAGE
            qo[b, :, :n] = turned(s["q"][b], b)[:, :n]
            for name, x in (("k_pages", turned(s["k_new"][b], b)), ("v_pages", s["v_new"][b].to(f))):
                rows, scale = x[:, :n].transpose(0, 1), s[name[0] + "_scale"]
                if case["cache"] == "fp4":
                    rows = _round4((rows / scale).unflatten(-1, (-1, 16))).flatten(-2) * scale
                elif case["cache"] == "fp8":
                    rows = (rows / scale).clamp(-448, 448)
                out[name][page, :, slot] = rows
        return out | dict(q=qo)
    # whole numbers and copies: the pages' contents, moved one at a time
    if case["op"] == "branch":
        table, ctx, parents, ref = (s[n].tolist() for n in ("table", "ctx", "parents", "ref"))
        P, W, rows, src, dst = s["P"], len(table[0]), [], [], []
        for b, p in enumerate(parents):
            keep = -(-ctx[p] // PAGE) if p >= 0 else 0
            rows.append(list(table[b]) if p == b else [table[p][j] if j < keep else -1 for j in range(W)])
        for t, sign in ((rows, 1), (table, -1)):
            for r in t:
                for e in r:
                    if e >= 0:
                        ref[e] += sign
        lens, free, frozen, asked = [ctx[p] if p >= 0 else 0 for p in parents], [i for i in range(P) if ref[i] <= 0], list(ref), 0
        for b, n in enumerate(lens):
            lp, to = n // PAGE, -(-(n + int(s["new"][b])) // PAGE)
            if not int(s["new"][b]) or to > W:
                continue
            new = [j for j in range(lp, to) if rows[b][j] < 0 or frozen[rows[b][j]] > 1]
            asked += len(new)
            if new and asked <= len(free) and n % PAGE and new[0] == lp and rows[b][lp] >= 0:
                src.append(rows[b][lp])
                dst.append(free[asked - len(new)])
    else:
        live = torch.nonzero(s["ref"] > 0)[:, 0]
        L = len(live)
        src = live[live >= L].tolist()
        dst = torch.nonzero(s["ref"][:L] <= 0)[:, 0].tolist()
    pools = [p.double() if p.numel() < 1 << 28 else p.float() for p in s["pools"]]
    for p in pools:
        p[dst] = p[src]
    return dict(pools=pools)
