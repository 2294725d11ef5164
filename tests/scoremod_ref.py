"""Attention with modified scores from its definition in 64 bits (CPU), for the tests."""
import torch

NEG = float("-inf")


def visible(B, Nq, Nkv, causal, key_begin=None, key_end=None, kv_lens=None):
    p = torch.arange(Nq)[:, None] + (Nkv - Nq)
    j = torch.arange(Nkv)[None, :]
    see = (j <= p if causal else j >= 0).expand(B, Nq, Nkv).clone()
    if key_begin is not None:
        see &= j >= key_begin.cpu().long()[:, :, None]
    if key_end is not None:
        see &= j < key_end.cpu().long()[:, :, None]
    if kv_lens is not None:
        see &= j < kv_lens.cpu().long()[:, None, None]
    return see


def forward(q, k, v, causal, scale, softcap=0.0, slopes=None, key_begin=None, key_end=None, kv_lens=None):
    """o, lse, and the weights and tanh of the backward, all float64."""
    B, H, Nq, d = q.shape
    Hkv, Nkv = k.shape[1], k.shape[2]
    see = visible(B, Nq, Nkv, causal, key_begin, key_end, kv_lens)[:, None]
    rep = H // Hkv
    q64 = q.detach().cpu().double()
    k64, v64 = (t.detach().cpu().double().repeat_interleave(rep, 1) for t in (k, v))
    dead = ~(torch.arange(Nkv)[None, :] < (torch.full((B,), Nkv) if kv_lens is None else kv_lens.cpu().long())[:, None])
    k64 = k64.masked_fill(dead[:, None, :, None], 0.0)  # rows past the keys may hold anything
    v64 = v64.masked_fill(dead[:, None, :, None], 0.0)
    x = q64 @ k64.transpose(2, 3) * scale
    t = None
    if softcap:
        t = torch.tanh(x / softcap)
        x = softcap * t
    if slopes is not None:
        far = (torch.arange(Nq)[:, None] + (Nkv - Nq) - torch.arange(Nkv)).abs().double()
        x = x - slopes.cpu().double()[None, :, None, None] * far
    x = x.masked_fill(~see, NEG)
    lse = torch.logsumexp(x, -1)
    w = torch.exp(x - lse.nan_to_num(neginf=0.0)[..., None])
    return w @ v64, lse, w, t


def backward(q, k, v, dout, causal, scale, softcap=0.0, slopes=None, key_begin=None, key_end=None, kv_lens=None):
    B, H, Nq, d = q.shape
    Hkv, Nkv = k.shape[1], k.shape[2]
    o, lse, w, t = forward(q, k, v, causal, scale, softcap, slopes, key_begin, key_end, kv_lens)
    rep = H // Hkv
    dead = ~(torch.arange(Nkv)[None, :] < (torch.full((B,), Nkv) if kv_lens is None else kv_lens.cpu().long())[:, None])
    q64, g = q.detach().cpu().double(), dout.detach().cpu().double()
    k64, v64 = (x.detach().cpu().double().masked_fill(dead[:, None, :, None], 0.0).repeat_interleave(rep, 1) for x in (k, v))
    dv = w.transpose(2, 3) @ g
    ds = w * (g @ v64.transpose(2, 3) - (g * o).sum(-1, keepdim=True))
    if t is not None:
        ds = ds * (1 - t * t)
    ds = ds * scale
    dq, dk = ds @ k64, ds.transpose(2, 3) @ q64
    return dq, dk.view(B, Hkv, rep, Nkv, d).sum(2), dv.view(B, Hkv, rep, Nkv, d).sum(2)


def documents(B, Nq, Nkv, lens, seed=0):
    """key_begin, key_end [B, Nq] of documents of the given lengths (cycled, shifted per row of the batch)."""
    kb, ke = torch.zeros(B, Nq, dtype=torch.int32), torch.zeros(B, Nq, dtype=torch.int32)
    for b in range(B):
        edges, i = [0], b + seed
        while edges[-1] < Nkv:
            edges.append(min(Nkv, edges[-1] + lens[i % len(lens)]))
            i += 1
        e = torch.tensor(edges)
        p = torch.arange(Nq) + (Nkv - Nq)
        at = torch.searchsorted(e, p.clamp(min=0), right=True) - 1
        kb[b], ke[b] = e[at], e[at + 1]
    return kb, ke


def prefix(B, Nq, Nkv, lens):
    """key_end [B, Nq] of a prefix that all see and a causal rest."""
    p = torch.arange(Nq) + (Nkv - Nq)
    return torch.stack([torch.clamp(p + 1, min=int(lens[b % len(lens)])) for b in range(B)]).to(torch.int32)
