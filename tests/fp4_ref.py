"""The 4-bit page format from its definition (CPU): places of codes and scales, reading, writing, quantising."""
import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def places(d, value):
    """Byte and nibble shift of the code of (token, dim), and the byte of its block's scale: [16, d] each."""
    t, x = torch.arange(16)[:, None], torch.arange(d)[None, :]
    if value:
        q, h = t % 8 // 2, t // 8
        return 128 * (x // 16) + 32 * q + 16 * h + x % 16, (t % 2 * 4).expand(16, d), 8 * d + q * (d // 4) + 4 * (x // 16) + 2 * h + t % 2
    return t * (d // 2) + x // 2, (x % 2 * 4).expand(16, d), 8 * d + t * (d // 16) + x // 16


def read(pages, value):
    """Values [P, Hkv, 16, d] in float64 (without the tensor's scale) of pages [P, Hkv, 9 d]."""
    d = pages.shape[-1] // 9
    at, shift, sc = places(d, value)
    code = pages[..., at].int() >> shift & 15
    return torch.where(code >= 8, -1.0, 1.0) * GRID[code & 7] * pages[..., sc].view(torch.float8_e4m3fn).double()


def quantise(x, scale):
    """Codes [..., d] and scales [..., d / 16] (uint8) of fp32 x by the definition's fp32 steps."""
    u = x.float() * (torch.tensor(1.0) / torch.tensor(scale, dtype=torch.float32))
    u = u.unflatten(-1, (-1, 16))
    s = (u.abs().amax(-1) * torch.tensor(1.0 / 6.0, dtype=torch.float32)).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float()[..., None].expand(u.shape)
    y = torch.where(f > 0, u / f, torch.zeros_like(u)).double()
    m = y.abs()
    dist = (m[..., None] - GRID).abs()
    best = dist.amin(-1, keepdim=True)
    tied = dist == best  # two neighbours at a tie: the even one
    even = tied & (torch.arange(8) % 2 == 0)
    code = torch.where(even.any(-1), even.int().argmax(-1), tied.int().argmax(-1)).to(torch.uint8)
    return (code | (torch.signbit(y).to(torch.uint8) << 3)).flatten(-2), s.view(torch.uint8)


def write(pages, page, slot, codes, scales, value):
    """Stores the codes [Hkv, d] and scales [Hkv, d / 16] of one token."""
    d = codes.shape[-1]
    at, shift, sc = (p[slot] for p in places(d, value))
    for nib in (0, 4):
        i = shift == nib
        row = pages[page]  # a view
        row[:, at[i]] = (row[:, at[i]] & (0xF0 if nib == 0 else 0x0F)) | (codes[:, i] << nib)
    pages[page][:, sc[::16]] = scales


def pool(n, Hkv, d, seed, scale):
    """Key and value pages of normal values, and one page of NaN scales at the end; its number."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for value in (False, True):
        p = torch.full((n + 1, Hkv, 9 * d), 0x7F, dtype=torch.uint8)
        x = torch.randn(n, Hkv, 16, d, generator=g)
        codes, scales = quantise(x, scale)
        at, shift, sc = places(d, value)
        b = torch.zeros(n, Hkv, 9 * d, dtype=torch.uint8)
        for nib in (0, 4):
            i = (shift == nib).nonzero(as_tuple=True)
            b[:, :, at[i]] |= codes[:, :, i[0], i[1]] << nib
        t = torch.arange(16).repeat_interleave(d // 16)
        x16 = torch.arange(0, d, 16).repeat(16)
        b[:, :, sc[t, x16]] = scales.flatten(-2)
        p[:n] = b
        out.append(p)
    return out[0], out[1], n


def poison(k, v, page, first, last):
    """Slots first <= i < last of a page get scales of NaN and codes of all ones."""
    d = k.shape[-1] // 9
    for t, value in ((k, False), (v, True)):
        for slot in range(first, last):
            write(t, page, slot, torch.full((t.shape[1], d), 15, dtype=torch.uint8),
                  torch.full((t.shape[1], d // 16), 0x7F, dtype=torch.uint8), value)
