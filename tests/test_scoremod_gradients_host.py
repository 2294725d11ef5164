"""The 64-bit backward that the GPU tests compare with, itself against central differences, without a GPU."""
import pytest
import torch

from scoremod_ref import backward, documents, forward


@pytest.mark.parametrize("cap", [0.0, 2.0])
@pytest.mark.parametrize("slopes", [None, [0.5, 0.03, 40.0, -0.2]], ids=["no_bias", "bias"])
@pytest.mark.parametrize("causal", [False, True])
def test_gradients_match_differences(causal, slopes, cap):
    torch.manual_seed(1)
    B, H, Hkv, Nq, Nkv, d = 2, 4, 2, 4, 6, 32
    q, k, v = (torch.randn(B, h, n, d, dtype=torch.float64) for h, n in ((H, Nq), (Hkv, Nkv), (Hkv, Nkv)))
    g = torch.randn(B, H, Nq, d, dtype=torch.float64)
    kb, ke = documents(B, Nq, Nkv, [3, 2])
    args = (causal, 0.3, cap, None if slopes is None else torch.tensor(slopes), kb, ke, torch.tensor([5, 6]))
    loss = lambda: float((forward(q, k, v, *args)[0] * g).sum())  # noqa: E731
    for x, dx in zip((q, k, v), backward(q, k, v, g, *args)):
        flat, dflat = x.view(-1), dx.reshape(-1)
        for i in range(0, flat.numel(), 29):
            old, h = float(flat[i]), 1e-5
            flat[i] = old + h
            up = loss()
            flat[i] = old - h
            down = loss()
            flat[i] = old
            # the third derivative's h^2 / 6 and the sum's 2^-52 / h, of values of a few hundred at most
            assert abs((up - down) / (2 * h) - float(dflat[i])) <= 1e-7
