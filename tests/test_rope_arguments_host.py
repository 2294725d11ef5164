"""Arguments of the rotation by several axes on the host: what names the pairs' axes, and outputs whose rows overlap."""
import array
import ctypes

import numpy as np
import pytest
import torch

A = 1 << 20  # fake, 16-byte aligned addresses: the checks fail before any use


@pytest.fixture(scope="module")
def binding():
    from attn_fwd_02_gb300 import binding as b
    from attn_fwd_02_gb300 import build as buildmod
    buildmod.build()
    return b


AXES = [0, 1, 2, 1] * 8


def axes_in(b, monkeypatch, pair):
    b._torch()
    monkeypatch.setattr(b, "_in", lambda *a, **k: A)
    return b._axes_in(torch.zeros(3, 2, 5, dtype=torch.int32), pair, 2, 5, torch.zeros(9, 64), None)


@pytest.mark.parametrize("pair", [bytes(AXES), AXES, tuple(AXES), bytearray(AXES), np.array(AXES), np.array(AXES, np.uint8),
                                  torch.tensor(AXES), array.array("i", AXES), range(0, 32)],
                         ids=["bytes", "list", "tuple", "bytearray", "numpy", "numpy8", "torch", "array", "range"])
def test_every_sequence_of_axis_numbers(binding, monkeypatch, pair):
    assert axes_in(binding, monkeypatch, pair) == (A, 3, bytes(range(32)) if isinstance(pair, range) else bytes(AXES))


@pytest.mark.parametrize("pair", [32, True, "0" * 32, None, [0.0] * 32, ["0"] * 32, [-1] * 32, [256] * 32, np.zeros(32), 1.5, np.int64(32)],
                         ids=["int", "bool", "str", "none", "floats", "strs", "negative", "large", "numpy_floats", "float", "numpy_int"])
def test_what_is_not_one(binding, monkeypatch, pair):
    with pytest.raises(TypeError, match="pair_axis"):
        axes_in(binding, monkeypatch, pair)


@pytest.mark.parametrize("pair", [AXES[:-1], AXES + [0], [], np.array(AXES[:4], np.int64)], ids=["few", "many", "none", "numpy_bytes"])
def test_its_length(binding, monkeypatch, pair):
    with pytest.raises(ValueError, match="pair_axis"):
        axes_in(binding, monkeypatch, pair)
