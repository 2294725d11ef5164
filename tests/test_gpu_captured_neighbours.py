"""Captured calls whose neighbours in the graph are copies, fills and the work of another stream: kernels that may start while
the one before them drains still wait for all of these."""
import pytest
import torch

from test_gpu_more_marshalling import NAMES, calls, lib, tensors  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("before", ["copies", "fill", "join", "kernel"])
@pytest.mark.parametrize("name", NAMES)
def test_a_captured_call_waits_for_what_precedes_it(lib, name, before):  # noqa: F811
    args, kw, _ = calls()[name]
    result = getattr(lib, name)(*args, **kw)
    torch.cuda.synchronize()
    want = [t.clone() for t in tensors([result, args, kw])]  # what it returns and writes
    args, kw, _ = calls()[name]
    live = [t for t in tensors([args, kw])]
    kept = [t.clone() for t in live]
    big = torch.zeros(1 << 26, device="cuda")  # what the preceding work also takes its time with
    other = torch.ones_like(big)
    side = torch.cuda.Stream()

    def stage():
        big.copy_(other)
        for t, k in zip(live, kept):
            t.copy_(k)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if before == "join":
            side.wait_stream(torch.cuda.current_stream())
            big.add_(1.0)
            with torch.cuda.stream(side):
                stage()
            torch.cuda.current_stream().wait_stream(side)
        else:
            stage()
            if before == "fill":
                big.zero_()
            elif before == "kernel":
                big.mul_(2.0)
        result = getattr(lib, name)(*args, **kw)
        big.copy_(other)  # and what follows waits for it
        after = [t.clone() for t in tensors([result, args, kw])]
    for turn in range(3):
        for t in live:
            t.zero_()
        for t in after:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(after, want)), (name, before, turn)
    assert lib.attn_check_device_status() == 0
