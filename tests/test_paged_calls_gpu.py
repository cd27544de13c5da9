"""How the paged cache's operators may be called: scales that are not Python floats, calls captured without a workspace
or an output of their own, and behind work of other streams."""
import numpy as np
import pytest
import torch

import test_paged_attn_gpu as paged
import test_prompt_attn_gpu as prompt
from test_paged_workspace_gpu import cut_pairs

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("kind", [np.float32, np.float64, torch.tensor, lambda x: torch.tensor(x, device="cuda")])
def test_scales_that_are_not_python_floats(dtlib, kind):
    """As dt_tree_attention takes them."""
    s, p = paged.make([70, 20], 2, 8, 2, 64, 16, mask="tree"), prompt.make([70], 4, 2, 64)
    s["scale"] = p["scale"] = 0.125
    want = paged.run(dtlib, s).clone(), prompt.run(dtlib, p).clone()
    s["scale"] = p["scale"] = kind(0.125)
    assert torch.equal(paged.run(dtlib, s), want[0]) and torch.equal(prompt.run(dtlib, p), want[1])


def test_captured_without_a_workspace_or_an_output(dtlib):
    """Each call's own output and workspace are the graph's; the calls depend on one another and on another stream."""
    s, p = cut_pairs(), prompt.make([300, 700], 8, 2, 64)
    want = paged.run(dtlib, s).clone(), prompt.run(dtlib, p).clone()
    N, Hkv, d = 40, 2, 128
    k = torch.randn(N, Hkv, d, device="cuda").to(BF)
    kc, vc = (torch.zeros(4, Hkv, 16, d, dtype=BF, device="cuda") for _ in range(2))
    slots = torch.arange(N, dtype=torch.int32, device="cuda")
    q0 = s["q"].clone()

    def calls(other):
        here = torch.cuda.current_stream()
        other.wait_stream(here)
        with torch.cuda.stream(other):
            s["q"].copy_(q0)
            dtlib.dt_kv_append(k, k, kc, vc, slots)
        b = prompt.run(dtlib, p)
        here.wait_stream(other)
        return paged.run(dtlib, s), b
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(other)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        a, b = calls(other)
    for _ in range(3):
        s["q"].zero_(), kc.zero_(), a.fill_(float("nan")), b.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
        assert torch.equal(kc.transpose(1, 2).reshape(-1, Hkv, d)[:N], k)
