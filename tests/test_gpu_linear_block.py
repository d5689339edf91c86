"""The linear-attention block of the example, all the calls together: prompts of
unlike length, single tokens, a draft to a spare slot and what is kept of it.

The replay in 64 bits holds each sequence's whole history of inputs in ordinary
arrays and runs the convolution and the delta rule over it from the first token,
so the states that the block carries from call to call are checked by what comes
out of them.  Each operator is given the block's own inputs to it (the others'
outputs, checked beside it), and held to the bounds of its own tests; the delta
rule's state has gone through as many calls as there were, each within its bound.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import test_gpu_linear as one
from oracle import linear as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_gemv_gemm_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("linear_attention_block",
                                                  os.path.join(ROOT, "examples", "linear_attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dims", [(1, 2, 64, 64), (2, 8, 128, 48)])
def test_block_from_prompt_through_drafts(example, dims):
    import bit_gemv_gemm_gb300 as tern
    Hk, Hv, Dk, Dv = dims
    hidden, B = 512, 3
    block = example.Block(hidden, Hk, Hv, Dk, Dv, slots=2 * B, seed=3)
    for t in (block.inputs, block.state):   # what an earlier conversation left: none of it may be seen
        t.fill_(7.0)
    g = torch.Generator(device="cuda").manual_seed(5)
    fresh = lambda n: torch.randn((n, hidden), device="cuda", generator=g)   # noqa: E731
    slots, past = [4, 0, 2], [0] * B
    lines = [dict(x=np.zeros((0, block.channels)), q=[], k=[], v=[], g=[], b=[]) for _ in range(B)]
    f64 = one.f64

    def run(new, dst=None, keep=True):
        x, res = fresh(sum(new)), fresh(sum(new))
        was = f64(res)
        y, s = block.forward(x, res, slots, new, past, dst)
        assert bool(torch.isfinite(y).all()) and tern.device_error() == 0
        one.check_norm(tern, x, block.norm, s["h"], None, res_out=res, residual_was=was)
        one.check_norm(tern, s["o"], block.head_norm, s["y"], gate=s["gate"])
        at = 0
        for b, n in enumerate(new):
            if n == 0:
                continue
            line, part = lines[b], slice(at, at + n)
            at += n
            whole = np.concatenate([line["x"], f64(s["p"][part, :block.channels])])
            want, _, size = ref.short_conv(whole, f64(block.conv), np.zeros((1, 3, block.channels)), [0], [0, len(whole)])
            one.within(s["mixed"][part], want[-n:],
                       (2.0 ** -8 + 2.0 ** -15) * np.abs(want[-n:]) + 1.2 * 2.0 ** -20 * size[-n:] + 1e-30, "conv")
            new_line = dict(x=whole, **{name: line[name] + [f64(s[full][part])] for name, full in
                                        (("q", "q"), ("k", "k"), ("v", "v"), ("g", "g"), ("b", "beta"))})
            cat = [np.concatenate(new_line[name]) for name in "qkvgb"]
            o, state, reach, mem = ref.gated_delta(*cat, np.zeros((1, Hv, Dv, Dk)), [0], [0, len(whole)], Dk ** -0.5, True,
                                                   f64(block.a_log), f64(block.dt_bias))
            step = 2.0 ** -17 * mem * reach
            bound = 2.0 ** -8 * np.abs(o[-n:]) + (Dk ** -0.5 * (step + 2.0 ** -17 * reach + 2.0 ** -7 * mem * reach))[None, :, None]
            one.within(s["o"][part], o[-n:], bound, "delta")
            to = slots[b] if dst is None else dst[b]
            if to >= 0:
                got = f64(block.state[to])
                assert (np.abs(got - state[0]) <= step[:, None, None] + 2.0 ** -22 * np.abs(state[0])).all()
                assert np.array_equal(f64(block.inputs[to]), whole[-3:] if len(whole) >= 3 else
                                      np.concatenate([np.zeros((3 - len(whole), block.channels)), whole]))
            if keep:
                lines[b] = new_line
                past[b] += n

    run([70, 2, 130])
    for _ in range(3):
        run([1, 1, 1])
    kept = [block.inputs.clone(), block.state.clone()]
    run([5, 5, 5], dst=[1, -1, 3], keep=False)               # a draft: the sequences' own slots stay
    for b in range(B):
        assert torch.equal(block.inputs[slots[b]], kept[0][slots[b]]) and torch.equal(block.state[slots[b]], kept[1][slots[b]])
    run([3, 0, 40])                                          # what follows instead
    run([1, 1, 1])


def test_example_runs(example, capsys):
    example.main()
    assert "drafts" in capsys.readouterr().out
