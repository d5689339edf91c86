"""The attention block of the example, all the calls together: prompts, single
tokens and evictions against a plain replay in 64 bits that holds each
sequence's keys, values and masses in ordinary arrays.

The replay takes the block's own turned queries and cached keys (bf16, checked
against the definition elsewhere), so its outputs carry only the attention's
rounding; the kept keys of an eviction have to be those that the replayed
masses choose, except where two masses lie within their own error of each other.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import cache as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_gemv_gemm_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("paged_attention_block",
                                                  os.path.join(ROOT, "examples", "paged_attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def test_block_from_prompt_through_evictions(example):
    hidden, B, Hq, Hk, D = 512, 2, 4, 2, 128
    block = example.Block(hidden, Hq, Hk, D, B, budget=64, recent=8, seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    masses = [np.zeros((Hk, 0)) for _ in range(B)]
    steps = [[70, 50]] + [[1, 1]] * 8 + [[5, 3]] + [[1, 1]] * 12
    evictions = 0
    for new in steps:
        x = torch.randn((sum(new), hidden), device="cuda", generator=g).bfloat16()
        y, q, o = block.forward(x, new)
        torch.cuda.synchronize()
        assert bool(torch.isfinite(y).all())
        qh, oh = f64(q), f64(o)
        kc, vc, mc = f64(block.pool.k), f64(block.pool.v), f64(block.pool.mass)
        at = 0
        for b, n in enumerate(new):
            L, row = block.keys[b], np.array(block.pages[b])
            start = np.array([0, n])
            want, lse, A, _ = ref.attention(qh[at:at + n], kc, vc, row[None], [L], start, D ** -0.5)
            bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -13) * A + 1e-30
            assert (np.abs(oh[at:at + n] - want) <= bound).all()
            old = np.zeros(mc.shape)
            j = np.arange(L)
            pg, sl = row[j // block.pool.size], j % block.pool.size
            before = np.concatenate([masses[b], np.zeros((Hk, L - masses[b].shape[1]))], axis=1)
            old[pg, :, sl] = before.T
            full, added = ref.mass(qh[at:at + n], kc, row[None], [L], start, D ** -0.5, 0, lse, block.decay, old,
                                   np.zeros(mc.shape))
            got = mc[pg, :, sl].T
            masses[b] = full[pg, :, sl].T
            assert (np.abs(got - masses[b]) <= 2.0 ** -11 * masses[b] + 1e-9).all()   # a few steps' errors add up
            at += n
        if max(block.keys) > block.budget + block.recent:
            device = [f64(block.pool.mass)[np.array(block.pages[b])[np.arange(block.keys[b]) // block.pool.size], :,
                                           np.arange(block.keys[b]) % block.pool.size].T for b in range(B)]
            keys = list(block.keys)
            keep, lens = block.evict()
            evictions += 1
            for b in range(B):
                n = min(keys[b], block.budget)
                assert int(lens[b]) == n == block.keys[b]
                kept = keep[b, :, :n].cpu().numpy()
                for h in range(Hk):
                    r = min(block.recent, n)
                    order = sorted(range(keys[b] - r), key=lambda j: (-device[b][h, j], j))[:n - r]
                    assert kept[h].tolist() == sorted(order) + list(range(keys[b] - r, keys[b]))
                masses[b] = np.stack([masses[b][h, kept[h]] for h in range(Hk)])
    assert evictions >= 2
    import bit_gemv_gemm_gb300 as tern
    assert tern.device_error() == 0


def test_example_runs(example, capsys):
    example.main()
    assert "evicted" in capsys.readouterr().out
