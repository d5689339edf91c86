"""The linear-attention block of a ternary-weight decoder, from prompts to drafts.

The block's matrices are ternary packs; between them a short causal convolution
mixes each channel with its last three tokens, the gated delta rule keeps one
state a head in place of keys, and norms stand before the block and over the
heads of its output, under a gate:

    rms_norm (with the residual stream) -> gemv / gemm [q | k | v | gate | decay, step]
      -> short_conv -> gated_delta -> rms_norm (by heads, gated) -> gemv / gemm

Both states are slots of pools.  A draft of several tokens is run from a
sequence's slot to a spare one, so that what is not accepted leaves no trace.

Run it:  python examples/linear_attention_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_gemv_gemm_gb300 as tern  # noqa: E402


class Block:
    def __init__(self, hidden, k_heads, v_heads, dk, dv, slots, width=4, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.k_heads, self.v_heads, self.dk, self.dv, self.hidden = k_heads, v_heads, dk, dv, hidden
        self.channels, self.values = 2 * k_heads * dk + v_heads * dv, v_heads * dv
        self.gates = -(-2 * v_heads // 64) * 64          # decay and step of each head, padded
        rows = self.channels + self.values + self.gates

        def matrix(n, k):
            t = torch.randint(-1, 2, (n, k), dtype=torch.int8, device="cuda", generator=g)
            s = (torch.rand((n, k // 128), device="cuda", generator=g) * 0.02 + 1e-3).half()
            return tern.pack(t), s

        def rand(*shape):
            return torch.rand(shape, device="cuda", generator=g)

        self.into, self.out = matrix(rows, hidden), matrix(hidden, self.values)
        self.norm, self.head_norm = 0.5 + rand(hidden), 0.5 + rand(dv)
        self.conv = (rand(self.channels, width) - 0.5) * 2 * width ** -0.5
        self.a_log, self.dt_bias = torch.log(1 + 15 * rand(v_heads)), -2 - 4 * rand(v_heads)
        # what a sequence keeps: its last inputs of the convolution, its heads' states
        self.inputs = torch.zeros((slots, width - 1, self.channels), device="cuda")
        self.state = torch.zeros((slots, v_heads, dv, dk), device="cuda")

    def forward(self, x, residual, slots, new, past, dst_slots=None):
        """x fp32 or bf16 [sum(new), hidden], the last block's output, and the residual stream, fp32, which
        takes x up; new[b] tokens of the sequence in slots[b], past[b] of it before.  Returns the block's
        output, fp32, and what it went through."""
        T, i32 = x.shape[0], dict(dtype=torch.int32, device="cuda")
        start = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], **i32)
        seq = dict(slots=torch.tensor(slots, **i32), q_start=start, max_new=max(new), past=torch.tensor(past, **i32),
                   dst_slots=None if dst_slots is None else torch.tensor(dst_slots, **i32))
        product = tern.gemv if T <= 16 else tern.gemm
        h = tern.rms_norm(x, self.norm, residual=residual, residual_out=residual)
        p = product(h, *self.into)                                                     # fp32 [T, rows]
        mixed = tern.short_conv(p[:, :self.channels], self.conv, self.inputs, **seq)   # bf16 [T, q | k | v]
        nk = self.k_heads * self.dk
        q, k = (mixed[:, i * nk:(i + 1) * nk].view(T, self.k_heads, self.dk) for i in range(2))
        v = mixed[:, 2 * nk:].view(T, self.v_heads, self.dv)
        gate = p[:, self.channels:self.channels + self.values].view(T, self.v_heads, self.dv)
        g, beta = p[:, -self.gates:][:, :2 * self.v_heads].split(self.v_heads, dim=1)
        o = tern.gated_delta(q, k, v, g, beta, self.state, qk_norm=True, a_log=self.a_log, dt_bias=self.dt_bias, **seq)
        y = tern.rms_norm(o, self.head_norm, gate=gate)
        return product(y.view(T, -1), *self.out), dict(h=h, p=p, mixed=mixed, o=o, y=y, q=q, k=k, v=v, gate=gate, g=g,
                                                       beta=beta)


def main():
    hidden = 1024
    block = Block(hidden, 4, 8, 128, 128, slots=5)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = lambda n: torch.randn((n, hidden), device="cuda", generator=g)   # noqa: E731
    slots, past = [0, 1, 2], [0, 0, 0]
    new = [300, 17, 90]
    y, _ = block.forward(tokens(sum(new)), tokens(sum(new)), slots, new, past)
    past = new
    print("prompts:", tuple(y.shape), "tokens so far", past)
    for step in range(8):
        y, _ = block.forward(tokens(3), tokens(3), slots, [1, 1, 1], past)
        past = [n + 1 for n in past]
    # five drafted tokens of the first two sequences, to spare slots; three and five of them are accepted
    draft, stream = tokens(10), tokens(10)
    y, _ = block.forward(draft, stream.clone(), slots[:2], [5, 5], past[:2], dst_slots=[3, 4])
    slots[1], spare = 4, 1                                       # all five: the spare slot is the sequence's now
    keep = torch.arange(3, device="cuda")                        # three: from the old slot again
    y3, _ = block.forward(draft[keep], stream[keep].clone(), slots[:1], [3], past[:1])
    past = [past[0] + 3, past[1] + 5, past[2]]
    torch.cuda.synchronize()
    assert tern.device_error() == 0 and bool(torch.isfinite(y).all()) and torch.allclose(y3, y[:3], rtol=1e-2, atol=1e-2)
    print("drafts: ", tuple(y.shape), "tokens so far", past, "slots", slots, "spare", [3, spare])


if __name__ == "__main__":
    main()
