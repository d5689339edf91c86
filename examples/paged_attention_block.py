"""The attention block of a ternary-weight decoder, from prompt to long generation.

One block's qkv and output matrices are ternary packs; between them its
queries and keys turn by their positions, its keys and values go to a paged
cache, new tokens attend over that cache, and when a conversation passes its
budget of keys the ones that drew the least attention are dropped:

    prompt   gemm -> rope_append -> paged_attention -> gemm, attention_mass
    token    gemv -> rope_append -> paged_attention -> gemv, attention_mass
    evict    cache_evict to fresh pages, the old ones returned

Run it:  python examples/paged_attention_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_gemv_gemm_gb300 as tern  # noqa: E402


class Pages:
    """A pool of cache pages and who holds them (host side)."""

    def __init__(self, pages, kv_heads, page_size, head_dim):
        self.k, self.v = (torch.zeros((pages, kv_heads, page_size, head_dim), dtype=torch.bfloat16, device="cuda")
                          for _ in range(2))
        self.mass = torch.zeros((pages, kv_heads, page_size), device="cuda")
        self.free, self.size = list(range(pages))[::-1], page_size

    def take(self, n):
        got = [self.free.pop() for _ in range(n)]
        self.mass[got] = 0            # a new key starts without weight
        return got

    def give(self, ids):
        self.free.extend(ids)


class Block:
    def __init__(self, hidden, q_heads, kv_heads, head_dim, batch, budget, recent, page_size=16, decay=0.95, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.hidden = q_heads, kv_heads, head_dim, hidden
        width = (q_heads + 2 * kv_heads) * head_dim

        def matrix(n, k):
            t = torch.randint(-1, 2, (n, k), dtype=torch.int8, device="cuda", generator=g)
            s = (torch.rand((n, k // 128), device="cuda", generator=g) * 0.02 + 1e-3).half()
            return tern.pack(t), s

        self.qkv, self.out = matrix(width, hidden), matrix(hidden, q_heads * head_dim)
        freq, self.factor = tern.rope_frequencies(head_dim)
        self.freq = torch.from_numpy(freq).cuda()
        self.batch, self.budget, self.recent, self.decay = batch, budget, recent, decay
        per = -(-2 * budget // page_size)
        self.pool = Pages(2 * batch * per, kv_heads, page_size, head_dim)
        self.pages = [[] for _ in range(batch)]
        self.keys = [0] * batch         # cached keys of each sequence
        self.seen = [0] * batch         # tokens so far: positions go on when keys are dropped
        self.ws = tern.workspace(1 << 27)

    def _table(self, lists, width=None):
        width = width or max(len(x) for x in lists)
        return torch.tensor([x + [0] * (width - len(x)) for x in lists], dtype=torch.int32, device="cuda")

    def forward(self, x, new):
        """x bf16 [sum(new), hidden]: new[b] tokens of each sequence in a row."""
        T, size = x.shape[0], self.pool.size
        slots, positions = [], []
        for b, n in enumerate(new):
            total = self.keys[b] + n
            self.pages[b] += self.pool.take(-(-total // size) - len(self.pages[b]))
            for i in range(n):
                j = self.keys[b] + i
                slots.append(self.pages[b][j // size] * size + j % size)
                positions.append(self.seen[b] + i)
            self.keys[b], self.seen[b] = total, self.seen[b] + n
        slots = torch.tensor(slots, device="cuda")
        positions = torch.tensor(positions, dtype=torch.int32, device="cuda")
        table, lens = self._table(self.pages), torch.tensor(self.keys, dtype=torch.int32, device="cuda")
        start = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device="cuda")

        product = tern.gemv if T <= 16 else tern.gemm
        qkv = product(x, *self.qkv)                                             # fp32 [T, q | k | v]
        q, k, v = qkv.view(T, -1, self.head_dim).split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)
        q = tern.rope_append(q, k, v, positions, slots, self.freq, self.pool.k, self.pool.v, attn_factor=self.factor)
        lse = torch.empty((T, self.q_heads), device="cuda")
        o = tern.paged_attention(q, self.pool.k, self.pool.v, table, lens, q_start=start, max_new=max(new), lse=lse,
                                 ws=self.ws)
        tern.attention_mass(q, self.pool.k, table, lens, lse, self.pool.mass, q_start=start, max_new=max(new),
                            decay=self.decay)
        return product(o.view(T, -1), *self.out), q, o

    def evict(self):
        """Cuts every sequence to its budget, into pages of their own."""
        size = self.pool.size
        fresh = [self.pool.take(-(-self.budget // size)) for _ in range(self.batch)]
        keep, lens = tern.cache_evict(self.pool.k, self.pool.v, self.pool.mass, self._table(self.pages),
                                      torch.tensor(self.keys, dtype=torch.int32, device="cuda"), self.budget, self.recent,
                                      self.pool.k, self.pool.v, self.pool.mass, self._table(fresh))
        self.keys = [min(n, self.budget) for n in self.keys]
        for old in self.pages:
            self.pool.give(old)            # (calls on one stream: the copy is over before they are written again)
        self.pages = fresh
        return keep, lens


def main():
    hidden, batch = 1024, 3
    block = Block(hidden, 8, 2, 128, batch, budget=256, recent=32)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = lambda n: torch.randn((n, hidden), device="cuda", generator=g).bfloat16()   # noqa: E731
    y, _, _ = block.forward(tokens(200 + 90 + 150), [200, 90, 150])
    print("prompts: ", tuple(y.shape), "keys", block.keys)
    for step in range(120):
        y, _, _ = block.forward(tokens(batch), [1] * batch)
        if max(block.keys) > block.budget + block.recent:
            block.evict()
            print("step %3d: evicted, keys" % step, block.keys, "tokens so far", block.seen)
    torch.cuda.synchronize()
    assert tern.device_error() == 0 and bool(torch.isfinite(y).all())
    print("tokens:  ", tuple(y.shape), "keys", block.keys)


if __name__ == "__main__":
    main()
