"""The paged-cache operators against their definitions in 64 bits: rotary
append, attention, attention mass and eviction, at the sizes and masks where
they can go wrong.

Tolerances, derived from the arithmetic (bf16 rounds to 8 bits: half a unit is
at most 2^-8 of the value):
  rope       2^-8 |y| (the one rounding) + 2^-19 (|a| + |b|) factor (fp32
             products of the pair and the fp32 sine and cosine);
  attention  2^-8 |o| (output rounding) + 2^-8 A (rounding of the
             probabilities, A = sum p |v|) + 2^-13 A (fp32 scores: an error of
             2^-21 of sum |q k| scale, itself below 2^7 in these inputs, moves
             a probability by less than 2^-14, and the normaliser as much);
  lse        2^-21 (S + |lse|) + 2^-20, S the row's largest sum |q k| scale;
  mass       (2^-13) of the added sum + 2^-22 |decay mass|;
  evict      equal.
"""
import numpy as np
import pytest
import torch

from oracle import cache as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tern():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_gemv_gemm_gb300 import build
    build.build()
    import bit_gemv_gemm_gb300 as t
    return t


def f64(t):
    return t.detach().double().cpu().numpy()


class Problem:
    """A cache with scattered pages, unused slots full of NaN, and new tokens."""

    def __init__(self, seed, lens, new, q_heads, kv_heads, D, page=16, layout="hnd", spread=2.0, q_pad=0,
                 wide_table=0):
        g = torch.Generator().manual_seed(seed)
        need = [-(-x // page) for x in lens]
        self.W = max(max(need), 1) + wide_table
        total = sum(need) + 2
        ids = torch.randperm(total, generator=g).to(torch.int32)
        table = torch.full((len(lens), self.W), -1, dtype=torch.int32)     # past the end: never read
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = ids[at:at + k]
            at += k
        shape = (total, kv_heads, page, D)
        nan = float("nan")
        k, v = torch.full(shape, nan).bfloat16(), torch.full(shape, nan).bfloat16()
        for b, L in enumerate(lens):
            if L == 0:
                continue
            j = torch.arange(L)
            pg, sl = table[b].long()[j // page], j % page
            k[pg, :, sl] = torch.randn(L, kv_heads, D, generator=g).bfloat16()
            v[pg, :, sl] = torch.randn(L, kv_heads, D, generator=g).bfloat16()
        self.lens, self.new, self.page = list(lens), list(new), page
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(self.q_start[-1])
        wide = torch.randn(T, q_heads * D + q_pad, generator=g).mul_(spread).bfloat16()
        if layout == "nhd":
            dev = lambda x: x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)   # noqa: E731
        else:
            dev = lambda x: x.cuda()   # noqa: E731
        self.k, self.v = dev(k), dev(v)
        self.table, self.lens_d = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        self.q_start_d = torch.from_numpy(self.q_start).cuda()
        self.q = wide.cuda()[:, :q_heads * D].view(T, q_heads, D) if T else torch.empty(
            (0, q_heads, D), dtype=torch.bfloat16, device="cuda")
        self.T, self.q_heads, self.kv_heads, self.D, self.pages = T, q_heads, kv_heads, D, total
        self.scale = D ** -0.5
        self.host = (f64(self.q), f64(self.k), f64(self.v), table.numpy())


def run_attention(tern, p, window=0, uniform=False, ws=None):
    out = torch.full((p.T, p.q_heads, p.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.T, p.q_heads), float("nan"), device="cuda")
    tern.paged_attention(p.q, p.k, p.v, p.table, p.lens_d, q_start=None if uniform else p.q_start_d,
                         max_new=max(p.new), scale=p.scale, window=window, out=out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    assert tern.device_error() == 0
    return out, lse


def check_attention(p, out, lse, window=0):
    q, k, v, table = p.host
    o, l, A, S = ref.attention(q, k, v, table, p.lens, p.q_start, p.scale, window)
    got, gl = f64(out), f64(lse)
    bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -13) * A + 1e-30
    err = np.abs(got - o)
    assert (err <= bound).all(), f"worst {np.nanmax(err / bound):.3g}, {(~(err <= bound)).sum()} of {err.size}"
    empty = np.isneginf(l)
    assert np.array_equal(np.isneginf(gl), empty) and (got[empty] == 0).all()
    with np.errstate(invalid="ignore"):
        lerr, lb = np.abs(gl - l)[~empty], (2.0 ** -21 * (S + np.abs(l)) + 2.0 ** -20)[~empty]
    assert (lerr <= lb).all(), f"lse worst {np.max(lerr / lb):.3g}"


def run_mass(tern, p, lse, window=0, decay=0.75, in_place=False):
    g = torch.Generator().manual_seed(p.T + 17)
    m = (torch.rand((p.pages, p.kv_heads, p.page), generator=g) * 3).cuda()
    m_in = f64(m)
    out = m if in_place else torch.full_like(m, -5.0)
    before = f64(out)
    tern.attention_mass(p.q, p.k, p.table, p.lens_d, lse, m, out=out, q_start=p.q_start_d, max_new=max(p.new),
                        scale=p.scale, window=window, decay=decay)
    torch.cuda.synchronize()
    assert tern.device_error() == 0
    q, k, _, table = p.host
    want, added = ref.mass(q, k, table, p.lens, p.q_start, p.scale, window, f64(lse), decay, m_in, before.copy())
    err = np.abs(f64(out) - want)
    bound = 2.0 ** -13 * added + 2.0 ** -22 * np.abs(decay * m_in) + 1e-12
    bound[want == before] = 0 if not in_place else bound[want == before]
    assert (err <= bound).all(), f"mass worst {np.max(err / np.maximum(bound, 1e-30)):.3g}"
    return out


def check_both(tern, p, window=0):
    out, lse = run_attention(tern, p, window)
    check_attention(p, out, lse, window)
    if p.T:
        run_mass(tern, p, lse, window)


# ---------------------------------------------------------------------------
# attention and mass
# ---------------------------------------------------------------------------

HEADS = [(8, 2, 128), (4, 4, 64), (7, 1, 64), (4, 1, 256), (10, 2, 128), (2, 2, 256), (16, 1, 128)]


@pytest.mark.parametrize("q_heads,kv_heads,D", HEADS)
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 129, 1000])
def test_one_token(tern, q_heads, kv_heads, D, length):
    check_both(tern, Problem(length, [length], [1], q_heads, kv_heads, D))


@pytest.mark.parametrize("page,layout", [(16, "nhd"), (32, "hnd"), (48, "nhd"), (64, "hnd"), (128, "nhd"), (256, "hnd")])
@pytest.mark.parametrize("new", [1, 5, 33, 200])
def test_pages_and_layouts(tern, page, layout, new):
    check_both(tern, Problem(page + new, [new, new + page - 1, new + 3 * page + 5], [new] * 3, 8, 2, 128, page, layout))


@pytest.mark.parametrize("q_heads,kv_heads,D", HEADS)
@pytest.mark.parametrize("new", [2, 5, 16, 31, 130, 257])
def test_chunk_over_context(tern, q_heads, kv_heads, D, new):
    check_both(tern, Problem(new, [new + 301], [new], q_heads, kv_heads, D, 32))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_ragged_batch(tern, D):
    """Sequences without new tokens, without keys, with more new tokens than
    keys (their first queries see nothing), and of many lengths."""
    lens = [700, 0, 40, 5, 64, 1, 333, 128]
    new = [150, 3, 0, 9, 64, 1, 130, 1]
    check_both(tern, Problem(9, lens, new, 6, 2, D, 16, q_pad=24, wide_table=3))


@pytest.mark.parametrize("lens,new", [([3], [8]), ([0, 0], [1, 4]), ([1, 100], [300, 140]), ([5] * 40, [1] * 40)])
def test_rows_that_see_nothing(tern, lens, new):
    check_both(tern, Problem(5, lens, new, 4, 2, 128))


@pytest.mark.parametrize("window", [1, 7, 16, 100, 129, 5000])
@pytest.mark.parametrize("new", [1, 6, 150])
def test_window(tern, window, new):
    check_both(tern, Problem(window, [new + 405, new + 12, max(new - 3, 1)], [new] * 3, 8, 2, 128, 16), window)


@pytest.mark.parametrize("D,window", [(64, 0), (64, 50), (256, 0), (256, 300)])
def test_window_other_heads(tern, D, window):
    check_both(tern, Problem(D, [900, 411], [300, 2], 8, 2, D, 64, "nhd"), window)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 20, 150])
def test_window_leaves_earlier_pages_alone(tern, D, new):
    """Pages that hold no visible key are not read: their table entries may be
    anything, as a cache that drops them leaves it."""
    p = Problem(new, [new + 700, new + 64], [new, new], 4, 2, D, 32)
    gone = p.table.clone()
    for b, L in enumerate(p.lens):
        first = max(L - new - 100 + 1, 0) // p.page
        gone[b, :first] = p.pages + 5
    kept, p.table = p.table, gone
    out, lse = run_attention(tern, p, 100)
    p.table = kept
    check_attention(p, out, lse, 100)


@pytest.mark.parametrize("q_heads,kv_heads,D,new", [(64, 1, 64, 1), (64, 1, 128, 3), (48, 1, 256, 2), (126, 2, 64, 5),
                                                    (33, 1, 128, 40), (3, 3, 64, 129), (1, 1, 128, 257)])
def test_group_sizes(tern, q_heads, kv_heads, D, new):
    """Up to 64 query heads a key head, and groups that do not divide 128."""
    check_both(tern, Problem(new, [new + 333, new], [new, new], q_heads, kv_heads, D, 16))


def test_many_sequences(tern):
    """More sequences than threads look for their share, most of them without
    new tokens or keys, and row tiles that few of them have."""
    lens = [(37 * b) % 300 for b in range(900)]
    new = [min(L, (0, 1, 0, 3)[b % 4]) for b, L in enumerate(lens)]
    lens[450], new[450] = 500, 200
    check_both(tern, Problem(2, lens, new, 4, 1, 64, 16))


def test_long_context(tern):
    """Enough keys for every split of the keys over the GPU."""
    check_both(tern, Problem(3, [20011], [1], 8, 2, 128, 16))
    check_both(tern, Problem(4, [9001, 17], [5, 17], 8, 1, 128, 64, "nhd"))


@pytest.mark.parametrize("page,layout,window", [(16, "nhd", 0), (48, "hnd", 0), (64, "hnd", 8200), (256, "nhd", 0)])
@pytest.mark.parametrize("new", [33, 150, 300])
def test_wide_heads_over_a_long_table(tern, page, layout, window, new):
    """Heads of 256 take another kernel where the table has room for 8192 keys;
    the second sequence's last row tile is alone, the third has one only."""
    p = Problem(new, [new + 777, new + 130, 9, 2 * new], [new, new - 1, 9, 2], 8, 2, 256, page, layout,
                wide_table=8192 // page)
    check_attention(p, *run_attention(tern, p, window), window)


@pytest.mark.parametrize("new", [40, 150])
def test_wide_heads_with_a_growing_maximum(tern, new):
    """The running maximum moves with every key tile: what was added is scaled down."""
    p = Problem(new, [new + 1500], [new], 4, 1, 256, 64, wide_table=128, spread=1.0)
    grow = torch.linspace(0, 24, p.lens[0])
    for i in range(p.lens[0]):
        pg, sl = int(p.table[0, i // p.page]), i % p.page
        p.k[pg, :, sl] *= float(grow[i])
    p.host = (p.host[0], f64(p.k), p.host[2], p.host[3])
    check_attention(p, *run_attention(tern, p))


@pytest.mark.parametrize("B", [1, 3, 200])
def test_uniform_tokens_without_q_start(tern, B):
    p = Problem(B, [30 + 7 * b for b in range(B)], [2] * B, 4, 2, 64)
    out, lse = run_attention(tern, p, uniform=True)
    check_attention(p, out, lse)


@pytest.mark.parametrize("new", [1, 140])
def test_sharp_and_flat_scores(tern, new):
    """Scores of a standard deviation of about 12 (one key takes the row), all
    equal scores, a negative scale and none."""
    p = Problem(1, [new + 500], [new], 8, 2, 128, spread=12.0)
    check_both(tern, p)
    p = Problem(2, [new + 500], [new], 8, 2, 128, spread=0.0)
    check_both(tern, p)
    p = Problem(3, [new + 500], [new], 8, 2, 128)
    p.scale = -p.scale
    check_both(tern, p)
    p.scale = 0.0
    check_both(tern, p)


@pytest.mark.parametrize("new", [1, 20, 150])
def test_growing_maximum(tern, new):
    """Keys whose scores grow along the sequence, so that the running maximum
    moves at every tile."""
    p = Problem(8, [new + 600], [new], 4, 1, 128)
    with torch.no_grad():
        L, page = new + 600, p.page
        j = torch.arange(L, device="cuda")
        pg, sl = p.table[0].long()[j // page], j % page
        unit = torch.randn(128, device="cuda")
        unit /= unit.norm()
        p.k[pg, :, sl] = (unit * (j.float()[:, None] * 0.12))[:, None].bfloat16().expand(L, 1, 128)
        p.q.copy_((unit * 11.3).bfloat16().expand(new, 4, 128))
    p.host = (f64(p.q), f64(p.k), f64(p.v), p.host[3])
    check_both(tern, p)


@pytest.mark.parametrize("new", [1, 5, 150])
def test_calls_repeat_bit_for_bit_on_one_workspace(tern, new):
    p = Problem(new, [4000 + new, 77 + new], [new, new], 8, 2, 128)
    r = Problem(new + 1, [900 + new], [new], 8, 2, 64)
    ws = tern.workspace(1 << 27)
    a = run_attention(tern, p, ws=ws)
    other = run_attention(tern, r, ws=ws)
    check_attention(r, *other)
    b = run_attention(tern, p, ws=ws)
    check_attention(p, *b)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    m = run_mass(tern, p, a[1])
    assert torch.equal(m, run_mass(tern, p, a[1]))


def test_mass_in_place_and_without_new_tokens(tern):
    p = Problem(3, [200, 31], [3, 0], 4, 2, 64)
    _, lse = run_attention(tern, p)
    run_mass(tern, p, lse, in_place=True)


@pytest.mark.parametrize("new", [1, 140])
def test_side_stream_and_graph(tern, new):
    p = Problem(6, [2000 + new], [new], 8, 2, 128)
    ws = tern.workspace(tern.paged_attention_workspace_bytes(1, p.T, new, 8, 2, 128))
    out = torch.empty((p.T, 8, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((p.T, 8), device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call = lambda s=None: tern.paged_attention(p.q, p.k, p.v, p.table, p.lens_d, q_start=p.q_start_d, max_new=new,   # noqa: E731
                                               out=out, lse=lse, ws=ws, stream=s)
    call(side)
    side.synchronize()
    check_attention(p, out, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    out.fill_(float("nan"))
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    check_attention(p, out, lse)


@pytest.mark.parametrize("new", [1, 140])
def test_pool_past_two_to_the_31_values(tern, new):
    """Pages whose offsets pass 32 bits (a strided pool of 2.2e9 values)."""
    page, D = 16, 64
    stride = 1 << 24
    pages = 135
    k, v = (torch.empty(pages * stride, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    view = lambda t: t.as_strided((pages, 1, page, D), (stride, page * D, D, 1))   # noqa: E731
    L = new + 70
    p = Problem(2, [L], [new], 2, 1, D, page)
    used = p.table[0].long()[:-(-L // page)]
    far = torch.arange(pages - 1, pages - 1 - used.numel(), -1, device="cuda")
    kv, vv = view(k), view(v)
    kv[far], vv[far] = p.k[used], p.v[used]
    out = torch.empty((new, 2, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((new, 2), device="cuda")
    tern.paged_attention(p.q, kv, vv, far.to(torch.int32)[None].contiguous(), p.lens_d, out=out, lse=lse)
    torch.cuda.synchronize()
    check_attention(p, out, lse)


@pytest.mark.parametrize("new", [1, 140])
def test_bad_device_values_are_reported(tern, new):
    """A page id outside the pool, a length past the table, a token range past
    T: reported through the device error word, nothing followed."""
    p = Problem(4, [100 + new], [new], 4, 2, 128)
    for change, code in ((lambda: p.table.fill_(p.pages), tern.DEVERR_CACHE_PAGE),
                         (lambda: p.lens_d.fill_(1 << 30), tern.DEVERR_CACHE_SEQUENCE),
                         (lambda: p.q_start_d.fill_(p.T + 1), tern.DEVERR_CACHE_SEQUENCE)):
        keep = [x.clone() for x in (p.table, p.lens_d, p.q_start_d)]
        p.table.clamp_(min=0)
        change()
        ws = tern.workspace(1 << 27)
        out, lse = torch.zeros((p.T, 4, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((p.T, 4), device="cuda")
        tern.paged_attention(p.q, p.k, p.v, p.table, p.lens_d, q_start=p.q_start_d, max_new=new, out=out, lse=lse, ws=ws)
        assert tern.device_error() == code
        m = torch.zeros((p.pages, 2, p.page), device="cuda")
        tern.attention_mass(p.q, p.k, p.table, p.lens_d, lse, m, q_start=p.q_start_d, max_new=new)
        assert tern.device_error() == code
        for x, y in zip((p.table, p.lens_d, p.q_start_d), keep):
            x.copy_(y)
    out, lse = run_attention(tern, p)
    check_attention(p, out, lse)


# ---------------------------------------------------------------------------
# rotary append
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,q_heads,kv_heads,D,rot", [(1, 32, 8, 128, 128), (3, 4, 2, 64, 32), (77, 6, 1, 256, 64),
                                                      (5, 3, 3, 128, 0), (2, 2, 1, 64, 2), (130, 5, 2, 128, 100),
                                                      (600, 8, 2, 96, 96), (9, 1, 1, 8, 6)])
def test_rope_append(tern, dtype, interleaved, T, q_heads, kv_heads, D, rot):
    g = torch.Generator().manual_seed(T + rot)
    page, layout = (16, "hnd") if T % 2 else (48, "nhd")
    pages = -(-T // page) + 3
    x = torch.randn(T, (q_heads + 2 * kv_heads) * D + 16, generator=g).to(dtype).cuda()
    q = x[:, :q_heads * D].view(T, q_heads, D)
    k = x[:, q_heads * D:(q_heads + kv_heads) * D].view(T, kv_heads, D)
    v = x[:, (q_heads + kv_heads) * D:(q_heads + 2 * kv_heads) * D].view(T, kv_heads, D)
    pos = torch.randint(0, 200000, (T,), generator=g).to(torch.int32)
    pos[0] = 0
    pos[-1] = 2147483647 if T > 1 else pos[-1]
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int64)
    if T > 2:
        slots[1] = -1                                                      # a padding token: not stored
    inv, factor = (tern.rope_frequencies(rot, 10000.0, "yarn", 4.0, 4096) if rot > 2 else
                   (np.ones(rot // 2, np.float32), 1.25))
    shape = (pages, kv_heads, page, D) if layout == "hnd" else (pages, page, kv_heads, D)
    caches = [torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    views = [c if layout == "hnd" else c.permute(0, 2, 1, 3) for c in caches]
    out = tern.rope_append(q, k, v, pos.cuda(), slots.cuda(), torch.from_numpy(inv).cuda(), *views,
                           interleaved=interleaved, attn_factor=factor)
    torch.cuda.synchronize()
    assert tern.device_error() == 0

    def close(got, src, want):
        a = np.abs(f64(src))
        pair = np.zeros_like(a)
        if rot:
            ia = 2 * np.arange(rot // 2) if interleaved else np.arange(rot // 2)
            ib = ia + 1 if interleaved else ia + rot // 2
            pair[..., ia] = pair[..., ib] = a[..., ia] + a[..., ib]
        err, bound = np.abs(got - want), 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * factor * pair + 1e-38
        assert (err <= bound).all(), f"worst {np.max(err / bound):.3g}"

    close(f64(out), q, ref.rope(f64(q), pos.numpy(), inv, factor, interleaved))
    kept = slots >= 0
    pg, sl = (slots[kept] // page).cuda(), (slots[kept] % page).cuda()
    close(f64(views[0][pg, :, sl]), k[kept.cuda()], ref.rope(f64(k), pos.numpy(), inv, factor, interleaved)[kept.numpy()])
    assert torch.equal(views[1][pg, :, sl], v[kept.cuda()].to(torch.bfloat16))
    for w in views:                                                        # every other slot untouched
        flat = torch.ones(pages, page, dtype=torch.bool, device="cuda")
        flat[pg, sl] = False
        assert (w.permute(0, 2, 1, 3)[flat] == 7.0).all()


def test_rope_keys_only_and_bad_slot(tern):
    pages, page, D = 3, 16, 64
    k = torch.randn(2, 1, D, device="cuda")
    q = torch.empty((2, 0, D), device="cuda")
    kc, vc = (torch.zeros((pages, 1, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    inv = torch.from_numpy(tern.rope_frequencies(D)[0]).cuda()
    pos = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    tern.rope_append(q, k, k, pos, torch.tensor([5, pages * page], device="cuda"), inv, kc, vc)
    assert tern.device_error() == tern.DEVERR_CACHE_SLOT
    assert torch.equal(kc[0, 0, 5], k[0, 0].bfloat16()) and torch.equal(vc[0, 0, 5], k[0, 0].bfloat16())
    kc[0, 0, 5] = 0
    assert not kc.any()
    tern.rope_append(q[:0], k[:0], k[:0], pos[:0], pos[:0].long(), inv, kc, vc)      # no tokens: no launch
    assert tern.last_launch_count() == 0


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------

def masses(kind, shape, seed):
    r = np.random.default_rng(seed)
    m = r.random(shape).astype(np.float32) ** 6 * 10
    if kind == "ties":
        m = r.integers(0, 4, shape).astype(np.float32)
    elif kind == "equal":
        m[:] = 0.25
    elif kind == "odd":
        m = r.standard_normal(shape).astype(np.float32)
        m[r.random(shape) < 0.1] = np.nan
        m[r.random(shape) < 0.1] = np.inf
        m[r.random(shape) < 0.1] = -np.inf
        m[r.random(shape) < 0.1] = -0.0
        m[r.random(shape) < 0.1] = 0.0
        m[r.random(shape) < 0.05] = 1e-42
    return m


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd"])
@pytest.mark.parametrize("lens,budget,recent", [([1], 1, 0), ([5, 0, 17], 8, 3), ([100, 31, 64], 64, 64),
                                                ([1000, 64, 65, 2049], 64, 0), ([5000, 4999], 1025, 100),
                                                ([33, 40], 39, 1), ([40000, 123], 3000, 17)])
def test_evict(tern, kind, lens, budget, recent):
    D, H = (64, 3) if len(lens) % 2 else (128, 2)
    p = Problem(budget, lens, [0] * len(lens), H, H, D, 16, "hnd" if recent % 2 else "nhd")
    m = masses(kind, (p.pages, H, p.page), budget)
    md = torch.from_numpy(m).cuda()
    dpage = 32
    per = -(-budget // dpage)
    dpages = per * len(lens) + 1
    dtable = torch.randperm(dpages)[:per * len(lens)].view(len(lens), per).to(torch.int32)
    dk, dv = (torch.full((dpages, H, dpage, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dm = torch.full((dpages, H, dpage), -9.0, device="cuda")
    keep, dl = tern.cache_evict(p.k, p.v, md, p.table, p.lens_d, budget, recent, dk, dv, dm, dtable.cuda())
    torch.cuda.synchronize()
    assert tern.device_error() == 0
    want = ref.evict(m, p.host[3], lens, budget, recent)
    keep, dk, dv, dm = keep.cpu().numpy(), dk.float().cpu().numpy(), dv.float().cpu().numpy(), dm.cpu().numpy()
    k, v = p.k.float().cpu().numpy(), p.v.float().cpu().numpy()
    touched = np.zeros((dpages, dpage), dtype=bool)
    for b, L in enumerate(lens):
        n = min(L, budget)
        assert int(dl[b]) == n
        i = np.arange(n)
        pg, sl = dtable[b].numpy()[i // dpage], i % dpage
        touched[pg, sl] = True
        for h in range(H):
            assert keep[b, h, :n].tolist() == want[b][h] and (keep[b, h, n:] == -1).all()
            j = np.array(want[b][h], dtype=np.int64)
            spg, ssl = p.host[3][b][j // p.page], j % p.page
            assert np.array_equal(dk[pg, h, sl], k[spg, h, ssl]) and np.array_equal(dv[pg, h, sl], v[spg, h, ssl])
            assert np.array_equal(dm[pg, h, sl], m[spg, h, ssl], equal_nan=True)
    assert (dk.transpose(0, 2, 1, 3)[~touched] == 9).all() and (dm.transpose(0, 2, 1)[~touched] == -9).all()


def test_evict_within_one_pool_and_bad_values(tern):
    """The destination pages may lie in the source pool, apart from the
    sequence's own; a bad page id or length is reported."""
    p = Problem(1, [300], [0], 2, 2, 64, 16)
    extra = 8
    k, v = (torch.cat([t, torch.zeros((extra, 2, 16, 64), dtype=torch.bfloat16, device="cuda")]) for t in (p.k, p.v))
    m = torch.rand((p.pages + extra, 2, 16), device="cuda")
    m0 = m.clone()
    dst = torch.arange(p.pages, p.pages + extra, dtype=torch.int32, device="cuda")[None].contiguous()
    keep, dl = tern.cache_evict(k, v, m, p.table, p.lens_d, 100, 10, k, v, m, dst)
    torch.cuda.synchronize()
    assert tern.device_error() == 0 and int(dl) == 100
    want = ref.evict(m0.cpu().numpy(), p.host[3], [300], 100, 10)
    assert keep[0].tolist() == want[0]
    j = keep[0, 1].long()
    i = torch.arange(100, device="cuda")
    assert torch.equal(k[dst[0].long()[i // 16], 1, i % 16], p.k[p.table[0].long()[j // 16], 1, j % 16])
    for bad, code in ((dict(table=torch.full_like(p.table, 1 << 20)), tern.DEVERR_CACHE_PAGE),
                      (dict(lens=torch.full_like(p.lens_d, 1 << 30)), tern.DEVERR_CACHE_SEQUENCE),
                      (dict(dst_table=torch.full_like(dst, -3)), tern.DEVERR_CACHE_PAGE)):
        a = dict(table=p.table.clamp(min=0), lens=p.lens_d, dst_table=dst, **{})
        a.update(bad)
        tern.cache_evict(k, v, m, a["table"], a["lens"], 100, 10, k, v, m, a["dst_table"])
        assert tern.device_error() == code


def test_device_tensor_refusals(tern):
    """What the binding refuses on tensors that are on the GPU."""
    p = Problem(1, [40], [1], 4, 2, 128)
    with pytest.raises(TypeError, match="bfloat16"):
        tern.paged_attention(p.q, p.k.float(), p.v.float(), p.table, p.lens_d)
    with pytest.raises(TypeError, match="q must"):
        tern.paged_attention(p.q.float(), p.k, p.v, p.table, p.lens_d)
    with pytest.raises(ValueError, match="v_cache"):
        tern.paged_attention(p.q, p.k, p.v[:1], p.table, p.lens_d)
    with pytest.raises(TypeError, match="table"):
        tern.paged_attention(p.q, p.k, p.v, p.table.long(), p.lens_d)
    with pytest.raises(ValueError, match="lens"):
        tern.paged_attention(p.q, p.k, p.v, p.table, p.lens_d[:0])
    with pytest.raises(ValueError, match="heads"):
        tern.paged_attention(p.q.permute(0, 2, 1), p.k, p.v, p.table, p.lens_d)
    with pytest.raises(tern.TernError):
        tern.paged_attention(p.q[:, :3], p.k, p.v, p.table, p.lens_d)
    with pytest.raises(tern.TernError):
        tern.paged_attention(p.q, p.k, p.v, p.table, p.lens_d, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="mass"):
        tern.attention_mass(p.q, p.k, p.table, p.lens_d, torch.zeros(1, 4, device="cuda"),
                            torch.zeros(3, device="cuda"))
    assert tern.device_error() == 0
