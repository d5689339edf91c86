"""The paged-cache operators where their arguments are at their ends: windows
past every key, values that are not finite, streams of their own, groups that do
not fill a row tile.  Bounds as in test_gpu_cache.py, where they are derived."""
import numpy as np
import pytest
import torch

from oracle import cache as ref
from test_gpu_cache import Problem, check_attention, check_both, f64, run_attention, run_mass

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tern():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_gemv_gemm_gb300 import build
    build.build()
    import bit_gemv_gemm_gb300 as t
    return t


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("length,new", [(3, 8), (20, 40), (100, 300)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 100])
def test_window_past_every_key(tern, D, length, new, window):
    """The largest windows hide nothing, in sequences whose first tokens see no key either."""
    check_both(tern, Problem(new, [length, new + 50], [new, 1], 4, 2, D), window)


def rows_but(p, out, lse, hit, window=0):
    """Every row but those of `hit` [T, q_heads] against the definition."""
    q, k, v, table = p.host
    q = np.where(hit[..., None], 0.0, q)
    o, l, A, S = ref.attention(q, np.nan_to_num(k), np.nan_to_num(v), table, p.lens, p.q_start, p.scale, window)
    err, bound = np.abs(f64(out) - o), 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -13) * A + 1e-30
    assert (err <= bound)[~hit].all()
    lerr, lb = np.abs(f64(lse) - l), 2.0 ** -21 * (S + np.abs(l)) + 2.0 ** -20
    assert (lerr <= lb)[~hit].all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 20, 150])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_row_whose_query_is_not_finite(tern, D, new, value):
    """Its output and lse are NaN (an lse of -inf says that a row sees no key), and no other row's."""
    p = Problem(new, [new + 900], [new], 8, 2, D)
    hit = np.zeros((new, 8), dtype=bool)
    for t, h in ((0, 1), (new - 1, 6)):
        p.q[t, h, 5] = value
        hit[t, h] = True
    out, lse = run_attention(tern, p)
    assert np.isnan(f64(out)[hit]).all() and np.isnan(f64(lse)[hit]).all()
    rows_but(p, out, lse, hit)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [5, 40, 150])
def test_a_key_that_is_not_a_number(tern, D, new):
    """The rows that see it are NaN, the others not."""
    p = Problem(new, [new + 500], [new], 4, 2, D)
    j = 500 + new // 2
    p.k[p.table[0, j // p.page].long(), 1, j % p.page, 3] = float("nan")
    out, lse = run_attention(tern, p)
    hit = np.zeros((new, 4), dtype=bool)
    hit[new // 2:, 2:] = True
    assert np.isnan(f64(out)[hit]).all() and np.isnan(f64(lse)[hit]).all()
    p.host = (p.host[0], np.nan_to_num(p.host[1]), p.host[2], p.host[3])
    rows_but(p, out, lse, hit)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [2, 140])
def test_mass_of_a_row_with_an_infinite_lse(tern, D, new):
    """exp(s - inf) is 0: the row weighs nothing, the others what they do."""
    p = Problem(new, [new + 300], [new], 4, 2, D)
    _, lse = run_attention(tern, p)
    lse[0, 1] = lse[new - 1, 3] = float("inf")
    run_mass(tern, p, lse)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("new", [1, 20, 150])
def test_keys_before_every_window_may_hold_anything(tern, D, page, new):
    """Keys and values that no query sees any more, in the pages and tiles of those that some do."""
    p = Problem(new, [new + 405, new + 1000], [new, new], 4, 2, D, page)
    for b, L in enumerate(p.lens):
        for j in range(L - new - 100 + 1):
            page_id = p.table[b, j // page].long()
            p.k[page_id, :, j % page] = float("nan")
            p.v[page_id, :, j % page] = float("inf") if j % 2 else float("nan")
    out, lse = run_attention(tern, p, 100)
    check_attention(p, out, lse, 100)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [3, 5, 7, 11])
@pytest.mark.parametrize("new", [9, 90])
def test_results_do_not_depend_on_the_calls_before(tern, D, group, new):
    """A group that does not divide 128 leaves rows of a row tile over: what the
    last kernel left in them changes no bit of the others."""
    p = Problem(new, [new + 3000] * 6, [new] * 6, 2 * group, 2, D)
    ws, got = tern.workspace(1 << 27), []
    for spread in (0.0, 60.0, 300.0):
        r = Problem(1, [new + 2000] * 12, [max(new, 10)] * 12, 8, 2, D, spread=spread)
        run_attention(tern, r, ws=ws)
        got.append(run_attention(tern, p, ws=ws))
    check_attention(p, *got[0])
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("new", [9, 90])
def test_results_do_not_depend_on_the_sequences_beside(tern, new):
    """A sequence's rows are the same bits whatever queries follow them in the call."""
    got = []
    for spread in (0.0, 100.0):
        p = Problem(new, [new + 700, new + 700], [new, new], 8, 2, 128)
        p.q[new:] = torch.randn(p.q[new:].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) * spread
        got.append([x[:new].clone() for x in run_attention(tern, p)])
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def leave_garbage(nbytes, stream=None):
    """Freed blocks of device memory, full of ones, for the allocator to hand out again."""
    with torch.cuda.stream(stream):
        x = [torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    del x


@pytest.mark.parametrize("new", [1, 5, 150])
def test_attention_on_another_stream_without_a_workspace(tern, new):
    """The call makes its workspace and output ready on the stream that it runs on."""
    p = Problem(new, [4000 + new, 900 + new], [new, new], 8, 2, 128)
    side = torch.cuda.Stream()
    lse = torch.empty((p.T, 8), device="cuda")
    leave_garbage(1 << 26)
    leave_garbage(1 << 26, side)
    torch.cuda._sleep(200_000_000)             # the current stream is busy meanwhile (0.1 s)
    out = tern.paged_attention(p.q, p.k, p.v, p.table, p.lens_d, q_start=p.q_start_d, max_new=new, lse=lse, stream=side)
    side.synchronize()
    got, glse = out.clone(), lse.clone()
    torch.cuda.synchronize()
    assert tern.device_error() == 0
    check_attention(p, got, glse)


@pytest.mark.parametrize("new", [1, 5, 150])
def test_a_workspace_is_zero_only_where_it_counts(tern, new):
    """The call's own workspace in memory full of ones, and one that is zero in its first bytes alone."""
    p = Problem(new, [4000 + new, 900 + new], [new, new], 8, 2, 128)
    leave_garbage(1 << 26)
    check_attention(p, *run_attention(tern, p))
    ws = torch.full((tern.paged_attention_workspace_bytes(2, p.T, new, 8, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    ws[:tern.ATTENTION_COUNTER_BYTES] = 0
    for _ in range(2):
        check_attention(p, *run_attention(tern, p, ws=ws))


@pytest.mark.parametrize("call,M", [("gemv", 1), ("gemv", 5), ("gemv", 16), ("gemm", 200), ("fwht_gemm", 1)])
def test_products_on_another_stream_without_a_workspace(tern, call, M):
    """The same of the products: bf16 weights and fp32 sums of 4096 terms are off by less than
    (2^-9 + 2^-12) of the sum of the magnitudes; the rotation rounds its result to bf16 once more."""
    N, K = 512, 4096
    g = torch.Generator("cuda").manual_seed(M)
    t = torch.randint(-1, 2, (N, K), dtype=torch.int8, device="cuda", generator=g)
    s = (torch.rand((N, K // 128), device="cuda", generator=g) + 0.5).half()
    x = torch.randn((M, K), device="cuda", generator=g).bfloat16()
    codes, signs = tern.pack(t), torch.ones(K, dtype=torch.int8, device="cuda")
    turned = tern.fwht(x, signs) if call == "fwht_gemm" else x
    w = t.double() * s.double().repeat_interleave(128, dim=1)
    want, most = turned.double() @ w.T, turned.double().abs() @ w.abs().T
    side = torch.cuda.Stream()
    leave_garbage(1 << 24)
    leave_garbage(1 << 24, side)
    torch.cuda._sleep(200_000_000)
    y = getattr(tern, call)(*((x, signs, codes, s) if call == "fwht_gemm" else (x, codes, s)), stream=side)
    side.synchronize()
    got = y.clone()
    torch.cuda.synchronize()
    assert tern.device_error() == 0
    assert bool(((got.double() - want).abs() <= 2.0 ** -7 * most).all())


@pytest.mark.parametrize("max_new", [0, 1, 512])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_mass_of_a_step_without_tokens(tern, D, max_new):
    """No token at all, whatever max_new allows: every key decays."""
    p = Problem(3, [200, 31, 0], [0, 0, 0], 8, 2, D)
    m = torch.rand((p.pages, 2, p.page), device="cuda") + 1.0
    out = torch.full_like(m, -5.0)
    lse = torch.empty((0, 8), device="cuda")
    tern.attention_mass(p.q, p.k, p.table, p.lens_d, lse, m, out=out, q_start=p.q_start_d, max_new=max_new, decay=0.5)
    torch.cuda.synchronize()
    assert tern.device_error() == 0
    want = np.full(m.shape, -5.0)
    for b, L in enumerate(p.lens):
        for j in range(L):
            pg, sl = int(p.table[b, j // p.page]), j % p.page
            want[pg, :, sl] = 0.5 * f64(m)[pg, :, sl]
    assert np.array_equal(f64(out), want)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 16, 140])
def test_mass_in_place_is_the_same_bits(tern, D, new):
    """The running mass may be its own output, as it is by default."""
    p = Problem(new, [new + 700, new + 50], [new, new], 4, 2, D)
    _, lse = run_attention(tern, p)
    apart, same = run_mass(tern, p, lse), run_mass(tern, p, lse, in_place=True)
    for b, L in enumerate(p.lens):
        j = torch.arange(L, device="cuda")
        pg, sl = p.table[b].long()[j // p.page], j % p.page
        assert torch.equal(apart[pg, :, sl], same[pg, :, sl])


@pytest.mark.parametrize("new", [1, 140])
def test_a_bad_page_changes_no_other_page(tern, new):
    """A page id outside the pool is reported, and nothing of its sequence is written elsewhere."""
    p = Problem(4, [100 + new, 20 + new], [new, new], 4, 2, 128)
    _, lse = run_attention(tern, p)
    for bad in (-7, p.pages, 2 ** 31 - 1):
        table = p.table.clone()
        table[0] = bad
        m = torch.full((p.pages, 2, p.page), 3.0, device="cuda")
        tern.attention_mass(p.q, p.k, table, p.lens_d, lse, m, q_start=p.q_start_d, max_new=new, decay=0.5)
        assert tern.device_error() == tern.DEVERR_CACHE_PAGE
        own = torch.zeros(p.pages, dtype=torch.bool)
        own[p.table[1, :-(-p.lens[1] // p.page)].long().cpu()] = True
        assert bool((m[~own.cuda()] == 3.0).all())


def test_a_bad_destination_page_changes_no_other_page(tern):
    p = Problem(1, [300], [0], 2, 2, 64, 16)
    m = torch.rand((p.pages, 2, 16), device="cuda")
    for bad in (-3, 7, 2 ** 31 - 1):
        dk, dv = (torch.full((7, 2, 16, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        dm = torch.full((7, 2, 16), 9.0, device="cuda")
        dst = torch.full((1, 7), bad, dtype=torch.int32, device="cuda")
        dst[0, 3] = 5
        tern.cache_evict(p.k, p.v, m, p.table, p.lens_d, 100, 10, dk, dv, dm, dst)
        assert tern.device_error() == tern.DEVERR_CACHE_PAGE
        rest = [0, 1, 2, 3, 4, 6]
        assert all(bool((x[rest] == 9.0).all()) for x in (dk, dv, dm)) and not bool((dm[5] == 9.0).any())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [4, 8])
def test_many_short_sequences_of_one_key_tile(tern, D, group):
    """Items of a single key tile, in which the second stream of the tiles kernel has no product."""
    lens = [1 + (37 * b) % 128 for b in range(700)]
    new = [min(L, 5 + (7 * b) % 11) for b, L in enumerate(lens)]
    p = Problem(2, lens, new, 2 * group, 2, D)
    a = run_attention(tern, p)
    check_attention(p, *a)
    for _ in range(20):
        b = run_attention(tern, p)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tensors_of_another_gpu_are_refused(tern, monkeypatch):
    """With another device current than the tensors', each call says so before anything is launched."""
    p = Problem(1, [40], [1], 4, 2, 128)
    lse, m = torch.zeros((1, 4), device="cuda"), torch.zeros((p.pages, 2, p.page), device="cuda")
    inv = torch.from_numpy(tern.rope_frequencies(128)[0]).cuda()
    pos, slots = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    k0, m0 = p.k.clone(), m.clone()
    kv, dst = torch.zeros((1, 2, 128), device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    now = torch.cuda.current_device()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now + 1)
    for call in (lambda: tern.paged_attention(p.q, p.k, p.v, p.table, p.lens_d, out=p.q.clone()),
                 lambda: tern.attention_mass(p.q, p.k, p.table, p.lens_d, lse, m),
                 lambda: tern.rope_append(p.q.float(), kv, kv, pos, slots, inv, p.k, p.v, q_out=p.q.clone()),
                 lambda: tern.cache_evict(p.k, p.v, m, p.table, p.lens_d, 16, 1, p.k, p.v, m, dst)):
        with pytest.raises(ValueError, match="current device"):
            call()
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert torch.equal(p.k.view(torch.int16), k0.view(torch.int16)) and torch.equal(m, m0)
    _, _ = run_attention(tern, p)
