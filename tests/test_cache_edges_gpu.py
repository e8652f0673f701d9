"""The cache operators at their edges: waits that run out, pools above 4 GiB,
captured calls with a workspace of their own, aliased results, queries of a
wide range, many short sequences.  Bounds are those of test_cache_gpu."""
import numpy as np
import pytest
import torch

from block_sparse_masked_mask_gb300 import _native, api
from block_sparse_masked_mask_gb300 import build as B
from oracle import cache as C
from test_cache_gpu import Pair, check_attend, cu_of, dev, filled, randn, run_attend, run_evict, table_for

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ waits

@pytest.fixture(scope="module")
def short_wait_library():
    return B.build_variant("waitshort", {"ATTN_WAIT_TIMEOUT_NS": "100ull"})


@pytest.mark.parametrize("new", [40, 300])
def test_short_waits_of_the_weights_run_out(short_wait_library, new):
    lens = [4000, 2500]
    p = filled(lens, 2, 128, 64, seed=3)
    cu, q = cu_of([new // 2, new // 2]), randn(new, 4, 128, seed=1)
    args = (q.cuda(), run_attend(p, q, cu, lens)[1], p.dev, dev(cu), dev(lens), new // 2, 4000)
    want = api.attn_cache_weights(*args)
    with _native.use_library(short_wait_library):
        for _ in range(2):
            api.attn_cache_weights(*args)
        assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_TIMEOUT
    assert torch.equal(want, api.attn_cache_weights(*args))
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK


@pytest.mark.parametrize("rows", [40, 300])
def test_short_waits_run_out_and_the_launch_returns(short_wait_library, rows):
    """With waits of 100 ns the tcgen05 kernel gives up, the status says so, later
    launches return at once until it has been read, and the context stays usable."""
    lens = [4000, 2500]
    p = filled(lens, 2, 128, 64, seed=3)
    cu, q = cu_of([rows // 2, rows // 2]), randn(rows, 4, 128, seed=1)
    want = [x.clone() for x in check_attend(p, q, cu, lens)]
    with _native.use_library(short_wait_library):
        for _ in range(2):
            run_attend(p, q, cu, lens)
        assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_TIMEOUT
        assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
        # single tokens need no such waits
        one = run_attend(p, q[:2], cu_of([1, 1]), lens)
        assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
        one = [x.clone() for x in one]
    for a, b in zip(one, run_attend(p, q[:2], cu_of([1, 1]), lens)):
        assert torch.equal(a, b)
    for a, b in zip(want, run_attend(p, q, cu, lens)):
        assert torch.equal(a, b)
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK


# ------------------------------------------------------------------ far pages

class Far(Pair):
    """A Pair whose device pages are the last ones of a pool above 4 GiB per side
    (the oracle has them alone)."""

    def __init__(self, lens, heads, dim, page_size, pool, seed, shared=None):
        rng = np.random.default_rng(seed)
        self.table, self.pages = table_for(lens, page_size, rng)
        codes = [rng.integers(0, 256, (self.pages, heads, page_size, dim)).astype(np.uint8) for _ in range(2)]
        scale = [2.0 ** rng.integers(-3, 4, (self.pages, heads)).astype(np.float64) for _ in range(2)]
        self.ref = C.Cache(*codes, *scale, self.table)
        self.first = (shared.first if shared else pool) - self.pages
        if shared:
            d = shared.dev
            bufs = (d.k_pages, d.v_pages, d.k_scale, d.v_scale)
        else:
            bufs = [torch.zeros((pool, heads, page_size, dim), dtype=torch.uint8, device="cuda") for _ in range(2)]
            bufs += [torch.ones((pool, heads), device="cuda") for _ in range(2)]
        for buf, x in zip(bufs, codes + [s.astype(np.float32) for s in scale]):
            buf[self.first:self.first + self.pages] = torch.from_numpy(x).cuda()
        self.dev = api.KVCache(*bufs, torch.from_numpy(self.table + np.int32(self.first)).cuda())

    def check_codes(self):
        here = slice(self.first, self.first + self.pages)
        for got, want in ((self.dev.k_pages, self.ref.codes[0]), (self.dev.v_pages, self.ref.codes[1])):
            assert np.array_equal(got[here].cpu().numpy(), want)
        for got, want in ((self.dev.k_scale, self.ref.scale[0]), (self.dev.v_scale, self.ref.scale[1])):
            assert np.array_equal(got[here].cpu().double().numpy(), want)


def test_pages_past_32_bits():
    heads, dim, ps = 8, 128, 128
    pool = (1 << 32) // (heads * dim * ps) + 64
    lens = [700, 300]
    p = Far(lens, heads, dim, ps, pool, seed=1)
    assert int(p.dev.page_table[0, 0]) * heads * dim * ps > 2 ** 31
    k, v = randn(1000, heads, dim, seed=1), randn(1000, heads, dim, seed=2)
    p.append(k, v, cu_of(lens), lens)
    p.check_codes()
    _, lse = check_attend(p, randn(2, 16, dim, seed=3), cu_of([1, 1]), lens)
    check_attend(p, randn(60, 16, dim, seed=4), cu_of([40, 20]), lens)
    q = randn(2, 16, dim, seed=3)
    w = api.attn_cache_weights(q.cuda(), lse, p.dev, dev([0, 1, 2]), dev(lens), 1, 700).cpu()
    ref, _ = p.ref.weights(q.double().numpy(), lse.cpu().numpy(), cu_of([1, 1]), lens)
    for b, n in enumerate(lens):
        assert np.abs(w[b, :, :n].double().numpy() - ref[b]).max() <= 1e-4
    dst = Far([200, 200], heads, dim, ps, pool, seed=2, shared=p)
    run_evict(p, dst, w, lens, [200, 200], 32)
    p.check_codes()


# ------------------------------------------------------------------ capture

@pytest.mark.parametrize("new", [1, 40])
def test_captured_calls_draw_workspaces_of_their_own(new):
    """Two graphs of calls without a workspace argument, replayed alternately and
    at once on two streams, between eager calls."""
    cases = []
    for seed, lens in ((1, [9000, 1500]), (2, [8600, 8900])):
        p = filled(lens, 2, 128, 64, seed=seed)
        cu, q = dev(cu_of([new, new])), randn(2 * new, 8, 128, seed=seed).cuda()
        args = (q, p.dev, cu, dev(lens), new, max(lens))
        assert api.attn_cache_fwd_workspace_size(p.dev, 2 * new, 8, new, max(lens)) > 0
        want = [x.clone() for x in api.attn_cache_fwd(*args)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = api.attn_cache_fwd(*args)
        cases.append((graph, out, want, args))
    sides = [torch.cuda.Stream() for _ in range(2)]
    for together in (False, True, False):
        for _, out, _, _ in cases:
            for x in out:
                x.fill_(9)
        torch.cuda.synchronize()
        for side, (graph, out, want, args) in zip(sides, cases):
            with torch.cuda.stream(side):
                graph.replay()
            if not together:
                torch.cuda.synchronize()
                junk = torch.full((1 << 22,), 7.0, device="cuda")  # what the allocator holds free is overwritten
                for a, b in zip(want, api.attn_cache_fwd(*args)):
                    assert torch.equal(a, b)
                del junk
        torch.cuda.synchronize()
        for _, out, want, _ in cases:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


# ------------------------------------------------------------------ arguments that the documentation allows

@pytest.mark.parametrize("new", [1, 3, 20, 200])
@pytest.mark.parametrize("length", [400, 5000, 20000])
def test_results_over_the_queries(new, length):
    lens = [length, 300]
    p = filled(lens, 2, 64, 32, seed=7)
    cu, q = cu_of([new, new]), randn(2 * new, 6, 64, seed=1).cuda()
    want = [x.clone() for x in run_attend(p, q, cu, lens)]
    o, lse = run_attend(p, q, cu, lens, out=q)
    assert o is q and torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_a_page_twice_in_one_sequence():
    p = filled([192, 64], 2, 64, 64, seed=9)
    p.table[0, 2] = p.table[0, 0]
    p.dev.page_table.copy_(torch.from_numpy(p.table))
    p.ref.table = p.table
    for new in (1, 30):
        check_attend(p, randn(2 * new, 4, 64, seed=1), cu_of([new, new]), [192, 64])


def test_workspaces_that_do_not_fit():
    p = filled([9000], 1, 64, 32, seed=2)
    q, cu, lens = randn(1, 4, 64).cuda(), dev([0, 1]), dev([9000])
    need = api.attn_cache_fwd_workspace_size(p.dev, 1, 4, 1, 9000)
    ws = torch.empty(need + 512, dtype=torch.uint8, device="cuda")
    api.attn_cache_fwd(q, p.dev, cu, lens, 1, 9000, workspace=ws[256:])
    for bad in (ws[1:], ws[128:], ws[:need].cpu()):
        with pytest.raises(api.AttnError):
            api.attn_cache_fwd(q, p.dev, cu, lens, 1, 9000, workspace=bad)


@pytest.mark.parametrize("new", [1, 2])
def test_thousands_of_short_sequences(new):
    """More sequences than a CTA's threads and than the GPU's CTAs, some empty, some
    without new tokens."""
    rng = np.random.default_rng(4)
    n = rng.integers(0, new + 1, 3000)
    lens = [int(x) for x in n + rng.integers(0, 40, 3000)]
    p = filled(lens, 1, 32, 16, seed=11)
    cu = cu_of(n)
    q = randn(int(cu[-1]), 2, 32, seed=12)
    check_attend(p, q, cu, lens, max_new=new)
    o, lse = run_attend(p, q, cu, lens, max_new=new)
    w = api.attn_cache_weights(q.cuda(), lse, p.dev, dev(cu), dev(lens), new, max(lens)).cpu()
    ref, _ = p.ref.weights(q.double().numpy(), lse.cpu().numpy(), cu, lens)
    for b, L in enumerate(lens):
        if L:
            assert np.abs(w[b, :, :L].double().numpy() - ref[b]).max() <= 1e-4


@pytest.mark.parametrize("rows", [1, 48, 200])
def test_queries_of_a_wide_range(rows):
    """Elements from 2^-14 of the row's largest up: with many rows an element below
    2^-9 of the largest, m, may be off by 2^-17 m, a score by scale 2^-17 m
    sum |k|, on top of the usual bounds."""
    lens = [500]
    p = filled(lens, 1, 64, 64, seed=21, spread=False)
    g = torch.Generator().manual_seed(1)
    q = torch.randn((rows, 1, 64), generator=g) * 2.0 ** torch.randint(-14, 1, (rows, 1, 64), generator=g)
    q = (4 * q).to(torch.bfloat16)
    o, lse = run_attend(p, q, cu_of([rows]), lens)
    O, L, terms, spread = p.ref.attend(q.double().numpy(), cu_of([rows]), lens)
    K = np.abs(p.ref.numbers(0, 0, 500)).sum(-1).max()
    m = np.abs(q.double().numpy()).max(-1)
    off = 0.0 if rows <= 16 else 2.0 ** -17 * m * K / 8  # [rows, 1]
    A = terms[0].max()
    rel = 2 * ((64 + 4) * 2.0 ** -24 * A) + 2.0 ** -22 + 2.0 ** -23 * (2 * A + 16) + 500 * 2.0 ** -24
    assert (np.abs(lse.double().cpu().numpy() - L) <= rel + np.transpose(off + 0 * m) + 2.0 ** -22 * np.abs(L)).all()
    small = 2.0 ** -25 * p.ref.code_sums(1, 0, 500)[None]
    # each weight moves by e^+-(off + rel), the sum too
    tol = (2.0 ** -11 + 3 * rel + 2 * np.expm1(2 * (off + 0 * m))[..., None]) * spread + small
    tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(O)
    assert (np.abs(o.double().cpu().numpy() - O) <= tol).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,page_size,heads,group,new", [
    (128, 64, 2, 1, [25, 0, 3, 25]), (64, 16, 1, 5, [64, 1, 0, 60]), (32, 128, 3, 2, [70, 64, 1, 129]),
    (128, 32, 1, 8, [64, 9, 33, 0]), (128, 128, 2, 2, [150, 1, 2, 300])])
def test_weights_of_many_rows(dim, page_size, heads, group, new, causal):
    """More than 24 rows, in one and in several passes of 128; sequences without
    queries; sums on top of others, in place too.  Every score may be off by the
    usual roundings and by scale 2^-17 m sum |k|, m the row's largest element."""
    lens = [700, 64, 130, 1300]
    p = filled(lens, heads, dim, page_size, seed=dim + page_size, spread=False)
    cu = cu_of(new)
    q = randn(int(cu[-1]), heads * group, dim, seed=5)
    _, lse = run_attend(p, q, cu, lens, causal)
    g = torch.Generator().manual_seed(2)
    before = torch.rand((4, heads, 1301), generator=g)
    ref, terms = p.ref.weights(q.double().numpy(), lse.cpu().numpy(), cu, lens, causal)
    args = (q.cuda(), lse, p.dev, dev(cu), dev(lens), max(new), 1300, "causal" if causal else "none")
    out = torch.full((4, heads, 1301), 3.0, device="cuda")
    apart = api.attn_cache_weights(*args, prev=before.cuda(), out=out)
    x = before.cuda()
    assert torch.equal(api.attn_cache_weights(*args, prev=x, out=x)[:, :, :64], apart[:, :, :64])
    alone = api.attn_cache_weights(*args)
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
    for got, was, behind in ((apart, before, 3.0), (x, before, None), (alone, 0 * before, 0.0)):
        got = got.double().cpu().numpy()
        for b, n in enumerate(lens):
            A = terms[b].max(initial=0)
            m = np.abs(q[cu[b]:cu[b + 1]].double().numpy()).max(initial=0)
            off = 2.0 ** -17 * m * np.abs(p.ref.numbers(0, b, n)).sum(-1).max() / np.sqrt(dim)
            rel = 2 * (dim + 4) * 2.0 ** -24 * A + 2.0 ** -22 + 2.0 ** -22 * (2 * A + 16) + new[b] * group * 2.0 ** -24
            w = was[b, :, :n].double().numpy()
            err = np.abs(got[b, :, :n] - (w + ref[b]))
            # a pass of 128 rows adds to what the last one left: a rounding of the sum each
            assert (err <= (rel + np.expm1(off)) * ref[b] + (-(-new[b] * group // 128) + 1) * 2.0 ** -24 * (w + ref[b])
                    + 1e-37).all()
            want = was[b, :, n:got.shape[2]].double().numpy() if behind is None else behind
            assert (got[b, :, n:] == want).all()


def test_weights_of_many_rows_leave_out_bad_pages():
    p = filled([300, 200], 2, 64, 32, seed=1)
    cu, lens = dev([0, 40, 80]), dev([300, 200])
    q = randn(80, 4, 64, seed=1).cuda()
    lse = torch.zeros((4, 80), device="cuda")
    good = api.attn_cache_weights(q, lse, p.dev, cu, lens, 40, 300)
    for bad in (-1, p.dev.num_pages):
        was = p.dev.page_table[0, 2].item()
        p.dev.page_table[0, 2] = bad
        got = api.attn_cache_weights(q, lse, p.dev, cu, lens, 40, 300)
        assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT
        assert (got[0, :, 64:96] == 0).all()
        got[0, :, 64:96] = good[0, :, 64:96]
        assert torch.equal(got, good)
        p.dev.page_table[0, 2] = was


@pytest.mark.parametrize("dim", [64, 128])
def test_attention_and_weights_of_many_rows_at_once(dim):
    """Two streams, both kernels on the tensor cores; captured and replayed with other
    lengths and queries too."""
    lens = [3000, 1800, 2500]
    p = filled(lens, 2, dim, 64, seed=5)
    cu, q = cu_of([40, 40, 40]), randn(120, 4, dim, seed=1).cuda()
    d_cu, d_lens = dev(cu), dev(lens)
    attend = lambda **kw: api.attn_cache_fwd(q, p.dev, d_cu, d_lens, 40, 3000, **kw)  # noqa: E731
    o, lse = [x.clone() for x in attend()]
    weigh = lambda **kw: api.attn_cache_weights(q, lse, p.dev, d_cu, d_lens, 40, 3000, **kw)  # noqa: E731
    w = weigh().clone()
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        outs.append((attend(stream=sides[0]), weigh(stream=sides[1])))
    torch.cuda.synchronize()
    for (a, b), c in outs:
        assert torch.equal(a, o) and torch.equal(b, lse) and torch.equal(c, w)
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK

    go, glse, gw = torch.empty_like(o), torch.empty_like(lse), torch.zeros_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attend(out=go, lse=glse)
        api.attn_cache_weights(q, glse, p.dev, d_cu, d_lens, 40, 3000, out=gw)
    new = [40, 1799, 2000]
    q.copy_(randn(120, 4, dim, seed=2))
    d_lens.copy_(dev(new))
    graph.replay()
    torch.cuda.synchronize()
    want_o, want_lse = attend()
    want_w = api.attn_cache_weights(q, want_lse, p.dev, d_cu, d_lens, 40, 3000)
    assert torch.equal(go, want_o) and torch.equal(glse, want_lse) and torch.equal(gw, want_w)


@pytest.mark.parametrize("new,group", [(1, 1), (1, 8), (4, 4), (2, 5)])
@pytest.mark.parametrize("batch,heads,most", [(1, 1, 8192), (1, 1, 8193), (3, 2, 5000), (2, 20, 4096), (5, 20, 2000),
                                              (20, 10, 900), (20, 10, 1025), (9, 30, 800), (48, 10, 700)])
def test_sequences_cut_in_every_way(batch, heads, most, new, group):
    """A (sequence, head) by one CTA, by clusters of 2, 4 and 8, and on the cut line;
    lengths from 0 up, shorter than the cluster has pieces, uneven."""
    rng = np.random.default_rng(batch * most)
    n = [int(x) for x in rng.integers(0, new + 1, batch)]
    n[0] = new
    lens = [max(a, int(most * rng.random() ** 3)) for a in n]
    lens[0] = most
    if batch > 2:
        lens[1], lens[2] = max(n[1], 60), n[2]
    p = filled(lens, heads, 32, 32, seed=batch)
    cu, q = cu_of(n), randn(sum(n) + 2, heads * group, 32, seed=most)
    for causal in (True, False):
        o, lse = check_attend(p, q, cu, lens, causal)
        for a, b in zip((o, lse), run_attend(p, q, cu, lens, causal)):
            rows = sum(n)
            assert torch.equal(a[:rows] if a is o else a[:, :rows], b[:rows] if a is o else b[:, :rows])
