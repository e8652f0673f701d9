"""The 8-bit key / value cache on the GPU against the fp64 oracle.

Codes, scales, kept indices and lengths have to be equal.  Computed outputs
have tolerances from the arithmetic (attend_bounds, weight_bounds):
  * a score is a sum of D products, exact in fp16 x fp16, accumulated in fp32,
    then three fp32 roundings: off by at most ds = (D + 4) 2^-24 A, A = the row's
    largest scale sum |q k|; ex2 is good to 2^-22, and its argument, a difference
    of numbers up to |s| + |m|, to 2^-23 of them (A bounds both, the page scales'
    exponents, at most 16 here, add 16 2^-23);
    q is exact in fp16 down to 2^-25 of its row's largest value: D 2^-25 relative
    to A at most, within ds doubled;
  * a weight is rounded to fp16 (2^-11 of itself, or 2^-25 where it is below 2^-14
    of the largest), which the sum of the weights is not;
  * sums over L tokens in fp32 add L 2^-24; O is rounded to bf16, 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

from block_sparse_masked_mask_gb300 import api
from oracle import cache as C

pytestmark = pytest.mark.gpu


def cu_of(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def table_for(lens, page_size, rng, extra=2, width=None):
    """Shuffled pages for sequences of these lengths; entries that no token
    needs hold a number outside the pool (they must not be read)."""
    need = [-(-t // page_size) for t in lens]
    pool = sum(need) + extra
    order = rng.permutation(pool)
    width = max(1, max(need)) if width is None else width
    table = np.full((len(lens), width), 1 << 28, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pool


class Pair:
    """The same cache on the device and in the oracle, filled with junk codes
    (NaN among them) so that stale slots matter."""

    def __init__(self, lens, heads, dim, page_size, seed=0, width=None):
        rng = np.random.default_rng(seed)
        self.table, pool = table_for(lens, page_size, rng, width=width)
        codes = [rng.integers(0, 256, (pool, heads, page_size, dim)).astype(np.uint8) for _ in range(2)]
        scale = [2.0 ** rng.integers(-3, 4, (pool, heads)).astype(np.float64) for _ in range(2)]
        self.ref = C.Cache(*codes, *scale, self.table)
        dev = [torch.from_numpy(x).cuda() for x in codes]
        devs = [torch.from_numpy(x.astype(np.float32)).cuda() for x in scale]
        self.dev = api.KVCache(*dev, *devs, torch.from_numpy(self.table).cuda())

    def append(self, k, v, cu, lens, max_new=None):
        n = int(np.diff(cu).max())
        api.attn_cache_append(k.cuda(), v.cuda(), self.dev, dev(cu), dev(lens), n if max_new is None else max_new)
        self.ref.append(k.double().numpy(), v.double().numpy(), cu, lens)

    def check_codes(self):
        for got, want in ((self.dev.k_pages, self.ref.codes[0]), (self.dev.v_pages, self.ref.codes[1])):
            assert np.array_equal(got.cpu().numpy(), want)
        for got, want in ((self.dev.k_scale, self.ref.scale[0]), (self.dev.v_scale, self.ref.scale[1])):
            assert np.array_equal(got.cpu().double().numpy(), want)


def dev(x):
    return torch.from_numpy(np.asarray(x, np.int32)).cuda()


def randn(*shape, seed=0, dtype=torch.bfloat16, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


def filled(lens, heads, dim, page_size, seed=0, spread=True):
    """A cache whose sequences hold random tokens, appended in one call."""
    p = Pair(lens, heads, dim, page_size, seed)
    T = int(np.sum(lens))
    k, v = randn(max(T, 1), heads, dim, seed=seed + 1), randn(max(T, 1), heads, dim, seed=seed + 2)
    if spread and T:  # values of very different size from token to token
        v = v * (2.0 ** torch.randint(-4, 4, (T, 1, 1), generator=torch.Generator().manual_seed(seed))).to(v.dtype)
    if T:
        p.append(k[:T], v[:T], cu_of(lens), lens)
    return p


def attend_bounds(ref, ref_o, spread, terms, cu, lens, dim):
    """(O bound, LSE slack per sequence) from the docstring's arithmetic."""
    tol = np.zeros(ref_o.shape)
    slack = []
    for b, L in enumerate(lens):
        A = terms[b].max(initial=0)
        rel = 2 * ((dim + 4) * 2.0 ** -24 * A) + 2.0 ** -22 + 2.0 ** -23 * (2 * A + 16) + L * 2.0 ** -24
        slack.append(rel)
        s = slice(cu[b], cu[b + 1])
        # weights below 2^-14 of the largest: 2^-25 times each code, in units of the largest scale
        small = 2.0 ** -25 * ref.code_sums(1, b, L)
        tol[s] = (2.0 ** -11 + 3 * rel) * spread[s] + np.repeat(small, ref_o.shape[1] // small.shape[0], 0)[None]
        tol[s] = tol[s] * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref_o[s])
    return tol, slack


def run_attend(pair, q, cu, lens, causal=True, scale=0.0, max_new=None, max_seqlen=None, **kw):
    n = int(np.diff(cu).max()) if max_new is None else max_new
    L = int(max(lens)) if max_seqlen is None else max_seqlen
    return api.attn_cache_fwd(q.cuda(), pair.dev, dev(cu), dev(lens), n, L, kind="causal" if causal else "none",
                              scale=scale, **kw)


def check_attend(pair, q, cu, lens, causal=True, scale=0.0, **kw):
    o, lse = run_attend(pair, q, cu, lens, causal, scale, **kw)
    assert api.attn_cache_get_status(pair.dev) == api.ATTN_OK
    T = int(cu[-1])
    q = q[:T]
    O, L, terms, spread = pair.ref.attend(q.double().numpy(), cu, lens, causal, scale)
    tol, slack = attend_bounds(pair.ref, O, spread, terms, cu, lens, q.shape[2])
    got = o.double().cpu().numpy()
    err = np.abs(got[:T] - O[:T])
    assert (err <= tol[:T]).all(), f"O: max err {err.max()}, worst ratio {(err / np.maximum(tol[:T], 1e-300)).max()}"
    gl = lse.double().cpu().numpy()[:, :T]
    for b in range(len(lens)):
        s = slice(cu[b], cu[b + 1])
        seen = np.isfinite(L[:, s])
        assert np.array_equal(np.isneginf(gl[:, s]), ~seen)
        d = np.abs(gl[:, s][seen] - L[:, s][seen])
        assert (d <= slack[b] + 2.0 ** -22 * np.abs(L[:, s][seen])).all(), f"LSE: {d.max()} vs {slack[b]}"
    return o, lse


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
def test_append_in_steps(page_size, dim, dtype):
    """Ragged appends one behind the other: new pages, pages begun earlier whose
    scale stays or grows, empty additions; codes and scales equal the oracle's."""
    final = [page_size * 2 + 3, 1, 0, page_size, 5 * page_size - 1]
    p = Pair(final, 3, dim, page_size, seed=page_size + dim)
    held = np.zeros(5, np.int64)
    for step, share in enumerate((0.3, 0.3, 0.5, 1.0)):
        left = np.asarray(final) - held
        n = np.ceil(left * share).astype(np.int64)
        if step == 1:
            n[0] = 0
        T = int(n.sum())
        if T == 0:
            continue
        # each step's values are larger or smaller than the one before
        k = randn(T, 3, dim, seed=step, dtype=dtype, scale=(1.0, 30.0, 0.01, 5.0)[step])
        v = randn(T, 3, dim, seed=10 + step, dtype=dtype, scale=(2.0, 0.5, 1e4, 1e-3)[step])
        held = held + n
        p.append(k, v, cu_of(n), held, max_new=int(n.max()) + (7 if step == 2 else 0))
        assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
        p.check_codes()


def test_append_values_at_the_edges():
    """Zeros, the border of a scale (448 2^e and the next number), subnormal
    codes, the scales' limits, infinities and NaN."""
    rows = [torch.zeros(32), torch.full((32,), 7.0), torch.full((32,), 7.0 * (1 + 2.0 ** -7)), torch.full((32,), 1e-38),
            torch.full((32,), 3e38), torch.linspace(-1, 1, 32) * 2.0 ** -8]
    rows[5][0] = 448.0
    special = torch.linspace(-3, 3, 32)
    special[3], special[4], special[5] = float("inf"), float("-inf"), float("nan")
    rows += [special, torch.full((32,), float("inf")), torch.full((32,), float("nan")), -torch.zeros(32)]
    n = len(rows)
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.stack(rows)[:, None, :].to(dtype)
        # each row in a page of its own: n sequences of one token
        p = Pair([1] * n, 1, 32, 16, seed=3)
        p.append(x, x.flip(0), cu_of([1] * n), [1] * n)
        p.check_codes()


def test_append_again_and_strided():
    """The same append twice stores the same codes; k and v may be slices of one
    projection; rows behind the last sequence and slots behind the last token
    are left alone (check_codes compares the whole pools)."""
    lens, n = [70, 33], [40, 33]
    p = Pair(lens, 2, 64, 32, seed=9)
    k0, v0 = randn(30, 2, 64, seed=1), randn(30, 2, 64, seed=2)
    p.append(k0, v0, cu_of([30, 0]), [30, 0])
    wide = randn(80, 6 * 64 + 16, seed=3).cuda()
    k, v = wide[:, :128].unflatten(1, (2, 64)), wide[:, 256:384].unflatten(1, (2, 64))
    for _ in range(2):
        api.attn_cache_append(k, v, p.dev, dev(cu_of(n)), dev(lens), 40)
    p.ref.append(k.double().cpu().numpy()[:73], v.double().cpu().numpy()[:73], cu_of(n), lens)
    p.check_codes()


# ------------------------------------------------------------------ attention

LENGTHS = [[1], [16, 17, 15], [0, 5, 300], [1000, 64, 0, 129], [2047, 1], [4097]]


@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4), (1, 16), (3, 5)])
@pytest.mark.parametrize("dim,page_size", [(128, 64), (64, 16), (32, 128), (128, 32)])
def test_decode(dim, page_size, heads, group, lens):
    """One query per sequence, lengths from none to several chunks."""
    p = filled(lens, heads, dim, page_size, seed=len(lens) + dim)
    n = [1 if t else 0 for t in lens]
    cu = cu_of(n)
    q = randn(max(int(cu[-1]), 1), heads * group, dim, seed=5)
    check_attend(p, q, cu, lens)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,page_size,heads,group", [(128, 128, 2, 2), (64, 32, 1, 8), (32, 16, 2, 3), (128, 64, 4, 1)])
def test_several_new_tokens(dim, page_size, heads, group, causal):
    """Queries of chunks: causal inside the chunk, sequences that are all new,
    that have no new token, and whose rows see nothing (more queries than
    tokens)."""
    lens, n = [700, 130, 257, 64, 3, 0], [33, 130, 1, 0, 9, 4]
    p = filled(lens, heads, dim, page_size, seed=21)
    cu = cu_of(n)
    q = randn(int(cu[-1]), heads * group, dim, seed=6, scale=2.0)
    check_attend(p, q, cu, lens, causal)


@pytest.mark.parametrize("n", [2, 17, 64, 129, 300])
def test_long_chunks(n):
    lens = [n + 900, n, n + 1]
    p = filled(lens, 2, 128, 64, seed=n)
    cu = cu_of([n] * 3)
    check_attend(p, randn(3 * n, 8, 128, seed=n), cu, lens)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,page_size,heads,group", [(64, 16, 4, 4), (128, 64, 5, 3)])
def test_many_items_of_many_rows(dim, page_size, heads, group, causal):
    """Several tiles of rows per sequence, tiles of one and of two halves in turn,
    more of them than there are SMs, sequences with no new token or no token between."""
    n = [(37 * i) % 150 if i % 7 else 0 for i in range(45)]
    lens = [x + (53 * i) % 700 if i % 11 else x // 2 for i, x in enumerate(n)]
    p = filled(lens, heads, dim, page_size, seed=23)
    cu = cu_of(n)
    check_attend(p, randn(int(cu[-1]), heads * group, dim, seed=3), cu, lens, causal)


def test_one_long_item_over_many_ctas():
    """Few rows above 16 over a long sequence, and a tile and a half of rows."""
    for rows in (20, 390):
        p = filled([9001], 1, 64, 64, seed=rows)
        check_attend(p, randn(rows, 1, 64, seed=rows), cu_of([rows]), [9001])


def test_large_scores_and_scales():
    """Scores in the hundreds (a one-hot softmax), a given scale, tiny and huge queries."""
    lens = [333, 80]
    p = filled(lens, 2, 64, 32, seed=33)
    cu = cu_of([2, 2])
    for size, scale in ((60.0, 0.0), (1.0, 3.0), (1e-30, 0.0), (1e30, 1e-30)):
        check_attend(p, randn(4, 4, 64, seed=7, scale=size), cu, lens, scale=scale)


def test_rows_behind_the_last_sequence_and_bounds_above_the_sizes():
    lens = [100, 40]
    p = filled(lens, 1, 128, 64, seed=41)
    cu = cu_of([3, 2])
    q = randn(9, 4, 128, seed=8)
    q[5:] = float("nan")
    o, lse = torch.full((9, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, 9), 5.0, device="cuda")
    check_attend(p, q[:5], cu, lens)
    # (bounds choose the cut into tiles and with it the order of the sums: within the same tolerance, not bit for bit)
    check_attend(p, q, cu, lens, max_new=9, max_seqlen=128, out=o, lse=lse)
    assert (o[5:] == 5).all() and (lse[:, 5:] == 5).all()


def test_shared_pages():
    """Two sequences that read one prefix's pages."""
    p = filled([128, 200], 2, 64, 64, seed=51)
    p.table[0, :2] = p.table[1, :2]
    p.dev.page_table.copy_(torch.from_numpy(p.table))
    p.ref.table = p.table
    check_attend(p, randn(2, 4, 64, seed=9), cu_of([1, 1]), [128, 200])


def test_attention_after_appends_step_by_step():
    """rope -> append -> attend, a prompt and then single tokens, against the
    oracle's own cache."""
    heads, group, dim, ps = 2, 3, 64, 32
    prompt, steps = np.array([37, 64, 1]), 4
    p = Pair(list(prompt + steps), heads, dim, ps, seed=61)
    plan = api.attn_rope_plan(dim, interleaved=True)
    held = np.zeros(3, np.int64)
    for step in range(1 + steps):
        n = prompt if step == 0 else np.ones(3, np.int64)
        held = held + n
        cu, T = cu_of(n), int(n.sum())
        q, k, v = (randn(T, h, dim, seed=100 * step + i).cuda() for i, h in enumerate((heads * group, heads, heads)))
        q, k = api.attn_rope(q, k, plan, cu_seqlens=dev(cu), seq_lens=dev(held))
        p.append(k.cpu(), v.cpu(), cu, held)
        p.check_codes()
        check_attend(p, q.cpu(), cu, held)


def test_repeats_streams_and_graphs():
    """Bit-identical repeats; two calls at once on two streams; a captured step
    replayed on other inputs, lengths and pages."""
    lens = [3000, 1500, 70]
    p = filled(lens, 2, 128, 64, seed=71)
    cu, q = cu_of([1, 1, 1]), randn(3, 8, 128, seed=1).cuda()
    first = [x.clone() for x in run_attend(p, q, cu, lens)]
    for _ in range(3):
        for a, b in zip(first, run_attend(p, q, cu, lens)):
            assert torch.equal(a, b)
    d_cu, d_lens = dev(cu), dev(lens)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = [api.attn_cache_fwd(q, p.dev, d_cu, d_lens, 1, 3000, stream=s) for s in sides]
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(first, out))

    o, lse = torch.empty_like(q), torch.empty((8, 3), device="cuda")
    w = torch.zeros((3, 2, 3000), device="cuda")
    ws = torch.empty(max(1, api.attn_cache_fwd_workspace_size(p.dev, 3, 8, 1, 3000)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.attn_cache_fwd(q, p.dev, d_cu, d_lens, 1, 3000, out=o, lse=lse, workspace=ws)
        api.attn_cache_weights(q, lse, p.dev, d_cu, d_lens, 1, 3000, out=w)
    new = [1000, 1400, 1]
    q.copy_(randn(3, 8, 128, seed=2))
    d_lens.copy_(dev(new))
    graph.replay()
    torch.cuda.synchronize()
    want = run_attend(p, q, cu, new, max_seqlen=3000)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    ref, _ = p.ref.weights(q.double().cpu().numpy(), lse.cpu().numpy(), cu, new)
    assert np.abs(w[1, :, :1400].cpu().numpy() - ref[1]).max() <= 1e-4
    assert (w[0, :, 1000:] == 0).all()


# ------------------------------------------------------------------ weights

def check_weights(p, q, cu, lens, causal=True, width=None, prev=None, in_place=False):
    o, lse = run_attend(p, q, cu, lens, causal)
    L = int(max(lens))
    heads = p.dev.num_kv_heads
    width = width or max(L, 1)
    before = torch.rand((len(lens), heads, width), generator=torch.Generator().manual_seed(1)) if prev else None
    start = torch.full((len(lens), heads, width), 3.0) if before is None else before
    out = start.cuda()
    prev_dev = None if before is None else (out if in_place else before.cuda())
    n = int(np.diff(cu).max())
    got = api.attn_cache_weights(q.cuda(), lse, p.dev, dev(cu), dev(lens), n, L, kind="causal" if causal else "none",
                                 prev=prev_dev, out=out)
    assert got is out and api.attn_cache_get_status(p.dev) == api.ATTN_OK
    ref, terms = p.ref.weights(q.double().numpy(), lse.cpu().numpy(), cu, lens, causal)
    got = got.double().cpu().numpy()
    for b, total in enumerate(lens):
        was = 0 if before is None else before[b, :, :total].double().numpy()
        A = terms[b].max(initial=0)
        rows = (cu[b + 1] - cu[b]) * q.shape[1] // heads
        rel = 2 * (q.shape[2] + 4) * 2.0 ** -24 * A + 2.0 ** -22 + 2.0 ** -22 * (2 * A + 16) + rows * 2.0 ** -24
        err = np.abs(got[b, :, :total] - (was + ref[b]))
        tol = rel * ref[b] + 2.0 ** -23 * (was + ref[b]) + 1e-37
        assert (err <= tol).all(), f"max err {err.max(initial=0)}, ratio {(err / tol).max(initial=0)}"
        assert np.array_equal(got[b, :, total:], start[b, :, total:].double().numpy())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,page_size,heads,group", [(128, 64, 2, 4), (64, 16, 1, 5), (32, 128, 3, 1), (128, 16, 1, 16)])
def test_weights_received(dim, page_size, heads, group, causal):
    lens, n = [700, 130, 257, 64, 3, 0, 33], [33, 130, 1, 0, 9, 4, 1]
    p = filled(lens, heads, dim, page_size, seed=81)
    cu = cu_of(n)
    q = randn(int(cu[-1]), heads * group, dim, seed=6)
    check_weights(p, q, cu, lens, causal)
    check_weights(p, q, cu, lens, causal, width=1024, prev=True)
    check_weights(p, q, cu, lens, causal, prev=True, in_place=True)


def test_weights_of_a_decode_step_sum_to_the_queries():
    """Each query's weights sum to one: a sequence's total is its number of rows
    (within the relative error of its terms, 1e-4 here)."""
    lens = [1, 511, 4097]
    p = filled(lens, 2, 128, 64, seed=91)
    q, cu = randn(3, 8, 128, seed=2).cuda(), dev(cu_of([1, 1, 1]))
    o, lse = api.attn_cache_fwd(q, p.dev, cu, dev(lens), 1, 4097)
    w = api.attn_cache_weights(q, lse, p.dev, cu, dev(lens), 1, 4097)
    assert (w.double().sum(-1) - 4).abs().max() <= 4e-4


# ------------------------------------------------------------------ eviction

def run_evict(p, dst, weights, lens, budgets, recent, max_keep=None, width=None):
    keep = [min(a, b) for a, b in zip(lens, budgets)]
    most = max(keep) if max_keep is None else max_keep
    nw = None if width is None else torch.full((len(lens), p.dev.num_kv_heads, width), 9.0, device="cuda")
    kept, nw, nl = api.attn_cache_evict(weights.cuda(), p.dev, dst.dev, dev(lens), dev(budgets), recent,
                                        int(max(lens)), most, new_weights=nw)
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK and api.attn_cache_get_status(dst.dev) == api.ATTN_OK
    ref = p.ref.evict(weights.numpy(), lens, budgets, recent, dst.ref)
    dst.check_codes()
    assert nl.cpu().tolist() == keep
    kept, nw = kept.cpu().numpy(), nw.cpu()
    for b, n in enumerate(keep):
        assert np.array_equal(kept[b, :, :n], ref[b]) and (kept[b, :, n:] == -1).all()
        want = torch.gather(weights[b], 1, torch.from_numpy(ref[b]))
        got = nw[b, :, :n]
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(5.), want.nan_to_num(5.))
        assert (nw[b, :, n:] == 0).all()
    return keep


@pytest.mark.parametrize("dim,page_size", [(128, 64), (64, 16), (32, 128), (128, 32)])
@pytest.mark.parametrize("recent", [0, 7, 10_000])
def test_evict(dim, page_size, recent):
    lens = [1, 300, 0, 2049, 64, 1500]
    budgets = [1, 100, 5, 1025, 100, 0]
    p = filled(lens, 2, dim, page_size, seed=recent + dim)
    g = torch.Generator().manual_seed(recent)
    w = torch.exp(2 * torch.randn((6, 2, 2050), generator=g))
    dst = Pair([min(a, b) for a, b in zip(lens, budgets)], 2, dim, page_size, seed=5)
    run_evict(p, dst, w, lens, budgets, recent)


def test_evict_ties_and_strange_weights():
    """Few distinct weights (ties to the lower index), all equal, zeros of both
    signs, infinities, NaN, negative and subnormal weights; a wide result."""
    L, keep = 1200, 500
    g = torch.Generator().manual_seed(0)
    few = torch.randint(0, 3, (L,), generator=g).float()
    same = torch.full((L,), 0.25)
    zeros = torch.where(torch.rand(L, generator=g) < 0.5, 0.0, -0.0)
    odd = torch.randn(L, generator=g)
    odd[::7], odd[1::7], odd[2::7], odd[3::7] = float("nan"), float("-inf"), float("inf"), 1e-42
    close = 1 + torch.randint(0, 4, (L,), generator=g) * 2.0 ** -23
    w = torch.stack([few, same, zeros, odd, close])[:, None].repeat(1, 2, 1)
    w[:, 1] = w[:, 1].flip(-1)
    lens = [L] * 5
    p = filled(lens, 2, 32, 16, seed=3)
    for recent in (0, 33):
        dst = Pair([keep] * 5, 2, 32, 16, seed=8)
        run_evict(p, dst, w, lens, [keep] * 5, recent, max_keep=keep + 12, width=700)


def test_evict_drops_the_thinking_first():
    """Weights of -inf name the tokens to drop: with a budget of the others the
    cache then holds just those, as the strip-thinking mask would show them."""
    L = 400
    role = np.zeros(L, bool)
    role[50:170], role[220:330] = True, True
    keep = int((~role).sum())
    p = filled([L], 2, 64, 32, seed=12)
    w = torch.rand((1, 2, L))
    w[:, :, torch.from_numpy(role)] = float("-inf")
    dst = Pair([keep], 2, 64, 32, seed=13)
    run_evict(p, dst, w, [L], [keep], 0)
    q = randn(1, 4, 64, seed=3)
    check_attend(dst, q, cu_of([1]), [keep])
    # the same as attention over all tokens with the thinking masked out
    o, _ = run_attend(dst, q, cu_of([1]), [keep])
    K, V = p.ref.numbers(0, 0, L)[:, ~role], p.ref.numbers(1, 0, L)[:, ~role]
    for h in range(4):
        s = K[h // 2] @ q[0, h].double().numpy() / 8
        x = np.exp(s - s.max())
        want = x @ V[h // 2] / x.sum()
        # both are within the attention's bound of it; moved codes lose nothing but subnormals
        assert np.abs(o[0, h].double().cpu().numpy() - want).max() <= 2.0 ** -6 * np.abs(V[h // 2]).max()


def test_the_whole_chain():
    """append -> attend -> weigh -> evict -> append -> attend, weights carried on."""
    heads, group, dim, ps, width = 2, 2, 64, 16, 256
    lens = [150, 97]
    p = filled(lens, heads, dim, ps, seed=31)
    cu = cu_of([4, 4])
    q = randn(8, heads * group, dim, seed=4)
    o, lse = check_attend(p, q, cu, lens)
    w = api.attn_cache_weights(q.cuda(), lse, p.dev, dev(cu), dev(lens), 4, 150).cpu()
    dst = Pair([81, 81], heads, dim, ps, seed=32)  # room for one more token
    keep = run_evict(p, dst, w, lens, [80, 80], 16, width=width)
    assert keep == [80, 80]
    k, v = randn(2, heads, dim, seed=5, scale=3.0), randn(2, heads, dim, seed=6)
    dst.append(k, v, cu_of([1, 1]), [81, 81])
    dst.check_codes()
    check_attend(dst, randn(2, heads * group, dim, seed=7), cu_of([1, 1]), [81, 81])


# ------------------------------------------------------------------ refusals on the device

def test_bad_numbers_are_reported_and_left_out():
    """Malformed cu_seqlens or lengths and page numbers outside the pool are read
    back as a status; nothing of the sequence is written, other sequences are
    right, and the status is cleared by the reading."""
    lens = [100, 90, 80]
    p = filled(lens, 1, 64, 32, seed=1)
    cu = cu_of([1, 1, 1])
    q = randn(3, 2, 64, seed=1)
    good, _ = run_attend(p, q, cu, lens)
    good = good.clone()
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
    codes = p.dev.k_pages.clone()
    for bad_cu, bad_lens in ((cu, [100, -1, 80]), (cu, [100, 97, 80]), ([0, 1, 3, 3], lens), ([0, 1, 0, 1], lens),
                             ([0, 1, 5, 3], lens)):
        out = torch.full((3, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        kw = dict(max_new=1, max_seqlen=96, out=out)
        run_attend(p, q, np.asarray(bad_cu), bad_lens, **{**kw, "max_seqlen": 100 if bad_lens[1] != 97 else 96})
        assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT
        assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
        assert (out[1] == 5).all()
        api.attn_cache_append(torch.ones((3, 1, 64), device="cuda"), torch.ones((3, 1, 64), device="cuda"), p.dev,
                              dev(bad_cu), dev([0, -1, 0]), 1)
        assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT
        assert torch.equal(p.dev.k_pages, codes)
    # a bad page: its tokens are left out, the rest of the sequence counts
    for bad in (-1, p.dev.num_pages, 2 ** 31 - 1):
        was = p.dev.page_table[1, 1].item()
        p.dev.page_table[1, 1] = bad
        out, _ = run_attend(p, q, cu, lens)
        assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2]) and torch.isfinite(out).all()
        w = api.attn_cache_weights(q.cuda(), torch.zeros((2, 3), device="cuda"), p.dev, dev(cu), dev(lens), 1, 100)
        assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT
        assert (w[1, :, 32:64] == 0).all() and (w[1, :, :32] > 0).all()
        p.dev.page_table[1, 1] = was
    # eviction: a budget above max_keep, a negative one
    dst = Pair([50, 50, 50], 1, 64, 32, seed=2)
    w = torch.rand((3, 1, 100), device="cuda")
    for budgets in ([50, 51, 50], [50, -1, 50]):
        before = dst.dev.k_pages.clone()
        nl = torch.full((3,), -7, dtype=torch.int32, device="cuda")
        api.attn_cache_evict(w, p.dev, dst.dev, dev(lens), dev(budgets), 4, 100, 50, new_lens=nl)
        assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT
        assert nl.cpu().tolist() == [50, -7, 50]
        pages = torch.from_numpy(dst.table[1].astype(np.int64))
        assert torch.equal(dst.dev.k_pages[pages], before[pages])


def test_the_binding_refuses_what_the_kernels_would_misread():
    p = filled([40], 2, 64, 32, seed=1)
    q, cu, lens = randn(1, 4, 64).cuda(), dev([0, 1]), dev([40])
    lse = torch.zeros((4, 1), device="cuda")
    bad = [
        lambda: api.attn_cache_fwd(q.float(), p.dev, cu, lens, 1, 40),
        lambda: api.attn_cache_fwd(q.cpu(), p.dev, cu, lens, 1, 40),
        lambda: api.attn_cache_fwd(q[..., :32].contiguous(), p.dev, cu, lens, 1, 40),
        lambda: api.attn_cache_fwd(q[:, :3].contiguous(), p.dev, cu, lens, 1, 40),
        lambda: api.attn_cache_fwd(q, p.dev, cu.long(), lens, 1, 40),
        lambda: api.attn_cache_fwd(q, p.dev, dev([0, 1, 1]), lens, 1, 40),
        lambda: api.attn_cache_fwd(q, p.dev, cu, lens, 1, 65),                     # above the page table
        lambda: api.attn_cache_fwd(q, p.dev, cu, lens, 1, 40, kind="strip_thinking"),
        lambda: api.attn_cache_fwd(q, p.dev, cu, lens, 1, 40, scale=-1.0),
        lambda: api.attn_cache_fwd(q, None, cu, lens, 1, 40),
        lambda: api.attn_cache_weights(q, lse, p.dev, cu, lens, 1, 40, out=torch.zeros((1, 2, 39), device="cuda")),
        lambda: api.attn_cache_weights(q, lse.t().contiguous(), p.dev, cu, lens, 1, 40),
        lambda: api.attn_cache_append(q, q, p.dev, cu, lens, 1),                   # 4 heads, not 2
        lambda: api.attn_cache_append(q[:, :2].half(), q[:, :2].half(), p.dev, cu, lens, 1),
        lambda: api.attn_cache_evict(torch.zeros((1, 2, 39), device="cuda"), p.dev, p.dev, lens, lens, 0, 40, 40),
        lambda: api.attn_cache_evict(torch.zeros((1, 2, 40), device="cuda"), p.dev, p.dev, lens, lens, 0, 40, 40,
                                     new_lens=lens),
        lambda: api.attn_cache_evict(torch.zeros((1, 2, 40), device="cuda"), p.dev, p.dev, lens, lens, -1, 40, 40),
        lambda: api.KVCache(p.dev.k_pages, p.dev.v_pages, p.dev.k_scale.double(), p.dev.v_scale, p.dev.page_table),
        lambda: api.KVCache(p.dev.k_pages, p.dev.v_pages[:-1], p.dev.k_scale, p.dev.v_scale, p.dev.page_table),
    ]
    for call in bad:
        with pytest.raises(api.AttnError):
            call()
    big = filled([9000], 1, 64, 32, seed=2)
    need = api.attn_cache_fwd_workspace_size(big.dev, 1, 4, 1, 9000)
    assert need > 0
    with pytest.raises(api.AttnError) as e:
        api.attn_cache_fwd(q, big.dev, cu, dev([9000]), 1, 9000,
                           workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == api.ATTN_ERR_WORKSPACE_TOO_SMALL


def test_nothing_to_do():
    """No tokens, no sequences' tokens, empty pools of work: calls return and write nothing."""
    p = filled([0, 0], 1, 64, 32, seed=1)
    e = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    cu, lens = dev([0, 0, 0]), dev([0, 0])
    api.attn_cache_append(e, e, p.dev, cu, lens, 0)
    o, lse = api.attn_cache_fwd(e, p.dev, cu, lens, 0, 0)
    assert o.shape == (0, 1, 64) and lse.shape == (1, 0)
    w = api.attn_cache_weights(e, lse, p.dev, cu, lens, 0, 32, prev=torch.ones((2, 1, 32), device="cuda"))
    assert (w == 0).all()  # nothing is held, so nothing is written
    kept, nw, nl = api.attn_cache_evict(w, p.dev, p.dev, lens, dev([4, 0]), 0, 0, 0)
    assert kept.shape == (2, 1, 0) and nl.cpu().tolist() == [0, 0]
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
    plan = api.attn_rope_plan(64)
    yq, yk = api.attn_rope(e, e, plan, cu_seqlens=cu)
    assert yq.shape == (0, 1, 64) and yk.shape == (0, 1, 64)
