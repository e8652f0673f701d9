"""The operators on drafted trees at their edges: waits that run out, values and
queries of a very wide range, pools above 4 GiB, captured steps and other streams,
aliased results, malformed batches.  Bounds are those of the tests of the cache
where no other is derived beside them."""
import math

import numpy as np
import pytest
import torch

from block_sparse_masked_mask_gb300 import _native, api
from block_sparse_masked_mask_gb300 import build as B
from oracle import tree as R
from test_cache_edges_gpu import Far
from test_cache_gpu import Pair, attend_bounds, cu_of, dev, filled, randn
from test_cache_range_gpu import ORDERS, far_bounds
from test_tree_gpu import check_cached_near, check_tree, device_bits, partners, random_parents, trees

pytestmark = pytest.mark.gpu


def words_of(masks, words=None):
    return R.to_bits(masks, words or max(1, -(-max(len(m) for m in masks) // 32)))


# ------------------------------------------------------------------ waits

@pytest.mark.parametrize("heads,group,n", [(8, 1, 9), (8, 2, 16), (2, 4, 16), (4, 4, 40)])
def test_launches_whose_waits_run_out_return(heads, group, n):
    """Waits of 100 ns: every launch returns, the status says whether a wait ran out in it, and the
    ordinary library is right afterwards."""
    lens = [n + 900 + 200 * i for i in range(12)]
    p = filled(lens, heads, 64, 32, seed=1)
    cu, q, masks = cu_of([n] * 12), randn(12 * n, heads * group, 64, seed=2), trees([n] * 12)
    args = (q.cuda(), p.dev, device_bits(words_of(masks)), dev(cu), dev(lens), n, max(lens))
    want = [x.clone() for x in api.attn_cache_tree_fwd(*args)]
    torch.cuda.synchronize()
    ran_out = 0
    with _native.use_library(B.build_variant("waitshort", {"ATTN_WAIT_TIMEOUT_NS": "100ull"})):
        for _ in range(20):
            api.attn_cache_tree_fwd(*args)
            status = api.attn_cache_get_status(p.dev)
            assert status in (api.ATTN_OK, api.ATTN_ERR_DEVICE_TIMEOUT)
            ran_out += status != api.ATTN_OK
    assert ran_out > 0
    assert all(torch.equal(a, b) for a, b in zip(want, api.attn_cache_tree_fwd(*args)))
    check_tree(p, q, cu, lens, masks)


# ------------------------------------------------------------------ the range of numbers

@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("dim,lens,n,group", [
    (64, [200, 70, 900], 5, 1), (32, [3000, 500], 4, 6), (128, [9000, 400], 12, 4), (32, [9000, 40], 33, 1),
    (128, [1100], 70, 4), (32, [9000, 2500], 90, 1)])
def test_values_of_very_different_size(order, dim, lens, n, group):
    """A page of zeros next to one of 2^60 keeps its share of every sum.  Queries are two e4m3
    numbers: an element below 2^-9 of the row's largest is off by 2^-17 of that at most, a score by
    that times scale sum |k|."""
    powers, run = ORDERS[order]
    p = Pair(lens, 1, dim, 32, seed=1)
    cu_all, T = cu_of(lens), sum(lens)
    k, v = 0.5 * randn(T, 1, dim, seed=2), randn(T, 1, dim, seed=3)
    for b, total in enumerate(lens):
        for j in range(0, total, 32):
            x = powers[(j // 32 // run + b) % len(powers)]
            v[cu_all[b] + j:cu_all[b] + min(total, j + 32)] *= 0.0 if x is None else 2.0 ** x
    p.append(k, v, cu_all, lens)
    new = [min(n, x) for x in lens]
    cu, masks = cu_of(new), trees(new)
    q = randn(int(cu[-1]), group, dim, seed=4)
    O, L, terms, spread = R.attend(p.ref, q.double().numpy(), cu, lens, masks)
    tol, slack = far_bounds(p, O, spread, terms, cu, lens, dim)
    o, lse = api.attn_cache_tree_fwd(q.cuda(), p.dev, device_bits(words_of(masks)), dev(cu), dev(lens), max(new), max(lens))
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
    got = lse.double().cpu().numpy()
    for b, total in enumerate(lens):
        s = slice(cu[b], cu[b + 1])
        most = float(q[s].float().abs().max()) * np.abs(p.ref.numbers(0, b, total)).sum(-1).max()
        off = 2.0 ** -17 * most / math.sqrt(dim)
        tol[s] += 2 * np.expm1(2 * off) * spread[s]
        d = np.abs(got[:, s] - L[:, s])
        assert (d <= slack[b] + off + 2.0 ** -22 * np.abs(L[:, s])).all(), f"LSE of {b}: {d.max()} vs {slack[b]}"
    err = np.abs(o.double().cpu().numpy() - O)
    assert (err <= tol).all(), f"O: worst ratio {(err / tol).max()}"


@pytest.mark.parametrize("n", [1, 20, 140])
def test_hidden_nodes_under_factors_that_underflow(n):
    """Keys of zeros (page scale 2^-80) and queries near 2^-70: the factor of a
    block's scores is 0 in fp32, and what is hidden stays hidden."""
    lens = [500, 150]
    p = Pair(lens, 1, 64, 32, seed=1)
    k, v = randn(650, 1, 64, seed=1), randn(650, 1, 64, seed=2)
    k[::2] = 0
    k[64:96] = 0
    k[480:] = 0
    p.append(k, v, cu_of(lens), lens)
    for size, scale in ((2.0 ** -70, 0.0), (1.0, 2.0 ** -100)):
        check_tree(p, randn(2 * n, 2, 64, seed=3, scale=size), cu_of([n, n]), lens, trees([n, n]), scale=scale)


@pytest.mark.parametrize("dim", [32, 128])
@pytest.mark.parametrize("n", [1, 12, 40, 300])
@pytest.mark.parametrize("length", [900, 9000])
def test_many_small_weights_beside_large_ones(length, n, dim):
    """Every 16th token takes almost all the weight and has no value; the others,
    2^-26 of it each, are all that O consists of.  A weight is fp16: 2^-19 of the
    reference, which the largest passes by 2^7, so off by 2^-25 / 2^-19 = 2^-6 of
    itself at most."""
    p = Pair([length], 1, dim, 64, seed=1)
    k, v = torch.zeros(length, 1, dim), torch.ones(length, 1, dim)
    k[::16, :, 0] = 1.0
    v[::16] = 0.0
    p.append(k.bfloat16(), v.bfloat16(), cu_of([length]), [length])
    q = torch.zeros(n, 1, dim, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    scale, masks, cu = 26 * math.log(2), trees([n]), cu_of([n])
    O, L, _, _ = R.attend(p.ref, q.double().numpy(), cu, [length], masks, scale=scale)
    assert np.abs(O).max() < 2.0 ** -20
    o, lse = api.attn_cache_tree_fwd(q.cuda(), p.dev, device_bits(words_of(masks)), dev(cu), dev([length]), n, length, scale=scale)
    # a score of 26 (base 2), a sum over `length` tokens in fp32
    slack = 2 * (dim + 4) * 2.0 ** -24 * 19 + 2.0 ** -22 + 2.0 ** -23 * (2 * 26 + 16) + length * 2.0 ** -24
    assert (np.abs(lse.double().cpu().numpy() - L) <= slack + 2.0 ** -22 * np.abs(L)).all()
    err = np.abs(o.double().cpu().numpy() - O)
    assert (err <= (2.0 ** -6 + 2.0 ** -8 + 2.0 ** -9) * np.abs(O)).all(), (err / np.abs(O)).max()


@pytest.mark.parametrize("rows", [1, 3, 16, 48, 200])
def test_small_elements_beside_a_large_one(rows):
    """The largest element of a query, m, meets keys of 0, so that scores consist of
    elements 2^-12 to 2^-24 of it: as two e4m3 numbers, whatever the number of rows, each is off by
    2^-17 m at most, a score by scale times that times sum |k|."""
    L, scale = 400, 8.0
    p = Pair([L], 1, 64, 64, seed=2)
    k, v = randn(L, 1, 64, seed=1), randn(L, 1, 64, seed=2)
    k[..., 0] = 0
    p.append(k, v, cu_of([L]), [L])
    g = torch.Generator().manual_seed(3)
    q = torch.randn((rows, 1, 64), generator=g) * 2.0 ** torch.randint(-24, -11, (rows, 1, 64), generator=g)
    q[..., 0] = 1.5
    q = q.to(torch.bfloat16)
    masks, cu = trees([rows]), cu_of([rows])
    o, lse = api.attn_cache_tree_fwd(q.cuda(), p.dev, device_bits(words_of(masks)), dev(cu), dev([L]), rows, L, scale=scale)
    O, Z, terms, spread = R.attend(p.ref, q.double().numpy(), cu, [L], masks, scale=scale)
    off = 2.0 ** -17 * 1.5 * np.abs(p.ref.numbers(0, 0, L)).sum(-1).max() * scale
    A = terms[0].max()
    rel = 2 * ((64 + 4) * 2.0 ** -24 * A) + 2.0 ** -22 + 2.0 ** -23 * (2 * A + 16) + L * 2.0 ** -24
    assert (np.abs(lse.double().cpu().numpy() - Z) <= rel + off + 2.0 ** -22 * np.abs(Z)).all()
    tol = (2.0 ** -11 + 3 * rel + 2 * np.expm1(2 * off)) * spread + 2.0 ** -32 * p.ref.code_sums(1, 0, L)[None]
    assert (np.abs(o.double().cpu().numpy() - O) <= tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(O)).all()


def test_rising_and_falling_scores():
    """References that move at every tile, never, and only in one warpgroup's tiles."""
    L, n = 2000, 9
    ramp = torch.linspace(0, 1, L)
    flip = torch.where(torch.arange(L) // 128 % 2 == 0, ramp, -ramp)
    for size in (ramp, -ramp, flip, ramp * (torch.arange(L) % 97 == 0)):
        p = Pair([L], 1, 64, 32, seed=4)
        k, v = 0.05 * randn(L, 1, 64, seed=1).float(), randn(L, 1, 64, seed=2)
        k[:, 0, 0] += 60 * size
        p.append(k.bfloat16(), v, cu_of([L]), [L])
        q = randn(n, 4, 64, seed=5)
        q[..., 0] = torch.linspace(-8, 8, 4 * n).view(n, 4)
        check_tree(p, q, cu_of([n]), [L], trees([n]))


# ------------------------------------------------------------------ far pages

def test_pages_past_32_bits():
    """All four on the last pages of a pool above 4 GiB per side."""
    heads, dim, ps = 8, 128, 128
    pool = (1 << 32) // (heads * dim * ps) + 64
    lens = np.array([700, 300], np.int32)
    p = Far(list(lens), heads, dim, ps, pool, seed=1)
    assert int(p.dev.page_table[0, 0]) * heads * dim * ps > 2 ** 31
    n = np.array([30, 16], np.int32)
    cu_text, text = cu_of(lens - n), lens - n
    p.append(randn(int(cu_text[-1]), heads, dim, seed=1), randn(int(cu_text[-1]), heads, dim, seed=2), cu_text, text)
    rng = np.random.default_rng(2)
    parents = [random_parents(int(x), rng) for x in n]
    masks, cu = [R.ancestors(x) for x in parents], cu_of(n)
    bits, positions = api.attn_cache_tree_build(dev(sum(parents, [])), p.dev, dev(cu), dev(lens), 30)
    q, k, v = (randn(46, h, dim, seed=3 + h).cuda() for h in (16, heads, heads))
    plan = api.attn_rope_plan(dim)
    turned = api.attn_cache_append_rope(q, k, v, plan, p.dev, dev(cu), dev(lens), 30, positions=positions)
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
    # the keys near attn_rope's (rounded to bf16 there); then the oracle takes the pages as they are
    want, _ = api.attn_rope(k, None, plan, positions=positions)
    here = slice(p.first, p.first + p.pages)
    p.ref.codes = [x[here].cpu().numpy().copy() for x in (p.dev.k_pages, p.dev.v_pages)]
    p.ref.scale = [x[here].cpu().double().numpy() for x in (p.dev.k_scale, p.dev.v_scale)]
    for b in range(2):
        got = p.ref.numbers(0, b, lens[b])[:, lens[b] - n[b]:]
        exact = want[cu[b]:cu[b + 1]].double().cpu().numpy().transpose(1, 0, 2)
        assert (np.abs(got - exact) <= 2.0 ** -4 * 1.02 * np.abs(exact) + 2.0 ** -9 * np.abs(exact).max()).all()
    check_tree(p, turned.cpu(), cu, lens, masks)
    check_tree(p, randn(46, 64, dim, seed=9), cu, lens, masks)  # (by the kernel of many rows)
    paths = [[0, 4, 29], [3, 9, 10, 15]]
    path = np.array([paths[0] + [0], paths[1]], np.int32)
    new = api.attn_cache_tree_keep(dev(path), dev([3, 4]), p.dev, dev(cu), dev(lens), 30)
    assert new.tolist() == R.keep(p.ref, paths, cu, lens).tolist()
    p.check_codes()


# ------------------------------------------------------------------ repeats, streams, graphs

def step_inputs(lens, n, heads, group, dim, seed):
    rng = np.random.default_rng(seed)
    cu, T = cu_of(n), int(np.sum(n))
    parents = [random_parents(int(x), rng) for x in n]
    q, k, v = (randn(T, h, dim, seed=seed + i) for i, h in enumerate((heads * group, heads, heads)))
    paths = [np.flatnonzero(R.ancestors(x)[-1]) for x in parents]
    path = np.zeros((len(n), max(n)), np.int32)
    for b, x in enumerate(paths):
        path[b, :len(x)] = x
    return dict(parents=dev(sum(parents, [])), cu=dev(cu), lens=dev(lens), q=q.cuda(), k=k.cuda(), v=v.cuda(), path=dev(path),
                counts=dev([len(x) for x in paths]))


def run_step(x, p, plan, max_new, max_seqlen, **kw):
    bits, positions = api.attn_cache_tree_build(x["parents"], p.dev, x["cu"], x["lens"], max_new, **kw)
    q = api.attn_cache_append_rope(x["q"], x["k"], x["v"], plan, p.dev, x["cu"], x["lens"], max_new, positions=positions, **kw)
    o, lse = api.attn_cache_tree_fwd(q, p.dev, bits, x["cu"], x["lens"], max_new, max_seqlen, **kw)
    new = api.attn_cache_tree_keep(x["path"], x["counts"], p.dev, x["cu"], x["lens"], max_new, **kw)
    return [bits, positions, q, o, lse, new]


STATE = ("k_pages", "v_pages", "k_scale", "v_scale")


@pytest.mark.parametrize("group", [1, 4, 9])
def test_a_step_captured_repeated_and_on_other_streams(group):
    """A whole step is the same bit by bit run again, on a stream of its own, two at once,
    and replayed from a graph on other trees, lengths and pages."""
    heads, dim, ps = 2, 64, 32
    lens, n = [3000, 150, 40], [16, 9, 16]
    plan = api.attn_rope_plan(dim)
    p = filled(lens, heads, dim, ps, seed=71)
    held = [getattr(p.dev, name).clone() for name in STATE]

    def again():
        for name, x in zip(STATE, held):
            getattr(p.dev, name).copy_(x)

    x = step_inputs(lens, n, heads, group, dim, 5)
    first = [y.clone() for y in run_step(x, p, plan, 16, 3000)]
    after = [getattr(p.dev, name).clone() for name in STATE]
    for stream in (None, torch.cuda.Stream()):
        again()
        torch.cuda.synchronize()
        got = run_step(x, p, plan, 16, 3000, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, got))
        assert all(torch.equal(a, getattr(p.dev, name)) for a, name in zip(after, STATE))
    # attentions at once on two streams
    again()
    run_step(x, p, plan, 16, 3000)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    args = (first[2], p.dev, first[0], x["cu"], x["lens"], 16, 3000)
    want = [y.clone() for y in api.attn_cache_tree_fwd(*args)]
    torch.cuda.synchronize()
    outs = [api.attn_cache_tree_fwd(*args, stream=s) for s in sides for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for out in outs for a, b in zip(want, out))
    # captured, and replayed on other inputs
    again()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run_step(x, p, plan, 16, 3000)
    other_lens, other_n = [2000, 20, 100], [16, 16, 9]
    y = step_inputs(other_lens, other_n, heads, group, dim, 50)
    table = p.dev.page_table.clone()
    table[2], table[1] = p.dev.page_table[1], torch.roll(p.dev.page_table[0], -70, 0)  # (of no other's)
    for name in x:
        x[name].copy_(y[name])
    p.dev.page_table.copy_(table)
    eager = run_step(y, p, plan, 16, 3000)
    eager = [z.clone() for z in eager]
    after = [getattr(p.dev, name).clone() for name in STATE]
    again()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, outs))
    assert all(torch.equal(a, getattr(p.dev, name)) for a, name in zip(after, STATE))
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK


@pytest.mark.parametrize("n", [4, 40])
def test_captured_calls_draw_workspaces_of_their_own(n):
    """Two graphs of calls without a workspace argument, replayed at once on two streams."""
    cases = []
    for seed, lens in ((1, [9000, 1500]), (2, [8600, 8900])):
        p = filled(lens, 2, 128, 64, seed=seed)
        q, masks = randn(2 * n, 8, 128, seed=seed).cuda(), trees([n, n], seed=seed)
        args = (q, p.dev, device_bits(words_of(masks)), dev(cu_of([n, n])), dev(lens), n, max(lens))
        assert api.attn_cache_tree_fwd_workspace_size(p.dev, 2 * n, 8, n, max(lens)) > 0
        want = [x.clone() for x in api.attn_cache_tree_fwd(*args)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = api.attn_cache_tree_fwd(*args)
        cases.append((graph, out, want, args))
    sides = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for _, out, _, _ in cases:
            for x in out:
                x.fill_(9)
        torch.cuda.synchronize()
        for (graph, _, _, _), side in zip(cases, sides):
            with torch.cuda.stream(side):
                graph.replay()
        for _, _, want, args in cases:
            assert all(torch.equal(a, b) for a, b in zip(want, api.attn_cache_tree_fwd(*args)))
        torch.cuda.synchronize()
        for _, out, want, _ in cases:
            assert all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.parametrize("n,group", [(1, 1), (9, 4), (40, 4), (100, 4)])
def test_results_over_the_queries(n, group):
    for length in (400, 5000, 20000):
        p = filled([length, 300], 2, 64, 64, seed=n)
        q, masks = randn(2 * n, 2 * group, 64, seed=3).cuda(), trees([n, n])
        args = (p.dev, device_bits(words_of(masks)), dev(cu_of([n, n])), dev([length, 300]), n, length)
        o, lse = api.attn_cache_tree_fwd(q, *args)
        got, again = api.attn_cache_tree_fwd(q, *args, out=q)
        assert got is q and torch.equal(q, o) and torch.equal(again, lse)


# ------------------------------------------------------------------ malformed batches

def test_bad_sequences_are_reported_and_left_out():
    """Malformed cu_seqlens or lengths, and lengths below the numbers of new tokens: the status
    says so, nothing of the sequence is written, the others are right."""
    lens, n = [100, 90, 80], [3, 5, 4]
    masks, cu = trees(n), cu_of(n)
    parents = dev(sum(([-1] + list(range(x - 1)) for x in n), []))
    plan = api.attn_rope_plan(64)
    q, k, v = (randn(12, h, 64, seed=h).cuda() for h in (4, 2, 1))
    k, v = k[:, :1].contiguous(), v
    for bad_cu, bad_lens in ((cu, [100, -1, 80]), (cu, [100, 129, 80]), (cu, [100, 4, 80]), ([0, 3, 2, 12], lens),
                             ([0, 3, 13, 12], lens)):
        for group in (2, 20):  # both kernels of attention
            p = filled(lens, 1, 64, 32, seed=1)
            was = [getattr(p.dev, name).clone() for name in STATE]
            d_cu, d_lens = dev(bad_cu), dev(bad_lens)
            wide = randn(12, group, 64, seed=4).cuda()
            good = [x.clone() for x in api.attn_cache_tree_fwd(wide, p.dev, device_bits(words_of(masks)), dev(cu), dev(lens), 5, 128)]
            out = torch.full((12, group, 64), 5.0, dtype=torch.bfloat16, device="cuda")
            api.attn_cache_tree_fwd(wide, p.dev, device_bits(words_of(masks)), d_cu, d_lens, 5, 128, out=out)
            assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT
            assert (out[3:8] == 5).all()
            if bad_cu is cu:
                assert torch.equal(out[8:], good[0][8:])
        bits = torch.full((12, 1), 99, dtype=torch.int32, device="cuda")
        positions = torch.full((12,), 99, dtype=torch.int32, device="cuda")
        api.attn_cache_tree_build(parents, p.dev, d_cu, d_lens, 5, bits=bits, positions=positions)
        assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT
        assert (bits[3:8] == 99).all() and (positions[3:8] == 99).all()
        rotated = torch.full((12, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        api.attn_cache_append_rope(q, k, v, plan, p.dev, d_cu, d_lens, 5, q_out=rotated)
        assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT
        assert (rotated[3:8] == 5).all()
        new = torch.full((3,), -7, dtype=torch.int32, device="cuda")
        api.attn_cache_tree_keep(dev([[0, 1], [1, 2], [1, 3]]), dev([2, 2, 2]), p.dev, d_cu, d_lens, 5, new_lens=new)
        assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT
        assert new[1] == -7
        mine = torch.from_numpy(p.table[1][p.table[1] < 1 << 28].astype(np.int64))
        for name, x in zip(STATE, was):
            assert torch.equal(getattr(p.dev, name)[mine], x[mine]), name
        assert api.attn_cache_get_status(p.dev) == api.ATTN_OK


@pytest.mark.parametrize("bad", [-1, 10 ** 6, 2 ** 31 - 1])
def test_bad_pages_are_reported_and_left_out(bad):
    """Tokens of a page that there is not do not count, are not written and not moved."""
    lens, n = [200, 90], [40, 5]
    masks, cu = trees(n), cu_of(n)
    for group in (1, 4):
        p = filled(lens, 1, 64, 32, seed=1)
        q = randn(45, group, 64, seed=1)
        good = check_tree(p, q, cu, lens, masks)[0].clone()
        p.dev.page_table[0, 1] = bad
        out, lse = api.attn_cache_tree_fwd(q.cuda(), p.dev, device_bits(words_of(masks, 2)), dev(cu), dev(lens), 40, 200)
        assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT
        assert torch.equal(out[40:], good[40:]) and torch.isfinite(out).all()
        # (the text without the tokens of that page: the same as a text that is shorter by it)
        short = Pair([168, 90], 1, 64, 32, seed=1)
        short.ref.codes, short.ref.scale = p.ref.codes, p.ref.scale
        short.ref.table = np.concatenate([p.table[:, :1], p.table[:, 2:]], 1)
        O, _, terms, spread = R.attend(short.ref, q[:40].double().numpy(), [0, 40], [168], masks[:1])
        tol, _ = attend_bounds(short.ref, O, spread, terms, [0, 40], [168], 64)
        assert (np.abs(out[:40].double().cpu().numpy() - O) <= tol).all()
    # appended and kept: pages that there are take what is theirs
    p = filled(lens, 1, 64, 32, seed=1)
    was = [getattr(p.dev, name).clone() for name in STATE]
    q, k, v = (randn(45, 1, 64, seed=h).cuda() for h in (4, 2, 1))
    p.dev.page_table[0, 5:7] = bad  # tokens 160 .. 199, all of the tree
    api.attn_cache_append_rope(q, k, v, api.attn_rope_plan(64), p.dev, dev(cu), dev(lens), 40)
    assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT
    mine = torch.from_numpy(p.table[0, :7].astype(np.int64))
    assert all(torch.equal(getattr(p.dev, name)[mine], x[mine]) for name, x in zip(STATE, was))
    for pages in ([5], [6], [5, 6]):
        p.dev.page_table[0, :7] = torch.from_numpy(p.table[0, :7])
        p.dev.page_table[0, pages] = bad
        api.attn_cache_tree_keep(dev([[2, 5, 36]]).expand(2, 3).contiguous(), dev([3, 0]), p.dev, dev(cu), dev(lens), 40)
        assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT


def test_workspaces_that_do_not_fit():
    p = filled([9000], 1, 64, 32, seed=2)
    for n in (4, 100):
        q, bits = randn(n, 4, 64).cuda(), device_bits(words_of(trees([n])))
        args = (q, p.dev, bits, dev([0, n]), dev([9000]), n, 9000)
        need = api.attn_cache_tree_fwd_workspace_size(p.dev, n, 4, n, 9000)
        assert need > 0
        with pytest.raises(api.AttnError) as e:
            api.attn_cache_tree_fwd(*args, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
        assert e.value.status == api.ATTN_ERR_WORKSPACE_TOO_SMALL
        room = torch.full((need + 64,), 77, dtype=torch.uint8, device="cuda")
        want = api.attn_cache_tree_fwd(*args)
        got = api.attn_cache_tree_fwd(*args, workspace=room[:need])
        assert all(torch.equal(a, b) for a, b in zip(want, got)) and (room[need:] == 77).all()


def test_nothing_to_do():
    """No tokens, or no sequence with any: calls return and write nothing."""
    p = filled([40, 0], 1, 64, 32, seed=1)
    was = [getattr(p.dev, name).clone() for name in STATE]
    cu, lens = dev([0, 0, 0]), dev([40, 0])
    for T in (0, 3):
        parents = torch.zeros(T, dtype=torch.int32, device="cuda")
        bits = torch.full((T, 1), 9, dtype=torch.int32, device="cuda")
        q = torch.ones((T, 2, 64), dtype=torch.bfloat16, device="cuda")
        k = torch.ones((T, 1, 64), dtype=torch.bfloat16, device="cuda")
        for most in (0, 1):
            api.attn_cache_tree_build(parents, p.dev, cu, lens, most, bits=bits)
            out = torch.full_like(q, 5)
            api.attn_cache_append_rope(q, k, k, api.attn_rope_plan(64), p.dev, cu, lens, most, q_out=out)
            assert (out == 5).all()
            o, lse = api.attn_cache_tree_fwd(q, p.dev, bits, cu, lens, most, 40, out=out)
            assert (out == 5).all() and (bits == 9).all()
            new = api.attn_cache_tree_keep(torch.zeros((2, 1), dtype=torch.int32, device="cuda"), dev([0, 0]), p.dev, cu, lens, most)
            assert new.tolist() == [40, 0]
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
    assert all(torch.equal(getattr(p.dev, name), x) for name, x in zip(STATE, was))


def test_thousands_of_short_sequences():
    n = [(i * 5) % 4 for i in range(3000)]
    lens = [x + i % 3 for i, x in enumerate(n)]
    p = filled(lens, 1, 32, 16, seed=5)
    check_tree(p, randn(sum(n), 2, 32, seed=3), cu_of(n), lens, trees(n))
    paths = [list(range(0, x, 2)) for x in n]
    path = np.zeros((len(n), 2), np.int32)
    for b, x in enumerate(paths):
        path[b, :len(x)] = x
    new = api.attn_cache_tree_keep(dev(path), dev([len(x) for x in paths]), p.dev, dev(cu_of(n)), dev(lens), 3)
    assert new.tolist() == R.keep(p.ref, paths, cu_of(n), lens).tolist()
    p.check_codes()


@pytest.mark.parametrize("batch,heads,most", [(1, 1, 8193), (3, 2, 5000), (2, 20, 4096), (5, 20, 2000), (40, 8, 700)])
@pytest.mark.parametrize("n,group", [(1, 8), (13, 4), (4, 16)])
def test_sequences_cut_in_every_way(batch, heads, most, n, group):
    """Pieces that begin and end anywhere in a sequence, several segments to a CTA."""
    lens = [max(n, most - 311 * b % most) for b in range(batch)]
    p = filled(lens, heads, 32, 32, seed=batch)
    check_tree(p, randn(n * batch, heads * group, 32, seed=1), cu_of([n] * batch), lens, trees([n] * batch, "deep"))


# ------------------------------------------------------------------ append at its edges

def test_append_rope_numbers_at_the_edges():
    """Infinities and NaN are stored as attn_cache_append stores them, zeros have the least scale, and
    elements that are not turned go over as they are."""
    n, dim, rot = 40, 64, 16
    k = randn(n, 2, dim, seed=1, dtype=torch.float32)
    k[3, 0, 20], k[4, 0, 21], k[5, 0, 22] = float("inf"), float("-inf"), float("nan")
    k[:, 1] = 0
    v = k.flip(0)
    one, two = (Pair([n], 2, dim, 32, seed=1) for _ in range(2))
    api.attn_cache_append_rope(None, k.cuda(), v.cuda(), api.attn_rope_plan(rot), one.dev, dev([0, n]), dev([n]), n)
    turned = api.attn_rope(k.cuda(), None, api.attn_rope_plan(rot), positions=dev(np.arange(n)))[0]
    api.attn_cache_append(turned, v.cuda(), two.dev, dev([0, n]), dev([n]), n)
    assert torch.equal(one.dev.v_pages, two.dev.v_pages) and torch.equal(one.dev.v_scale, two.dev.v_scale)
    assert torch.equal(one.dev.k_scale, two.dev.k_scale)
    assert torch.equal(one.dev.k_pages[..., rot:], two.dev.k_pages[..., rot:])
    pages = dev(one.table[0]).long()
    assert (one.dev.k_pages[pages, 1, :n - 32] & 127 == 0).all()


@pytest.mark.parametrize("held", [0, 1, 31, 32, 33, 127])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 129])
def test_append_rope_by_parts(held, n):
    """What is there is kept, re-scaled where a page's scale rises, and new tokens begin anywhere."""
    heads, dim = 5, 32
    p = Pair([held + n], heads, dim, 32, seed=held)
    if held:
        p.append(0.01 * randn(held, heads, dim, seed=1), randn(held, heads, dim, seed=2), cu_of([held]), [held])
    k, v = randn(n, heads, dim, seed=3), randn(n, heads, dim, seed=4)
    api.attn_cache_append_rope(None, k.cuda(), v.cuda(), api.attn_rope_plan(dim), p.dev, dev([0, n]), dev([held + n]), n)
    exact = k.double().numpy().copy()
    theta = np.array([api.attn_rope_plan(dim).struct.turn[i] for i in range(dim // 2)], np.float64) / 2.0 ** 64
    z = (exact[..., :dim // 2] + 1j * exact[..., dim // 2:]) * np.exp(2j * np.pi * np.outer(np.arange(held, held + n), theta))[:, None]
    off = 2.0 ** -20 * partners(exact, dim, False)
    exact[..., :dim // 2], exact[..., dim // 2:] = z.real, z.imag
    check_cached_near(p, exact, off, v.double().numpy(), cu_of([n]), [held + n])


def test_append_rope_of_many_heads_and_long_pages():
    """More heads and pages than one CTA's teams, pages whose keys do not fit its registers at once."""
    for heads, dim, ps, n in ((40, 128, 128, [300, 5]), (9, 32, 16, [700, 64]), (64, 64, 64, [128] * 6)):
        lens, T = [x + 7 * i for i, x in enumerate(n)], sum(n)
        one, two = (Pair(lens, heads, dim, ps, seed=2) for _ in range(2))
        plan = api.attn_rope_plan(dim)
        k, v = (randn(T, heads, dim, seed=i, dtype=torch.float32).cuda() for i in range(2))
        at = torch.cat([torch.arange(7 * i, 7 * i + x) for i, x in enumerate(n)]).int().cuda()
        api.attn_cache_append_rope(None, k, v, plan, one.dev, dev(cu_of(n)), dev(lens), max(n))
        api.attn_cache_append(api.attn_rope(k, None, plan, positions=at)[0], v, two.dev, dev(cu_of(n)), dev(lens), max(n))
        assert torch.equal(one.dev.v_pages, two.dev.v_pages) and torch.equal(one.dev.v_scale, two.dev.v_scale)
        # (turned in fp32 both times, with roundings that may differ in the last place: a code by one at most)
        far = (one.dev.k_pages.int() - two.dev.k_pages.int()).abs()
        assert (one.dev.k_scale == two.dev.k_scale).float().mean() >= 0.99
        assert (far <= 1).float().mean() >= 0.99 and api.attn_cache_get_status(one.dev) == api.ATTN_OK


@pytest.mark.parametrize("n", [4, 40])
def test_attention_behind_copies_and_kernels(n):
    """What was written just before the call, by a copy or a kernel, is what it reads, in a captured graph too."""
    p = filled([900, 2000], 2, 64, 32, seed=n)
    masks = trees([n, n])
    sources = [randn(2 * n, 8, 64, seed=i).cuda() for i in range(6)]
    args = (p.dev, device_bits(words_of(masks)), dev(cu_of([n, n])), dev([900, 2000]), n, 2000)
    want = [[x.clone() for x in api.attn_cache_tree_fwd(q, *args)] for q in sources]
    q = torch.empty_like(sources[0])

    def calls():
        got = []
        for i, x in enumerate(sources):
            if i % 2:
                torch.mul(x, 1, out=q)
            else:
                q.copy_(x)
            got.append(api.attn_cache_tree_fwd(q, *args))
        return got

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = calls()
    for _ in range(3):
        graph.replay()
        for got in (captured, calls()):
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for x, y in zip(want, got) for a, b in zip(x, y))


@pytest.mark.parametrize("sizes", [[20, 17, 32, 26], [33, 64, 40], [20, 64, 3, 33, 1, 17, 90]], ids=str)
@pytest.mark.parametrize("dim,heads,lengths", [(64, 8, 500), (32, 3, 1300), (128, 8, 130)])
def test_several_segments_of_a_cta(dim, heads, lengths, sizes):
    """More (sequence, head)s than three for each SM, of up to 128 rows, of more, and of both in turn."""
    batch = -(-152 * 7 // (2 * heads))
    n = [sizes[b % len(sizes)] for b in range(batch)]
    lens = [x + (b * 277) % lengths for b, x in enumerate(n)]
    p = filled(lens, heads, dim, 32, seed=batch)
    check_tree(p, randn(sum(n), heads * 4, dim, seed=2), cu_of(n), lens, trees(n))


@pytest.mark.parametrize("n", [1, 4, 40])
@pytest.mark.parametrize("scale", [1.0, 1e20, 1e28, 1e33])
def test_scores_far_below_zero(n, scale):
    """Equal scores of -64 scale, whatever that is: no row is lost, LSE is the score (off by fp32's roundings of it
    and, where the exponents of the values' scales, up to 2^4, are below those, by 2^4 and ln of the tokens), and at
    scale 1 O is the mean of the visible values.  (From scale 2^19 on a score's rounding is more than the
    exponents that go with it: pages' shares are then no better known than the scores.)"""
    length = 700 + n
    p = Pair([length], 1, 64, 32, seed=1)
    k, v = torch.ones(length, 1, 64).bfloat16(), randn(length, 1, 64, seed=2)
    p.append(k, v, cu_of([length]), [length])
    masks = trees([n])
    q = -torch.ones(n, 4, 64, dtype=torch.bfloat16)
    o, lse = api.attn_cache_tree_fwd(q.cuda(), p.dev, device_bits(words_of(masks)), dev([0, n]), dev([length]), n, length, scale=scale)
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
    V = p.ref.numbers(1, 0, length)[0]
    for i in range(n):
        seen = np.concatenate([np.ones(length - n, bool), masks[0][i]])
        want, size = V[seen].mean(0), np.abs(V[seen]).mean(0)
        # (weights are equal and exact; sums of `length` terms in fp32, a rounding to bf16)
        err = np.abs(o[i].double().cpu().numpy() - want)
        assert torch.isfinite(o[i]).all() and (o[i] != 0).any()
        assert scale > 1 or (err <= 2.0 ** -8 * np.abs(want) + (length + 8) * 2.0 ** -23 * size).all()
        exact = -64.0 * scale + math.log(seen.sum())
        assert (np.abs(lse[:, i].double().cpu().numpy() - exact) <= 2.0 ** -20 * abs(exact)).all()
