"""Cache attention over the whole range that codes, scales and queries may have:
values of very different size in one sequence, factors that underflow, weights far
below the largest.  Bounds are those of test_cache_gpu with the terms that grow here
written out (exponents of the value scales)."""
import math

import numpy as np
import pytest
import torch

from block_sparse_masked_mask_gb300 import api
from test_cache_gpu import Pair, check_attend, cu_of, randn, run_attend

pytestmark = pytest.mark.gpu


def far_bounds(p, O, spread, terms, cu, lens, dim):
    """A score's base-2 argument carries the value exponent, E at most: two roundings
    of numbers up to A + E; far weights' sums square one ex2 (2^-21)."""
    tol, slack = np.zeros(O.shape), []
    E = 128.0
    for b, L in enumerate(lens):
        A = terms[b].max(initial=0)
        rel = 2 * ((dim + 4) * 2.0 ** -24 * A) + 2.0 ** -21 + 2.0 ** -23 * (2 * A + 2 * E) + L * 2.0 ** -24
        slack.append(rel)
        s = slice(cu[b], cu[b + 1])
        small = 2.0 ** -25 * p.ref.code_sums(1, b, L)
        tol[s] = (2.0 ** -11 + 3 * rel) * spread[s] + np.repeat(small, O.shape[1] // small.shape[0], 0)[None]
        tol[s] = tol[s] * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(O[s])
    return tol, slack


# powers of two of the pages' values in turn (None: zeros, whose page has the least
# scale, 2^-80), and how many pages of each follow one another
ORDERS = {"zeros_first": ([None, 60], 1), "zeros_last": ([60, None], 1), "runs": ([None, 0, 60], 8),
          "far": ([110, None, -60, 20], 2), "up": ([-60, None, 0, 60, 110], 3), "down": ([110, 60, 0, -60], 5)}


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("dim,lens,new,group", [
    (64, [200, 70, 900], 1, 1),       # one CTA or a cluster per sequence
    (32, [3000, 500], 2, 6),          # clusters, 12 rows
    (32, [9000, 40], 1, 2),           # the cut line and its join
    (64, [200, 70, 900], 20, 1),      # tensor cores, both M tiles with the same rows
    (128, [1100], 70, 4),             # two M tiles
    (32, [9000, 2500], 40, 1)])       # chunks and their join
def test_values_of_very_different_size(order, dim, lens, new, group):
    """The softmax does not depend on the values: a page of zeros next to one of
    2^60 keeps its share of every sum, and LSE is that of the keys alone."""
    powers, run = ORDERS[order]
    p = Pair(lens, 1, dim, 32, seed=1)
    cu_all, T = cu_of(lens), sum(lens)
    k, v = 0.5 * randn(T, 1, dim, seed=2), randn(T, 1, dim, seed=3)
    for b, n in enumerate(lens):
        for j in range(0, n, 32):
            x = powers[(j // 32 // run + b) % len(powers)]
            v[cu_all[b] + j:cu_all[b] + min(n, j + 32)] *= 0.0 if x is None else 2.0 ** x
    p.append(k, v, cu_all, lens)
    cu = cu_of([new] * len(lens))
    q = randn(int(cu[-1]), group, dim, seed=4)
    O, L, terms, spread = p.ref.attend(q.double().numpy(), cu, lens)
    tol, slack = far_bounds(p, O, spread, terms, cu, lens, dim)
    o, lse = run_attend(p, q, cu, lens)
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
    got = lse.double().cpu().numpy()
    for b in range(len(lens)):
        s = slice(cu[b], cu[b + 1])
        d = np.abs(got[:, s] - L[:, s])
        assert (d <= slack[b] + 2.0 ** -22 * np.abs(L[:, s])).all(), f"LSE of {b}: {d.max()} vs {slack[b]}"
    err = np.abs(o.double().cpu().numpy() - O)
    assert (err <= tol).all(), f"O: worst ratio {(err / tol).max()}"


@pytest.mark.parametrize("new", [1, 20, 140])
def test_hidden_tokens_under_factors_that_underflow(new):
    """Keys of zeros (page scale 2^-80) and queries near 2^-70: the factor of a
    block's scores is 0 in fp32, and what is hidden stays hidden."""
    lens = [500, 150]
    p = Pair(lens, 1, 64, 32, seed=1)
    k, v = randn(650, 1, 64, seed=1), randn(650, 1, 64, seed=2)
    k[::2] = 0
    k[64:96] = 0
    k[480:] = 0
    p.append(k, v, cu_of(lens), lens)
    cu = cu_of([new, new])
    for size, scale in ((2.0 ** -70, 0.0), (1.0, 2.0 ** -100)):
        q = randn(2 * new, 2, 64, seed=3, scale=size)
        check_attend(p, q, cu, lens, scale=scale)


@pytest.mark.parametrize("dim", [32, 128])
@pytest.mark.parametrize("new", [1, 12, 40, 300])
@pytest.mark.parametrize("length", [900, 9000])
def test_many_small_weights_beside_large_ones(length, new, dim):
    """Every 16th token takes almost all the weight and has no value; the others,
    2^-26 of it each, are all that O consists of.  A weight is fp16: 2^-19 of the
    reference, which the largest passes by 2^7, so off by 2^-25 / 2^-19 = 2^-6 of
    itself at most."""
    p = Pair([length], 1, dim, 64, seed=1)
    k, v = torch.zeros(length, 1, dim), torch.ones(length, 1, dim)
    k[::16, :, 0] = 1.0
    v[::16] = 0.0
    p.append(k.bfloat16(), v.bfloat16(), cu_of([length]), [length])
    q = torch.zeros(new, 1, dim, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    scale = 26 * math.log(2)
    O, L, _, _ = p.ref.attend(q.double().numpy(), cu_of([new]), [length], scale=scale)
    assert np.abs(O).max() < 2.0 ** -20
    o, lse = run_attend(p, q, cu_of([new]), [length], scale=scale)
    # a score of 26 (base 2), a sum over `length` tokens in fp32
    slack = 2 * (dim + 4) * 2.0 ** -24 * 19 + 2.0 ** -22 + 2.0 ** -23 * (2 * 26 + 16) + length * 2.0 ** -24
    assert (np.abs(lse.double().cpu().numpy() - L) <= slack + 2.0 ** -22 * np.abs(L)).all()
    err = np.abs(o.double().cpu().numpy() - O)
    assert (err <= (2.0 ** -6 + 2.0 ** -8 + 2.0 ** -9) * np.abs(O)).all(), (err / np.abs(O)).max()


@pytest.mark.parametrize("rows", [1, 3, 16, 48, 200])
def test_small_elements_beside_a_large_one(rows):
    """The largest element of a query meets keys of 0, so that scores consist of
    elements 2^-12 to 2^-24 of it.  As fp16 (up to 16 rows) an element below 2^-17 of
    the largest, m, is off by 2^-25 m at most, as two e4m3 numbers one below 2^-9 by
    2^-17 m; a score by scale times that times sum |k|."""
    L, scale = 400, 2.0 ** (10 if rows <= 16 else 3)
    p = Pair([L], 1, 64, 64, seed=2)
    k, v = randn(L, 1, 64, seed=1), randn(L, 1, 64, seed=2)
    k[..., 0] = 0
    p.append(k, v, cu_of([L]), [L])
    g = torch.Generator().manual_seed(3)
    q = torch.randn((rows, 1, 64), generator=g) * 2.0 ** torch.randint(-24, -11, (rows, 1, 64), generator=g)
    q[..., 0] = 1.5
    q = q.to(torch.bfloat16)
    o, lse = run_attend(p, q, cu_of([rows]), [L], scale=scale)
    O, Z, terms, spread = p.ref.attend(q.double().numpy(), cu_of([rows]), [L], scale=scale)
    K = np.abs(p.ref.numbers(0, 0, L)).sum(-1).max()
    off = 2.0 ** (-25 if rows <= 16 else -17) * 1.5 * K * scale
    A = terms[0].max()
    rel = 2 * ((64 + 4) * 2.0 ** -24 * A) + 2.0 ** -22 + 2.0 ** -23 * (2 * A + 16) + L * 2.0 ** -24
    assert (np.abs(lse.double().cpu().numpy() - Z) <= rel + off + 2.0 ** -22 * np.abs(Z)).all()
    tol = (2.0 ** -11 + 3 * rel + 2 * np.expm1(2 * off)) * spread + 2.0 ** -32 * p.ref.code_sums(1, 0, L)[None]
    assert (np.abs(o.double().cpu().numpy() - O) <= tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(O)).all()
