"""The rotated append of so many pages and heads that a team of threads takes several heads in
turn, one's elements on their way while another's are stored: every code and scale against
the oracle."""
import numpy as np
import pytest
import torch

from block_sparse_masked_mask_gb300 import api
from test_cache_gpu import Pair, cu_of, dev, randn
from test_tree_gpu import check_cached_near, partners

pytestmark = pytest.mark.gpu

# new tokens, heads, head_dim, page size: heads in turn x teams of a CTA, of which some stay idle
CASES = {
    "4 x 2 for 5 heads": ([1000] * 12, 5, 128, 32),
    "8 x 2 for 9 heads": ([1000] * 12, 9, 128, 32),
    "2 x 2 for 3 heads, ragged": ([1000] * 6 + [1] * 6 + [700] * 4, 3, 128, 32),
    "4 x 2 for 11 heads": ([1500] * 8, 11, 64, 64),
    "2 x 1, pages of 64 x 128": ([700] * 10, 8, 128, 64),
    "4 x 8, short pages": ([900, 1, 300] * 6, 24, 64, 16),
    "2 x 1, turned twice": ([1280] * 8, 8, 128, 128),
    "2 x 1 for 13 heads, turned twice": ([640] * 8, 13, 128, 128),
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("part,inter", [(2, False), (2, True), (3, False)], ids=["halves", "interleaved", "odd_places"])
@pytest.mark.parametrize("name", CASES)
def test_heads_in_turn(name, part, inter, dtype):
    """Behind tokens that are there already, whose scales mostly rise.  Bounds are those of test_append_rope."""
    n, heads, dim, ps = CASES[name]
    rot = dim if part == 2 else 2 * (dim // 6)  # (halves of 21 or 10 pairs lie at odd places)
    held = [(37 * i) % 61 for i in range(len(n))]
    lens, cu, T = [a + b for a, b in zip(n, held)], cu_of(n), sum(n)
    p = Pair(lens, heads, dim, ps, seed=3)
    p.append(randn(sum(held), heads, dim, seed=8, scale=0.02), randn(sum(held), heads, dim, seed=9, scale=0.02), cu_of(held), held)
    plan = api.attn_rope_plan(rot, interleaved=inter)
    q, k, v = (randn(T, h, dim, seed=i, dtype=dtype, scale=1.5) for i, h in enumerate((2, heads, heads)))
    got = api.attn_cache_append_rope(q.cuda(), k.cuda(), v.cuda(), plan, p.dev, dev(cu), dev(lens), max(n))
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
    at = np.concatenate([np.arange(t - x, t) for t, x in zip(lens, n)]).astype(np.uint64)
    turn = np.array([plan.struct.turn[i] for i in range(rot // 2)], np.uint64)
    z = np.exp(2j * np.pi * ((at[:, None] * turn).astype(np.float64) / 2.0 ** 64))[:, None]  # (the product modulo 2^64)
    exact = []
    for x in (q.double().numpy(), k.double().numpy()):
        y = x.copy()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
        w = (a + 1j * b) * z
        if inter:
            y[..., 0:rot:2], y[..., 1:rot:2] = w.real, w.imag
        else:
            y[..., :rot // 2], y[..., rot // 2:rot] = w.real, w.imag
        exact.append(y)
    off = [2.0 ** -20 * partners(x.double().numpy(), rot, inter) for x in (q, k)]
    err = np.abs(got.double().cpu().numpy() - exact[0])
    assert (err <= off[0] + torch.finfo(dtype).eps / 2 * (np.abs(exact[0]) + off[0])).all()
    check_cached_near(p, exact[1], off[1], v.double().numpy(), cu, lens)
