"""Drafted trees behind an eviction: attn_cache_tree_build counts the tokens that are held, so
the caller adds what was dropped."""
import numpy as np
import pytest
import torch

from block_sparse_masked_mask_gb300 import api
from oracle import tree as R
from test_cache_gpu import Pair, cu_of, dev, randn, run_evict
from test_tree_gpu import device_bits, random_parents

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,group", [(9, 2), (40, 4)])
def test_trees_behind_an_eviction_keep_their_positions(n, group):
    """rope -> append -> evict -> build -> positions + dropped -> append_rope -> tree_fwd is attention over the
    whole text with the dropped tokens hidden."""
    L, dim, ps = 300, 64, 32
    plan = api.attn_rope_plan(dim)
    p = Pair([L], 1, dim, ps, seed=1)
    k, v = randn(L, 1, dim, seed=2), randn(L, 1, dim, seed=3)
    k, _ = api.attn_rope(k.cuda(), None, plan, positions=dev(np.arange(L)))
    p.append(k.cpu(), v, cu_of([L]), [L])
    drop = np.zeros(L, bool)
    drop[10:150] = True
    w = torch.rand((1, 1, L))
    w[..., torch.from_numpy(drop)] = float("-inf")
    keep = int((~drop).sum())
    dst = Pair([keep + n], 1, dim, ps, seed=4)
    run_evict(p, dst, w, [L], [keep], 8)
    parents = random_parents(n, np.random.default_rng(n))
    mask, cu, lens = R.ancestors(parents), dev([0, n]), dev([keep + n])
    bits, positions = api.attn_cache_tree_build(dev(parents), dst.dev, cu, lens, n)
    assert positions.tolist() == (keep + mask.sum(1) - 1).tolist()
    positions = positions + (L - keep)
    q, k, v = (randn(n, h, dim, seed=5 + h, scale=2.0).cuda() for h in (group, 1, 1))
    turned = api.attn_cache_append_rope(q, k, v, plan, dst.dev, cu, lens, n, positions=positions)
    rope_q, rope_k = api.attn_rope(q, k, plan, positions=dev(L + mask.sum(1) - 1))
    assert ((turned.float() - rope_q.float()).abs() <= 2.0 ** -7 * rope_q.float().abs() + 2.0 ** -20).all()
    o, _ = api.attn_cache_tree_fwd(turned, dst.dev, bits, cu, lens, n, keep + n)
    assert torch.equal(bits, device_bits(R.to_bits([mask], bits.shape[1]))) and api.attn_cache_get_status(dst.dev) == api.ATTN_OK
    codes = dst.dev.k_pages.cpu().numpy(), dst.dev.v_pages.cpu().numpy()
    dst.ref.codes, dst.ref.scale = list(codes), [x.cpu().double().numpy() for x in (dst.dev.k_scale, dst.dev.v_scale)]
    new_k, new_v = (dst.ref.numbers(s, 0, keep + n)[0][keep:] for s in (0, 1))
    # (a code is off by half a step, 2^-4 of itself or 2^-10 of the scale; attn_rope's keys by 2^-8)
    exact = rope_k[:, 0].double().cpu().numpy()
    assert (np.abs(new_k - exact) <= (2.0 ** -4 + 2.0 ** -7) * np.abs(exact) + 2.0 ** -9 * np.abs(exact).max()).all()
    K = np.concatenate([p.ref.numbers(0, 0, L)[0][~drop], new_k])
    V = np.concatenate([p.ref.numbers(1, 0, L)[0][~drop], new_v])
    seen = np.concatenate([np.ones((n, keep), bool), mask], 1)
    for g in range(group):
        s = np.where(seen, turned[:, g].double().cpu().numpy() @ K.T / np.sqrt(dim), -np.inf)
        x = np.exp(s - s.max(1, keepdims=True))
        want = x @ V / x.sum(1, keepdims=True)
        # bounds of test_cache_positions_gpu: moved codes lose subnormals only, fp16 weights and a bf16 result 2^-11 and
        # 2^-8; queries are two e4m3 numbers, 2^-17 of their largest element, which a score sums over the dimensions
        score = 2.0 ** -17 * float(turned.float().abs().max()) * np.abs(K).sum(1).max() / np.sqrt(dim)
        assert np.abs(o[:, g].double().cpu().numpy() - want).max() <= (2.0 ** -6 + 2 * score) * np.abs(V).max()
