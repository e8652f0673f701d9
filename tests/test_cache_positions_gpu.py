"""Rotary positions of tokens behind an eviction."""
import numpy as np
import pytest
import torch

from block_sparse_masked_mask_gb300 import api
from test_cache_gpu import Pair, cu_of, dev, randn, run_evict

pytestmark = pytest.mark.gpu


def test_tokens_behind_an_eviction_keep_their_positions():
    """rope -> append -> evict -> rope by positions -> append -> attend is attention over the
    whole text with the dropped tokens hidden; positions from the shortened length
    would turn the new query away from the kept keys."""
    L, dim, ps, group = 300, 64, 32, 2
    plan = api.attn_rope_plan(dim)
    p = Pair([L], 1, dim, ps, seed=1)
    q, k, v = randn(L, group, dim, seed=1), randn(L, 1, dim, seed=2), randn(L, 1, dim, seed=3)
    _, k = api.attn_rope(q.cuda(), k.cuda(), plan, cu_seqlens=dev([0, L]), seq_lens=dev([L]))
    p.append(k.cpu(), v, cu_of([L]), [L])
    drop = np.zeros(L, bool)
    drop[10:150] = True
    w = torch.rand((1, 1, L))
    w[..., torch.from_numpy(drop)] = float("-inf")
    keep = int((~drop).sum())
    dst = Pair([keep + 1], 1, dim, ps, seed=4)
    run_evict(p, dst, w, [L], [keep], 8)
    # the next token: place L of the text, slot `keep` of the cache
    q, k, v = randn(1, group, dim, seed=5, scale=3.0), randn(1, 1, dim, seed=6), randn(1, 1, dim, seed=7)
    there = api.attn_rope(q.cuda(), k.cuda(), plan, positions=dev([L]))
    near = api.attn_rope(q.cuda(), k.cuda(), plan, cu_seqlens=dev([0, 1]), seq_lens=dev([keep + 1]))
    assert not torch.equal(there[0], near[0])
    dst.append(there[1].cpu(), v, cu_of([1]), [keep + 1])
    o, _ = api.attn_cache_fwd(there[0], dst.dev, dev([0, 1]), dev([keep + 1]), 1, keep + 1)
    K = np.concatenate([p.ref.numbers(0, 0, L)[0][~drop], dst.ref.numbers(0, 0, keep + 1)[0][-1:]])
    V = np.concatenate([p.ref.numbers(1, 0, L)[0][~drop], dst.ref.numbers(1, 0, keep + 1)[0][-1:]])
    for g in range(group):
        s = K @ there[0][0, g].double().cpu().numpy() / np.sqrt(dim)
        x = np.exp(s - s.max())
        want = x @ V / x.sum()
        # moved codes lose nothing but subnormals (2^-10 of their page's scale); fp16 weights and
        # a bf16 result are 2^-11 and 2^-8
        assert np.abs(o[0, g].double().cpu().numpy() - want).max() <= 2.0 ** -6 * np.abs(V).max()
