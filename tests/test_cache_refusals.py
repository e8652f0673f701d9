"""Calls that are refused because their copies would read what they write."""
import ctypes

import pytest
import torch

from test_cache_abi import INVALID, a_cache, fake


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can be launched")
def test_eviction_into_its_own_pages_is_refused(native_lib):
    def evict(dst, max_keep=100):
        return native_lib.attn_cache_evict(fake(), 256, fake(0x11000), fake(0x12000), 0, 256, max_keep,
                                           ctypes.byref(a_cache()), ctypes.byref(dst), fake(0x90000), fake(0xA0000), 100,
                                           fake(0xB0000), None)
    assert evict(a_cache()) == INVALID
    assert evict(a_cache(v_pages=0x70000)) == INVALID       # the keys' pool alone is shared
    assert evict(a_cache(k_pages=0x70000)) == INVALID
    assert evict(a_cache(page_table=0x70000)) != INVALID    # one pool, other pages
    assert evict(a_cache(k_pages=0x70000, v_pages=0x80000)) != INVALID
    assert evict(a_cache(), max_keep=0) != INVALID          # nothing is copied


@pytest.mark.gpu
def test_the_binding_refuses_it_and_takes_other_pages_of_the_pool():
    from block_sparse_masked_mask_gb300 import api
    from test_cache_gpu import dev, filled
    p = filled([100, 90], 2, 64, 32, seed=1)
    d = p.dev
    w, lens, budgets = torch.rand((2, 2, 100), device="cuda"), dev([100, 90]), dev([30, 20])
    before = d.k_pages.clone()
    with pytest.raises(api.AttnError) as e:
        api.attn_cache_evict(w, d, d, lens, budgets, 4, 100, 30)
    assert e.value.status == api.ATTN_ERR_INVALID_ARG
    assert torch.equal(d.k_pages, before) and api.attn_cache_get_status(d) == api.ATTN_OK
    free = [x for x in range(d.num_pages) if x not in p.table]
    other = api.KVCache(d.k_pages, d.v_pages, d.k_scale, d.v_scale, dev([[free[0]], [free[1]]]))
    _, _, n = api.attn_cache_evict(w, d, other, lens, budgets, 4, 100, 30)
    assert n.cpu().tolist() == [30, 20] and api.attn_cache_get_status(d) == api.ATTN_OK
