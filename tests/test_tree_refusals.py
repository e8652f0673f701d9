"""Calls on drafted trees that are refused because their results lie over what is still read."""
import ctypes

import pytest
import torch

from test_cache_abi import INVALID, a_cache, fake


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can be launched")
def test_results_over_inputs_are_refused(native_lib):
    batch = a_cache().batch

    def build(parents=0x10000, cu=0x20000, lens=0x30000, bits=0x40000, pos=0x50000, T=8, words=2, max_new=8):
        return native_lib.attn_cache_tree_build(fake(parents), T, fake(cu), fake(lens), max_new, fake(bits), words,
                                                fake(pos) if pos else None, ctypes.byref(a_cache()), None)

    def keep(path=0x10000, stride=3, counts=0x20000, cu=0x30000, lens=0x40000, new=0x50000):
        return native_lib.attn_cache_tree_keep(fake(path), stride, fake(counts), fake(cu), fake(lens), 8, fake(new),
                                               ctypes.byref(a_cache()), None)

    assert build() != INVALID and keep() != INVALID
    for at, size in ((0x10000, 8 * 4), (0x20000, (batch + 1) * 4), (0x30000, batch * 4)):
        for name, own in (("pos", 8 * 4), ("bits", 8 * 2 * 4)):
            for over in (at, at + size - 4, at - own + 4):
                assert build(**{name: over}) == INVALID, (name, hex(over))
            for beside in (at + size, at - own):
                assert build(**{name: beside}) != INVALID, (name, hex(beside))
    assert build(pos=0x40000 + 60) == INVALID and build(pos=0x40000 + 64) != INVALID
    assert build(pos=0, bits=0x10000) == INVALID and build(pos=0) != INVALID
    assert build(pos=0x10000, T=0) != INVALID and build(pos=0x10000, max_new=0) != INVALID  # nothing is written
    for at, size in ((0x10000, batch * 3 * 4), (0x20000, batch * 4), (0x30000, (batch + 1) * 4), (0x40000, batch * 4)):
        for over in (at, at + size - 4, at - batch * 4 + 4):
            assert keep(new=over) == INVALID, hex(over)
        for beside in (at + size, at - batch * 4):
            assert keep(new=beside) != INVALID, hex(beside)
    assert keep(stride=1, new=0x10000) == INVALID and keep(stride=0, new=0x10000) != INVALID


@pytest.mark.gpu
def test_the_binding_refuses_them_and_takes_neighbours():
    from block_sparse_masked_mask_gb300 import api
    from test_cache_gpu import dev, filled
    p = filled([40, 50], 1, 64, 32, seed=1)
    cu, lens = dev([0, 300, 302]), dev([400, 50])
    room = torch.zeros(302 * 13, dtype=torch.int32, device="cuda")
    parents = room[:302]
    parents.copy_(torch.tensor(list(range(-1, 299)) + [-1, 0]))
    wide = api.KVCache(p.dev.k_pages, p.dev.v_pages, p.dev.k_scale, p.dev.v_scale, dev([[0] * 20, [1] * 20]))
    for kw in (dict(positions=parents), dict(bits=room[:3020].view(302, 10)), dict(positions=room[302:604], bits=room[302:3322].view(302, 10))):
        with pytest.raises(api.AttnError) as e:
            api.attn_cache_tree_build(parents, wide, cu, lens, 300, **kw)
        assert e.value.status == api.ATTN_ERR_INVALID_ARG
    bits, positions = api.attn_cache_tree_build(parents, wide, cu, lens, 300, positions=room[302:604],
                                                bits=room[604:3624].view(302, 10))
    assert api.attn_cache_get_status(wide) == api.ATTN_OK
    assert positions.tolist() == list(range(100, 400)) + [48, 49] and bits[301, 0] == 3 and bits[299, 9] == (1 << 12) - 1
    small = torch.tensor([2, 1, 1, 1, -1, -1], dtype=torch.int32, device="cuda")  # path [2, 1], counts [2], new_lens [2]
    args = (small[2:4], p.dev, dev([0, 4, 8]), dev([40, 50]), 4)
    with pytest.raises(api.AttnError):
        api.attn_cache_tree_keep(small[:2].view(2, 1), *args, new_lens=small[:2])
    assert small.tolist() == [2, 1, 1, 1, -1, -1]
    api.attn_cache_tree_keep(small[:2].view(2, 1), *args, new_lens=small[4:])
    assert small.tolist() == [2, 1, 1, 1, 37, 47] and api.attn_cache_get_status(p.dev) == api.ATTN_OK
