"""How attn_cache_fwd cuts its work: the workspace's ceiling."""
import ctypes

import pytest

from test_cache_abi import a_cache

CEILING = 512 << 20


def workspace(lib, T, H, max_new, max_len, **kw):
    c = a_cache(page_size=128, max_pages=1 << 13, **kw)
    out = ctypes.c_size_t()
    assert lib.attn_cache_fwd_workspace_size(ctypes.byref(c), T, H, max_new, max_len, ctypes.byref(out)) == 0
    return out.value


@pytest.mark.parametrize("max_len", [4096, 32768, 131072, 1 << 20])
@pytest.mark.parametrize("new", [17, 300, 2048, 8192, 16384, 32768])
@pytest.mark.parametrize("batch,heads,group,dim", [(1, 8, 4, 128), (16, 8, 4, 128), (64, 1, 8, 64), (3, 32, 1, 32)])
def test_the_workspace_has_a_ceiling(native_lib, batch, heads, group, dim, new, max_len):
    """Partial results of every chunk, but never more than the ceiling."""
    size = workspace(native_lib, new * batch, heads * group, new, max_len, num_kv_heads=heads, head_dim=dim, batch=batch)
    row = new * batch * heads * group * (4 * dim + 8)
    assert size <= CEILING and size % row == 0
    assert size != row  # one chunk's rows are not written twice


def test_few_rows_over_long_sequences_are_still_cut(native_lib):
    assert workspace(native_lib, 512, 32, 512, 131072, num_kv_heads=8, batch=1) >= 8 * 512 * 32 * 520


@pytest.mark.gpu
@pytest.mark.parametrize("bound", [1 << 19, 2000])
def test_attention_at_the_ceiling(bound):
    """64000 rows under a bound that would ask for 128 chunks, and under their own."""
    from block_sparse_masked_mask_gb300 import api
    from test_cache_gpu import Pair, check_attend, cu_of, randn
    lens, new = [2000, 1500, 700], [1000, 900, 100]
    p = Pair(lens, 1, 32, 64, seed=1, width=1 << 13)
    p.append(randn(4200, 1, 32, seed=1), randn(4200, 1, 32, seed=2), cu_of(lens), lens)
    assert api.attn_cache_fwd_workspace_size(p.dev, 2000, 32, 1000, bound) <= CEILING
    check_attend(p, randn(2000, 32, 32, seed=3), cu_of(new), lens, max_seqlen=bound)
