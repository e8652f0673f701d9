"""Waits of the tcgen05 cache kernels that run out while other warps are still
starting: every warp of a CTA starts its role or none does, so that meetings of
warps that have no bound of their own are reached by all of them."""
import os
import re

import pytest
import torch

from conftest import ROOT

CSRC = os.path.join(ROOT, "block_sparse_masked_mask_gb300", "csrc")


@pytest.mark.parametrize("name", ["cache_chunk.cu", "cache_weights_many.cu"])
def test_roles_start_by_a_word_that_no_wait_writes(name):
    """The waits set *abort_flag (misc[1]) at any time; the word that decides whether a
    warp takes its role is another one, written once, before the barrier behind
    which it is read."""
    code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    assert re.search(r"abort_flag = misc \+ 1;", code)
    assert not re.search(r"(=|if \()\s*\*abort_flag\b", code.replace("misc[2] = *abort_flag = ", ""))
    written = [m.start() for m in re.finditer(r"misc\[2\] = ", code)]
    read = [m.start() for m in re.finditer(r"misc\[2\] != 0u", code)]
    assert len(written) == 1 and len(read) == 1
    assert written[0] < code.index("__syncthreads();", written[0]) < read[0]


@pytest.mark.gpu
@pytest.mark.parametrize("heads,rows", [(8, 17), (8, 40), (2, 128), (4, 300)])
def test_many_launches_whose_waits_run_out_return(heads, rows):
    """Waits of 100 ns, one and two M tiles of rows, about as many CTAs as SMs: every
    launch returns, whether a wait ran out in it or none did; the ordinary library is
    right afterwards."""
    from block_sparse_masked_mask_gb300 import _native, api
    from block_sparse_masked_mask_gb300 import build as B
    from test_cache_gpu import check_attend, cu_of, dev, filled, randn, run_attend
    lens = [900 + 200 * i for i in range(12)]
    p = filled(lens, heads, 64, 32, seed=1)
    cu, q = cu_of([rows] * 12), randn(12 * rows, heads, 64, seed=2)
    lse = run_attend(p, q, cu, lens)[1].clone()
    args = (q.cuda(), p.dev, dev(cu), dev(lens), rows, max(lens))
    weigh = (args[0], lse) + args[1:]
    torch.cuda.synchronize()
    with _native.use_library(B.build_variant("waitshort", {"ATTN_WAIT_TIMEOUT_NS": "100ull"})):
        for _ in range(20):
            api.attn_cache_fwd(*args)
            assert api.attn_cache_get_status(p.dev) in (api.ATTN_OK, api.ATTN_ERR_DEVICE_TIMEOUT)
            api.attn_cache_weights(*weigh)
            assert api.attn_cache_get_status(p.dev) in (api.ATTN_OK, api.ATTN_ERR_DEVICE_TIMEOUT)
    check_attend(p, q, cu, lens)
