"""The entry points for drafted trees without a GPU: exported symbols, refused
arguments (before any launch), and the oracle against hand-written trees."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from conftest import ROOT
from oracle import tree as R
from test_cache_abi import BAD_CACHES, INVALID, OK, SMALL, UNSUPPORTED, a_cache, fake

HEADER = os.path.join(ROOT, "include", "attn_tree.h")


def test_library_exports_every_declared_symbol(native_lib):
    names = re.findall(r"ATTN_API\s+[\w\s\*]+?\b(attn_\w+)\s*\(", open(HEADER).read())
    assert len(names) == 5
    for name in names:
        assert hasattr(native_lib, name), name


def test_oracle_of_ancestors():
    seen = R.ancestors([-1, 0, 0, 1, -1, 3])
    want = ["100000", "110000", "101000", "110100", "000010", "110101"]
    assert ["".join("01"[x] for x in row) for row in seen.astype(int)] == want
    bits = R.to_bits([seen, R.ancestors([-1])], 2)
    assert bits.shape == (7, 2) and bits[:, 1].sum() == 0
    assert bits[:, 0].tolist() == [1, 3, 5, 11, 16, 43, 1]
    assert R.to_bits([np.eye(40, dtype=bool)], 2)[39].tolist() == [0, 1 << 7]


def calls(L):
    from block_sparse_masked_mask_gb300 import api
    plan = api.attn_rope_plan(128).struct
    build = dict(parents=fake(), T=8, cu=fake(), lens=fake(), max_new=4, bits=fake(), words=1, pos=fake())
    app = dict(q=fake(), qo=fake(0x90000), qs=512, qos=512, H=4, k=fake(), v=fake(), ks=256, vs=256, dtype=0, T=8,
               pos=fake(), cu=fake(), lens=fake(), max_new=4, plan=ctypes.byref(plan))
    fwd = dict(q=fake(), o=fake(), lse=fake(), dtype=0, T=8, H=4, scale=0.0, bits=fake(), words=1, cu=fake(), max_new=4,
               lens=fake(), max_len=256)
    keep = dict(path=fake(), stride=4, counts=fake(0x11000), cu=fake(0x12000), lens=fake(0x13000), max_new=4,
                new=fake(0x14000))

    def tree_fwd(cache=None, ws=fake(0x70000), nbytes=1 << 30, **kw):
        return L.attn_cache_tree_fwd(*dict(fwd, **kw).values(), ctypes.byref(cache or a_cache()), ws, nbytes, None)

    def of(f, base):
        return lambda cache=None, **kw: f(*dict(base, **kw).values(), ctypes.byref(cache or a_cache()), None)

    return (of(L.attn_cache_tree_build, build), of(L.attn_cache_append_rope, app), tree_fwd,
            of(L.attn_cache_tree_keep, keep), plan)


@pytest.mark.parametrize("bad,status", BAD_CACHES, ids=lambda x: str(x))
def test_bad_caches_are_refused(native_lib, bad, status):
    build, append, fwd, keep, _ = calls(native_lib)
    for call in (build, append, fwd, keep):
        assert call(a_cache(**bad)) == status
    out = ctypes.c_size_t()
    assert native_lib.attn_cache_tree_fwd_workspace_size(ctypes.byref(a_cache(**bad)), 8, 4, 4, 256, ctypes.byref(out)) == status


def test_bad_arguments_are_refused_before_any_launch(native_lib):
    from block_sparse_masked_mask_gb300 import _native, api
    build, append, fwd, keep, plan = calls(native_lib)
    for call, names in ((build, ("parents", "cu", "lens", "bits")), (append, ("q", "qo", "k", "v", "cu", "lens", "plan")),
                        (fwd, ("q", "o", "lse", "bits", "cu", "lens")), (keep, ("path", "counts", "cu", "lens", "new"))):
        for name in names:
            assert call(**{name: None}) == INVALID, name
    for call in (build, append, fwd, keep):
        assert call(max_new=-1) == INVALID
        assert call(cu=fake(0x10002)) == INVALID and call(lens=fake(0x10001)) == INVALID
    for call in (build, append, fwd):
        assert call(T=-1) == INVALID
        assert call(T=0) == OK and call(max_new=0) == OK
    assert build(words=0) == INVALID and build(words=-1) == INVALID and build(max_new=33) == INVALID
    assert build(parents=fake(0x10001)) == INVALID and build(bits=fake(0x10002)) == INVALID and build(pos=fake(0x10002)) == INVALID
    # the rotation's and the append's own
    assert append(plan=ctypes.byref(_native.AttnRopePlan())) == INVALID
    assert append(a_cache(head_dim=64)) == INVALID            # the plan turns 128 dimensions
    assert append(H=-1) == INVALID and append(H=40000) == UNSUPPORTED
    assert append(dtype=3) == INVALID
    assert append(qs=511) == INVALID and append(qos=511) == INVALID
    assert append(q=fake(0x20000), qo=fake(0x20000), qos=1024) == INVALID
    assert append(q=fake(0x10001)) == INVALID and append(dtype=1, q=fake(0x10002)) == INVALID
    assert append(k=fake(0x10008)) == INVALID and append(v=fake(0x10008)) == INVALID
    assert append(ks=255) == INVALID and append(vs=257) == INVALID and append(ks=260) == INVALID
    assert append(pos=fake(0x10002)) == INVALID
    # the attention's
    assert fwd(words=0) == INVALID and fwd(max_new=64) == INVALID and fwd(bits=fake(0x10002)) == INVALID
    assert fwd(dtype=1) == UNSUPPORTED and fwd(dtype=2) == INVALID
    assert fwd(H=3) == INVALID and fwd(H=0) == INVALID
    assert fwd(scale=-1.0) == INVALID and fwd(scale=float("nan")) == INVALID
    assert fwd(max_len=257) == INVALID and fwd(max_len=-1) == INVALID
    assert fwd(q=fake(0x10008)) == INVALID and fwd(o=fake(0x10008)) == INVALID and fwd(lse=fake(0x10002)) == INVALID
    assert fwd(T=1 << 29) == UNSUPPORTED
    out = ctypes.c_size_t()
    c = a_cache(page_size=128, max_pages=1 << 13)
    assert native_lib.attn_cache_tree_fwd_workspace_size(ctypes.byref(c), 8, 4, 8, 1 << 20, ctypes.byref(out)) == OK
    if out.value:
        assert fwd(c, max_new=8, max_len=1 << 20, ws=None, nbytes=0) in (INVALID, SMALL)
        assert fwd(c, max_new=8, max_len=1 << 20, nbytes=out.value - 1) == SMALL
        assert fwd(c, max_new=8, max_len=1 << 20, ws=fake(0x70010)) == INVALID
    assert native_lib.attn_cache_tree_fwd_workspace_size(ctypes.byref(c), 8, 4, 8, 1 << 20, None) == INVALID
    # the path's
    assert keep(stride=-1) == INVALID
    for name in ("lens", "counts", "cu"):  # lengths over what is still read
        assert keep(new=fake({"lens": 0x13000, "counts": 0x11000, "cu": 0x12000}[name])) == INVALID
    assert keep(path=fake(0x10002)) == INVALID and keep(new=fake(0x14001)) == INVALID


def test_the_binding_refuses_wrong_tensors(native_lib):
    from block_sparse_masked_mask_gb300 import api
    x = torch.zeros(3)
    for call in (lambda: api.attn_cache_tree_build(x, None, x, x, 1),
                 lambda: api.attn_cache_append_rope(x, x, x, None, None, x, x, 1),
                 lambda: api.attn_cache_tree_fwd(x, None, x, x, x, 1, 1),
                 lambda: api.attn_cache_tree_keep(x, x, None, x, x, 1)):
        with pytest.raises(api.AttnError):
            call()
