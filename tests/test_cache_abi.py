"""The rotary and cache entry points without a GPU: exported symbols, refused
arguments (before any launch), the rotation plan's numbers, workspace sizes,
and the oracle's e4m3 against the format's definition."""
import ctypes
import os
import re
from fractions import Fraction

import numpy as np
import pytest

from conftest import ROOT
from oracle import cache as C

HEADER = os.path.join(ROOT, "include", "attn_cache.h")
OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3


def fake(addr=0x10000):
    return ctypes.c_void_p(addr)


def a_cache(**kw):
    from block_sparse_masked_mask_gb300 import _native
    f = dict(k_pages=0x10000, v_pages=0x20000, k_scale=0x30000, v_scale=0x40000, page_table=0x50000, status=0x60000,
             num_pages=10, num_kv_heads=2, page_size=64, head_dim=128, batch=3, max_pages=4)
    f.update(kw)
    return _native.AttnKVCache(*(f[n] for n, _ in _native.AttnKVCache._fields_))


BAD_CACHES = [(dict(k_pages=0), INVALID), (dict(v_pages=0), INVALID), (dict(k_scale=0), INVALID),
              (dict(v_scale=0), INVALID), (dict(page_table=0), INVALID), (dict(status=0), INVALID),
              (dict(k_pages=0x10008), INVALID), (dict(v_scale=0x40002), INVALID), (dict(num_pages=0), INVALID),
              (dict(num_kv_heads=0), INVALID), (dict(batch=0), INVALID), (dict(max_pages=0), INVALID),
              (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
              (dict(batch=70000), UNSUPPORTED), (dict(max_pages=1 << 25), UNSUPPORTED)]


def test_library_exports_every_declared_symbol(native_lib):
    names = re.findall(r"ATTN_API\s+[\w\s\*]+?\b(attn_\w+)\s*\(", open(HEADER).read())
    assert len(names) == 8
    for name in names:
        assert hasattr(native_lib, name), name


def test_rope_plan_numbers(native_lib):
    """turn[i] is 2^64 theta_i / (2 pi), for every scaling."""
    from block_sparse_masked_mask_gb300 import api
    for scaling in ("none", "linear", "ntk", "ramp"):
        for rot in (2, 4, 40, 128):
            if scaling == "ntk" and rot == 2:
                continue
            kw = dict(scaling=scaling, factor=8.0, original_context=4096.0, alpha=1.0, beta=32.0)
            plan = api.attn_rope_plan(rot, base=10000.0, interleaved=True, **kw)
            theta, m = C.rope_angles(rot, 10000.0, **kw)
            turn = np.array([plan.struct.turn[i] for i in range(rot // 2)], np.float64) / 2.0 ** 64
            # a handful of fp64 operations on either side (2^-48 is far above their rounding), and the
            # fixed point's step of 2^-64 turn, which a position of 2^31 makes 2^-33
            assert (np.abs(turn - theta / (2 * np.pi)) <= 2.0 ** -48 * theta + 2.0 ** -64).all()
            assert plan.struct.interleaved == 1 and plan.rotary_dim == rot
            assert abs(plan.struct.result_factor - m) <= 2.0 ** -24 * m
    assert abs(api.attn_rope_plan(64, result_factor=0.5).struct.result_factor - 0.5) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(rotary_dim=0), 1), (dict(rotary_dim=7), 1), (dict(rotary_dim=130), 2), (dict(base=1.0), 1),
    (dict(base=float("nan")), 1), (dict(scaling="linear", factor=0.5), 1), (dict(scaling="ntk", factor=2.0, rotary_dim=2), 1),
    (dict(scaling="ramp", factor=2.0), 1), (dict(scaling="ramp", factor=2.0, original_context=10.0, alpha=3, beta=3), 1),
    (dict(result_factor=-1.0), 1), (dict(result_factor=float("inf")), 1), (dict(scaling="other"), 1)])
def test_rope_plan_refusals(native_lib, kw, status):
    from block_sparse_masked_mask_gb300 import api
    with pytest.raises(api.AttnError) as e:
        api.attn_rope_plan(**{"rotary_dim": 64, **kw})
    assert e.value.status == status


def test_rope_refuses_bad_arguments_before_any_launch(native_lib):
    from block_sparse_masked_mask_gb300 import _native, api
    plan = api.attn_rope_plan(64).struct
    base = dict(q=fake(), qo=fake(), qs=512, qos=512, H=4, k=fake(), ko=fake(), ks=256, kos=256, Hk=2, dtype=0, T=8,
                D=128, pos=fake(), cu=None, lens=None, B=0, plan=ctypes.byref(plan), inv=0)

    def call(**kw):
        a = dict(base, **kw)
        return native_lib.attn_rope(*(a[n] for n in base), None)

    for name in ("q", "qo", "k", "ko", "plan"):
        assert call(**{name: None}) == INVALID, name
    assert call(pos=None) == INVALID
    assert call(pos=None, cu=fake(), B=0) == INVALID
    assert call(H=0) == INVALID and call(Hk=-1) == INVALID and call(T=-1) == INVALID
    assert call(dtype=3) == INVALID
    assert call(D=96) == UNSUPPORTED
    assert call(D=32) == INVALID                      # the plan turns 64 dimensions
    assert call(qs=511) == INVALID and call(kos=255) == INVALID
    assert call(q=fake(0x20000), qo=fake(0x20000), qos=1024) == INVALID  # in place, rows over other rows
    assert call(k=fake(0x20000), ko=fake(0x20000), ks=1024) == INVALID
    assert call(q=fake(0x10001)) == INVALID and call(pos=fake(0x10002)) == INVALID
    assert call(dtype=1, k=fake(0x10002)) == INVALID
    assert call(plan=ctypes.byref(_native.AttnRopePlan())) == INVALID  # never initialised
    assert call(T=0) == OK


def test_cache_calls_refuse_bad_arguments_before_any_launch(native_lib):
    L = native_lib
    app = dict(k=fake(), v=fake(), ks=256, vs=256, dtype=0, T=8, cu=fake(), lens=fake(), max_new=4)
    fwd = dict(q=fake(), o=fake(), lse=fake(), dtype=0, T=8, H=4, scale=0.0, cu=fake(), max_new=4, lens=fake(),
               max_len=256, kind=0)
    wgt = dict(q=fake(), lse=fake(), dtype=0, T=8, H=4, scale=0.0, cu=fake(), max_new=4, lens=fake(), max_len=256, kind=0)
    ev = dict(w=fake(), ws=256, lens=fake(), budgets=fake(), recent=0, max_len=256, max_keep=100)

    def append(cache=None, **kw):
        return L.attn_cache_append(*dict(app, **kw).values(), ctypes.byref(cache or a_cache()), None)

    def attend(cache=None, ws=fake(0x70000), nbytes=1 << 30, **kw):
        return L.attn_cache_fwd(*dict(fwd, **kw).values(), ctypes.byref(cache or a_cache()), ws, nbytes, None)

    def weigh(cache=None, prev=None, out=fake(0x80000), stride=256, **kw):
        return L.attn_cache_weights(*dict(wgt, **kw).values(), ctypes.byref(cache or a_cache()), prev, out, stride, None)

    def evict(cache=None, dst=None, kept=fake(0x90000), nw=fake(0xA0000), ns=100, nl=fake(0xB0000), **kw):
        return L.attn_cache_evict(*dict(ev, **kw).values(), ctypes.byref(cache or a_cache()),
                                  ctypes.byref(dst or a_cache()), kept, nw, ns, nl, None)

    for kw, status in BAD_CACHES:
        bad = a_cache(**kw)
        for call in (append, attend, weigh, evict):
            assert call(cache=bad) == status, (call.__name__, kw)
        assert evict(dst=bad) == status
        assert L.attn_cache_get_status(ctypes.byref(bad), None) == status
    assert L.attn_cache_get_status(None, None) == INVALID

    for name in ("k", "v", "cu", "lens"):
        assert append(**{name: None}) == INVALID, name
    assert append(T=-1) == INVALID and append(max_new=-1) == INVALID and append(dtype=2) == INVALID
    assert append(ks=255) == INVALID and append(vs=257) == INVALID and append(k=fake(0x10008)) == INVALID
    assert append(T=0) == OK and append(max_new=0) == OK

    for call, names in ((attend, ("q", "o", "lse", "cu", "lens")), (weigh, ("q", "lse", "cu", "lens", "out"))):
        for name in names:
            assert call(**{name: None}) == INVALID, (call.__name__, name)
        assert call(dtype=1) == UNSUPPORTED and call(dtype=2) == INVALID
        assert call(kind=1) == UNSUPPORTED and call(kind=9) == INVALID
        assert call(scale=-1.0) == INVALID and call(scale=float("inf")) == INVALID
        assert call(H=3) == INVALID and call(H=0) == INVALID
        assert call(max_len=257) == INVALID and call(max_len=-1) == INVALID
        assert call(q=fake(0x10008)) == INVALID and call(lens=fake(0x10001)) == INVALID
        assert call(T=1 << 29) == UNSUPPORTED
    assert attend(o=fake(0x10004)) == INVALID
    assert weigh(stride=255) == INVALID and weigh(prev=fake(0x80002)) == INVALID
    assert attend(T=0) == OK and attend(max_new=0) == OK

    for name in ("w", "lens", "budgets", "kept", "nw", "nl"):
        assert evict(**{name: None}) == INVALID, name
    assert evict(recent=-1) == INVALID and evict(max_keep=-1) == INVALID and evict(max_len=257) == INVALID
    assert evict(ws=255) == INVALID and evict(ns=99) == INVALID and evict(max_keep=257, ns=300) == INVALID
    assert evict(nl=fake()) == INVALID                      # the lengths themselves
    assert evict(nw=fake()) == INVALID                      # the weights themselves
    for kw in (dict(num_kv_heads=1), dict(head_dim=64), dict(page_size=32), dict(batch=2)):
        assert evict(dst=a_cache(max_pages=8, **kw)) == INVALID, kw


def test_workspace_size(native_lib):
    L, out = native_lib, ctypes.c_size_t()

    def size(T, H, max_new, max_len, **kw):
        c = a_cache(max_pages=4096, **kw)
        assert L.attn_cache_fwd_workspace_size(ctypes.byref(c), T, H, max_new, max_len, ctypes.byref(out)) == OK
        return out.value

    assert size(3, 4, 1, 64) == 0                           # one chunk: nothing to join
    n = size(3, 4, 1, 20000)
    assert n > 0 and n % (3 * 4 * (128 * 4 + 8)) == 0       # O, m and the sum per row and chunk
    assert size(3, 4, 1, 200000) >= n
    assert L.attn_cache_fwd_workspace_size(ctypes.byref(a_cache()), 3, 4, 1, 64, None) == INVALID
    assert L.attn_cache_fwd_workspace_size(ctypes.byref(a_cache()), 3, 5, 1, 64, ctypes.byref(out)) == INVALID
    c = a_cache(max_pages=4096)
    L.attn_cache_fwd_workspace_size(ctypes.byref(c), 3, 4, 1, 20000, ctypes.byref(out))
    assert L.attn_cache_fwd(fake(), fake(), fake(), 0, 3, 4, 0.0, fake(), 1, fake(), 20000, 0, ctypes.byref(c),
                            fake(0x70000), out.value - 1, None) == SMALL
    assert L.attn_cache_fwd(fake(), fake(), fake(), 0, 3, 4, 0.0, fake(), 1, fake(), 20000, 0, ctypes.byref(c),
                            fake(0x70010), out.value, None) == INVALID


def test_binding_refuses_host_tensors_before_any_call():
    import torch
    from block_sparse_masked_mask_gb300 import api
    q = torch.zeros((8, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(api.AttnError) as e:
        api.attn_rope(q, None, None, positions=torch.zeros(8, dtype=torch.int32))
    assert e.value.status == 1 and "CUDA tensor" in str(e.value)
    pages = torch.zeros((2, 2, 64, 64), dtype=torch.uint8)
    with pytest.raises(api.AttnError) as e:
        api.KVCache(pages, pages, torch.ones(2, 2), torch.ones(2, 2), torch.zeros((1, 1), dtype=torch.int32))
    assert e.value.status == 1 and "CUDA tensor" in str(e.value)
    for call in (lambda: api.attn_cache_append(q, q, None, None, None, 1),
                 lambda: api.attn_cache_fwd(q, None, None, None, 1, 8),
                 lambda: api.attn_cache_weights(q, None, None, None, None, 1, 8),
                 lambda: api.attn_cache_evict(q, None, None, None, None, 0, 8, 8),
                 lambda: api.attn_cache_get_status(None)):
        with pytest.raises(api.AttnError) as e:
            call()
        assert e.value.status == 1


# ------------------------------------------------------------------ the oracle itself

def test_oracle_e4m3_is_the_format():
    assert C.E4M3[0x7E] == 448 and C.E4M3[1] == 2.0 ** -9 and C.E4M3[8] == 2.0 ** -6 and C.E4M3[0xB8] == -1
    finite = [c for c in range(256) if c & 0x7F != 0x7F]
    for c in finite:
        if c != 0x80:  # -0 encodes by its sign
            assert C.e4m3_encode(C.E4M3[c]) == c
    assert C.e4m3_encode(-0.0) == 0x80
    # nearest: no representable number is nearer, ties have an even mantissa
    rng = np.random.default_rng(0)
    vals = np.sort(C.E4M3[:0x7F])
    x = np.concatenate([rng.uniform(0, 460, 500), 2.0 ** rng.uniform(-12, 9, 500), (vals[1:] + vals[:-1]) / 2])
    for v, c in zip(x, C.e4m3_encode(x)):
        err = abs(Fraction(float(C.E4M3[c])) - Fraction(float(min(v, 448.0))))
        best = min(abs(Fraction(float(y)) - Fraction(float(min(v, 448.0)))) for y in vals)
        assert err == best
        if v < 448 and np.sum(np.abs(vals - v) == float(best)) == 2:
            assert c % 2 == 0
    assert C.e4m3_encode(np.inf) == 0x7E and C.e4m3_encode(-np.inf) == 0xFE and C.e4m3_encode(np.nan) == 0x7F


def test_oracle_scale_is_the_least_power_of_two():
    for x in (1.0, 448.0, 448.0001, 449.0, 7.0, 7.0000001, 1e-30, 3e38):
        s = C.scale_for([x, np.inf, np.nan])
        e = np.log2(s)
        assert e == int(e) and (x <= 448 * s or e == 120) and (x > 448 * s / 2 or e == -80)
    assert C.scale_for([0.0]) == 2.0 ** -80 and C.scale_for([np.nan]) == 2.0 ** -80


def test_oracle_rotation_is_the_matrix():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 6))
    theta, _ = C.rope_angles(4, 100.0)
    pos = np.array([0, 3, -2])
    for inter, pairs in ((False, [(0, 2), (1, 3)]), (True, [(0, 1), (2, 3)])):
        want = x.copy()
        for t in range(3):
            for i, (a, b) in enumerate(pairs):
                c, s = np.cos(pos[t] * theta[i]), np.sin(pos[t] * theta[i])
                want[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
                want[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
        got = C.rope(x, pos, theta, inter)
        assert np.allclose(got, want, atol=1e-14)
        assert np.allclose(C.rope(got, pos, theta, inter, inverse=True), x, atol=1e-14)


def test_oracle_cache_attends_like_plain_attention():
    rng = np.random.default_rng(2)
    lens, cu = [37, 20], [0, 5, 6]
    table = np.array([[3, 0, 1], [2, 5, 9]])
    codes = [rng.integers(0, 100, (6, 2, 16, 8)) for _ in range(2)]
    scale = [2.0 ** rng.integers(-8, -4, (6, 2)) for _ in range(2)]
    c = C.Cache(*codes, *scale, table)
    q = rng.standard_normal((6, 4, 8))
    o, lse, _, _ = c.attend(q, cu, lens)
    w, _ = c.weights(q, lse, cu, lens)
    assert np.allclose(w[0].sum(), 5 * 4) and np.allclose(w[1].sum(), 4)
    t, h = 3, 3  # token 3 of 5 stands at position 35
    K = np.array([codes[0][table[0, j // 16], 1, j % 16] for j in range(36)])
    K = C.E4M3[K] * np.array([scale[0][table[0, j // 16], 1] for j in range(36)])[:, None]
    V = C.E4M3[np.array([codes[1][table[0, j // 16], 1, j % 16] for j in range(36)])]
    V = V * np.array([scale[1][table[0, j // 16], 1] for j in range(36)])[:, None]
    s = K @ q[t, h] / np.sqrt(8)
    p = np.exp(s)
    assert np.allclose(o[t, h], p @ V / p.sum()) and np.allclose(lse[h, t], np.log(p.sum()))
