"""The rotated append where its parts have to agree (batches in which good sequences
stand behind bad ones), and from several host threads."""
import numpy as np
import pytest
import torch

from block_sparse_masked_mask_gb300 import api
from test_cache_gpu import Pair, dev, randn

pytestmark = pytest.mark.gpu

STATE = ("k_pages", "v_pages", "k_scale", "v_scale")


@pytest.mark.parametrize("given", [False, True], ids=["by_length", "positions"])
@pytest.mark.parametrize("rot,inter", [(64, False), (20, False), (48, True), (6, True)])
@pytest.mark.parametrize("cu,T", [
    ([0, 3, 100, 8, 12], 12), ([0, 3, -5, 8, 12], 12), ([5, 3, 100, 8, 12], 12), ([0, 3, 2 ** 31 - 1, -2 ** 31, 8, 12], 15),
    (list(range(40)) + [1000] + list(range(40, 70)) + [0], 75), ([200] * 90 + [60, 64], 64)], ids=lambda x: str(x)[:40])
def test_queries_and_keys_of_the_same_sequences(cu, T, rot, inter, given):
    """Every sequence whose own numbers hold has its queries turned and its keys and values stored, as in a call of
    its own; of the others, and of rows of no sequence, nothing is written."""
    dim, heads, held = 64, 2, 30
    n = [b - a for a, b in zip(cu, cu[1:])]
    good = [i for i, x in enumerate(n) if 0 <= cu[i] and 0 < x and cu[i + 1] <= T and (i > 0 or cu[0] == 0)]
    assert good and all(cu[a + 1] <= cu[b] for a, b in zip(good, good[1:]))
    lens = [x + held if i in good else held for i, x in enumerate(n)]
    q, k, v = (randn(T, h, dim, seed=h + 1).cuda() for h in (5, heads, heads))
    plan = api.attn_rope_plan(rot, interleaved=inter)
    positions = dev(np.random.default_rng(1).integers(0, 9999, T)) if given else None
    all_, own = (Pair([64] * len(n), heads, dim, 16, seed=3) for _ in range(2))
    got = torch.full_like(q, 5)
    api.attn_cache_append_rope(q, k, v, plan, all_.dev, dev(cu), dev(lens), T, positions=positions, q_out=got)
    assert api.attn_cache_get_status(all_.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT
    want = torch.full_like(q, 5)
    d = own.dev
    for i in good:
        rows = slice(cu[i], cu[i + 1])
        one = api.KVCache(d.k_pages, d.v_pages, d.k_scale, d.v_scale, d.page_table[i:i + 1].contiguous())
        want[rows] = api.attn_cache_append_rope(q[rows], k[rows], v[rows], plan, one, dev([0, n[i]]), dev([lens[i]]), n[i],
                                                positions=positions[rows].clone() if given else None)
        assert api.attn_cache_get_status(one) == api.ATTN_OK
    assert torch.equal(got, want)
    for name in STATE:
        assert torch.equal(getattr(all_.dev, name), getattr(d, name)), name
    # in place, the rows of the others stay as they are
    again = q.clone()
    api.attn_cache_append_rope(again, k, v, plan, all_.dev, dev(cu), dev(lens), T, positions=positions, q_out=again)
    mine = torch.zeros(T, dtype=torch.bool)
    for i in good:
        mine[cu[i]:cu[i + 1]] = True
    assert torch.equal(again[mine], want[mine]) and torch.equal(again[~mine], q[~mine])


def test_host_threads_of_very_different_calls():
    """Calls of one kernel from several host threads, each on a stream and a cache of its own, that ask for very
    different amounts of shared memory: none is refused, and all store what a call alone stores."""
    import ctypes
    import threading

    from block_sparse_masked_mask_gb300 import _native
    plan, heads, dim, ps = api.attn_rope_plan(128), 2, 128, 128
    fn, sides = _native.lib().attn_cache_append_rope, []
    for n in (1, 128, 20):
        stream, p = torch.cuda.Stream(), Pair([n], heads, dim, ps, seed=n)
        q, k, v = (randn(n, h, dim, seed=h).cuda() for h in (4, heads, heads))
        x = dict(n=n, p=p, q=q, k=k, v=v, cu=dev([0, n]), lens=dev([n]), out=torch.empty_like(q), stream=stream, bad=[])
        x["want"] = api.attn_cache_append_rope(q, k, v, plan, p.dev, x["cu"], x["lens"], n)
        x["state"] = [getattr(p.dev, name).clone() for name in STATE]
        x["args"] = (q.data_ptr(), x["out"].data_ptr(), 4 * dim, 4 * dim, 4, k.data_ptr(), v.data_ptr(), heads * dim, heads * dim, 0, n,
                     None, x["cu"].data_ptr(), x["lens"].data_ptr(), n, ctypes.byref(plan.struct), p.dev._ref, stream.cuda_stream)
        sides.append(x)
    torch.cuda.synchronize()
    start = threading.Barrier(len(sides))

    def calls(x):
        start.wait()
        for i in range(6000):
            status = fn(*x["args"])
            if status != api.ATTN_OK:
                x["bad"].append((i, status))
            if i % 64 == 63:
                x["stream"].synchronize()

    threads = [threading.Thread(target=calls, args=(x,)) for x in sides]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for x in sides:
        assert not x["bad"], (x["n"], len(x["bad"]), x["bad"][0])
        assert torch.equal(x["out"], x["want"]) and api.attn_cache_get_status(x["p"].dev) == api.ATTN_OK
        assert all(torch.equal(getattr(x["p"].dev, name), y) for name, y in zip(STATE, x["state"]))
