"""README's step of speculative decoding over a model's layers, run as it stands there."""
import os
import re
import types

import numpy as np
import pytest

from conftest import ROOT


def step():
    text = open(os.path.join(ROOT, "README.md")).read()
    return re.search(r"### Drafted trees\n.*?```python\n(.*?)```", text, re.S).group(1)


def names(**kw):
    """What the example takes as given, with numbers in the place of tensors."""
    given = dict(caches=["A", "B", "C"], cache="A", parents="parents", cu="cu", lens="lens", max_new=4, max_seqlen=9, plan="plan",
                 x="x", q="q", k="k", v="v", path="path", counts="counts", project=lambda layer, x: ("q", "k", "v"),
                 rest=lambda layer, x, o: x, accept=lambda x: ("path", "counts"))
    return dict(given, **kw)


def test_every_layer_moves_by_the_lengths_as_they_were():
    calls = []

    def record(name, result):
        def call(*args, **kw):
            calls.append((name, args))
            return result
        return call
    api = types.SimpleNamespace(attn_cache_tree_build=record("build", ("bits", "positions")), attn_cache_append_rope=record("append", "q"),
                                attn_cache_tree_fwd=record("fwd", ("o", "lse")), attn_cache_tree_keep=record("keep", "shorter"))
    space = names(api=api)
    exec(step(), space)
    for name in ("append", "fwd", "keep"):
        of = [args for n, args in calls if n == name]
        assert [next(x for x in args if x in ("A", "B", "C")) for args in of] == ["A", "B", "C"], name
        assert all("lens" in args and "shorter" not in args for args in of), name
    assert sum(n == "build" for n, _ in calls) == 1 and space["lens"] == "shorter"


@pytest.mark.gpu
def test_the_step_over_two_layers():
    """Two steps behind one another: every layer's cache holds what the oracle's does, the path moved together."""
    import torch

    from block_sparse_masked_mask_gb300 import api
    from oracle import tree as R
    from test_cache_gpu import cu_of, dev, filled, randn
    from test_tree_gpu import check_tree, mirror, random_parents
    text, n, heads, dim = np.array([70, 33, 64]), np.array([9, 14, 5]), 2, 64
    rng = np.random.default_rng(1)
    pairs = [filled(list(text + 40), heads, dim, 32, seed=7 * i) for i in range(2)]
    plan, cu = api.attn_rope_plan(dim), cu_of(n)
    for turn in range(2):
        lens = text + n
        parents = [random_parents(int(x), rng) for x in n]
        masks = [R.ancestors(x) for x in parents]
        paths = [np.flatnonzero(m[m.sum(1).argmax()]).tolist() for m in masks]
        path = np.zeros((3, max(map(len, paths))), np.int32)
        for b, x in enumerate(paths):
            path[b, :len(x)] = x
        qkv = [[randn(int(n.sum()), h, dim, seed=10 * turn + 3 * i + j).cuda() for j, h in enumerate((4, heads, heads))] for i in range(2)]
        seen = []

        def rest(layer, x, o):
            p = pairs[layer]
            mirror(p)  # (its rotated keys have tests of their own)
            seen.append((layer, o.clone(), check_tree(p, space["q"].cpu(), cu, lens, masks)[0]))
            return x
        space = names(api=api, caches=[p.dev for p in pairs], parents=dev(sum(parents, [])), cu=dev(cu), lens=dev(lens), max_new=14,
                      max_seqlen=int(lens.max()), plan=plan, project=lambda layer, x: qkv[layer], rest=rest,
                      accept=lambda x: (dev(path), dev([len(x) for x in paths])))
        exec(step(), space)
        assert [s[0] for s in seen] == [0, 1] and all(torch.equal(o, want) for _, o, want in seen)
        for p in pairs:
            kept = R.keep(p.ref, paths, cu, lens)
            p.check_codes()
            assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
        assert space["lens"].tolist() == kept.tolist()
        text = kept
