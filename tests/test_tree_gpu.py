"""Trees of drafted tokens on the GPU against the fp64 oracle: masks, positions, kept
codes and scales have to be equal; attention has the bounds of test_cache_gpu
(attend_bounds), rotated keys those written beside their test."""
import math

import numpy as np
import pytest
import torch

from block_sparse_masked_mask_gb300 import api
from oracle import cache as C
from oracle import tree as R
from test_cache_gpu import Pair, attend_bounds, cu_of, dev, filled, randn

pytestmark = pytest.mark.gpu


def random_parents(n, rng, reach=None):
    """Every node on one of those before it (at most `reach` back), or on none."""
    return [int(rng.integers(max(-1, -1 if reach is None else i - reach), i)) for i in range(n)]


TREES = {
    "random": lambda n, rng: random_parents(n, rng),
    "chain": lambda n, rng: list(range(-1, n - 1)),
    "star": lambda n, rng: [-1] * n,
    "deep": lambda n, rng: random_parents(n, rng, 3),
}


def device_bits(bits):
    return torch.from_numpy(bits.view(np.int32)).cuda()


# ------------------------------------------------------------------ masks and positions

@pytest.mark.parametrize("shape", TREES)
@pytest.mark.parametrize("n", [[1], [3, 0, 33, 32, 64, 31], [65, 200, 7], [1030, 5]], ids=str)
def test_build(n, shape):
    rng = np.random.default_rng(len(n))
    held = [17 * i for i in range(len(n))]
    lens, cu = [a + b for a, b in zip(held, n)], cu_of(n)
    p = Pair(lens, 1, 32, 128, seed=1)
    parents = [TREES[shape](x, rng) for x in n]
    T, words = int(cu[-1]), -(-max(n) // 32)
    flat = torch.tensor(sum(parents, []) + [7, -9], dtype=torch.int32, device="cuda")  # two rows behind the last
    seen = [R.ancestors(x) for x in parents]
    for more in (0, 2):
        bits = torch.full((T + 2, words + more), -5, dtype=torch.int32, device="cuda")
        positions = torch.full((T + 2,), -5, dtype=torch.int32, device="cuda")
        got = api.attn_cache_tree_build(flat, p.dev, dev(cu), dev(lens), max(n) + 31 * (more > 0), bits=bits, positions=positions)
        assert got[0] is bits and got[1] is positions and api.attn_cache_get_status(p.dev) == api.ATTN_OK
        assert np.array_equal(bits.cpu().numpy().view(np.uint32)[:T], R.to_bits(seen, words + more))
        want = np.concatenate([h + s.sum(1) - 1 for h, s in zip(held, seen)])
        assert np.array_equal(positions.cpu().numpy()[:T], want)
        assert (bits[T:] == -5).all() and (positions[T:] == -5).all()


@pytest.mark.parametrize("bad", [[0, 0], [-2, 0], [-1, 1], [-1, 5], [-1, 2 ** 30]], ids=str)
def test_build_leaves_out_a_sequence_of_wrong_parents(bad):
    p = Pair([10, 10, 10], 1, 32, 16, seed=1)
    flat = torch.tensor([-1] + bad + [-1, 0], dtype=torch.int32, device="cuda")
    bits = torch.full((5, 1), 99, dtype=torch.int32, device="cuda")
    positions = torch.full((5,), 99, dtype=torch.int32, device="cuda")
    api.attn_cache_tree_build(flat, p.dev, dev([0, 1, 3, 5]), dev([10, 10, 10]), 2, bits=bits, positions=positions)
    assert bits[:, 0].tolist() == [1, 99, 99, 1, 3] and positions.tolist() == [9, 99, 99, 8, 9]
    assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK


# ------------------------------------------------------------------ rotation on the way into the cache

CASES = [(128, 128, False, "none"), (128, 50, False, "linear"), (64, 64, True, "ramp"), (32, 6, True, "ntk"),
         (128, 24, False, "none"), (64, 16, False, "none"), (128, 10, True, "none"), (32, 2, False, "none")]


def partners(x, rot, inter):
    """|x| + |its partner| of the rotated dimensions, 0 of the others, which are copied."""
    x = np.abs(x)
    y = np.zeros_like(x)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    if inter:
        y[..., 0:rot:2], y[..., 1:rot:2] = a + b, a + b
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = a + b, a + b
    return y


def check_cached_near(p, exact, off, v, cu, lens):
    """The whole cache against the oracle, in which the exact numbers were appended.  New keys were
    turned in fp32 and are off by `off`: a code is the nearest one of such a value, so off by half a
    step (2^-4 of itself, or 2^-10 of the scale where it is subnormal) and that.  A page's
    scale can be another only where its largest lies within `off` of a border, 448 2^e."""
    ps, table = p.dev.page_size, p.table
    fresh, near = np.zeros(p.ref.codes[0].shape[:3], bool), np.zeros(p.ref.codes[0].shape[:2], bool)
    want, slack = np.zeros(p.ref.codes[0].shape), np.zeros(p.ref.codes[0].shape)
    for b, t in enumerate(lens):
        n = cu[b + 1] - cu[b]
        for i in range((t - n) // ps, -(-t // ps) if n else 0):
            lo, hi = max(t - n, i * ps), min(t, (i + 1) * ps)
            rows, slots, page = slice(cu[b] + lo - (t - n), cu[b] + hi - (t - n)), slice(lo - i * ps, hi - i * ps), table[b, i]
            fresh[page, :, slots] = True
            want[page, :, slots], slack[page, :, slots] = exact[rows].transpose(1, 0, 2), off[rows].transpose(1, 0, 2)
            low, high = (np.abs(exact[rows]) - off[rows]).max((0, 2)), (np.abs(exact[rows]) + off[rows]).max((0, 2))
            near[page] = [C.scale_for(x) != C.scale_for(y) for x, y in zip(low, high)]
    p.ref.append(exact, v, cu, lens)
    codes, scale = p.dev.k_pages.cpu().numpy(), p.dev.k_scale.cpu().double().numpy()
    assert near.sum() <= 2
    assert np.array_equal(scale[~near], p.ref.scale[0][~near])
    old = ~fresh & ~near[:, :, None]
    assert np.array_equal(codes[old], p.ref.codes[0][old])
    with np.errstate(invalid="ignore"):  # (NaN codes of slots that hold nothing)
        step = np.maximum(2.0 ** -4 * (np.abs(want) + slack), 2.0 ** -10 * scale[..., None, None])
        assert (np.abs(C.e4m3_decode(codes) * scale[..., None, None] - want)[fresh] <= (step + slack)[fresh]).all()
    assert np.array_equal(p.dev.v_pages.cpu().numpy(), p.ref.codes[1])
    assert np.array_equal(p.dev.v_scale.cpu().double().numpy(), p.ref.scale[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("given", [False, True], ids=["by_length", "positions"])
@pytest.mark.parametrize("dim,rot,inter,scaling", CASES)
def test_append_rope(dim, rot, inter, scaling, given, dtype):
    """Queries and the whole cache against the oracle.  A turned element x cos - y sin is off by the
    rounding of one product and of the result, by its sine's and cosine's (2 ulp, 2^-22, each, and 2^-24 of the
    factor) and by the angle's 2^-33 turns (2^-30): 2^-21 (|x| + |y|) at most, times the
    factor, which is below 2; a query is then rounded to its type, by half a step."""
    heads, group = 3, 2
    n, held = [40, 1, 0, 130, 17], [0, 63, 5, 70, 200]
    lens, cu, T = [a + b for a, b in zip(n, held)], cu_of(n), sum(n)
    for page_size in (16, 32, 64, 128):
        p = Pair(lens, heads, dim, page_size, seed=3)
        kw = dict(scaling=scaling, factor=4.0, original_context=4096.0) if scaling != "none" else {}
        plan = api.attn_rope_plan(rot, interleaved=inter, **kw)
        q, k, v = (randn(T, h, dim, seed=i, dtype=dtype, scale=1.5) for i, h in enumerate((heads * group, heads, heads)))
        at = np.concatenate([np.arange(t - x, t) for t, x in zip(lens, n)])
        if given:
            at = np.random.default_rng(1).integers(-5, 1 << 20, T)
        got = api.attn_cache_append_rope(q.cuda(), k.cuda(), v.cuda(), plan, p.dev, dev(cu), dev(lens), max(n),
                                         positions=dev(at) if given else None)
        assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
        # angles as the plan has them: 64-bit fractions of a turn (their own test is test_rope_plan_numbers)
        theta = np.array([plan.struct.turn[i] for i in range(rot // 2)], np.float64) / 2.0 ** 64
        turns = np.array([[(int(x) * int(plan.struct.turn[i])) % 2 ** 64 / 2.0 ** 64 for i in range(rot // 2)] for x in at])
        m = plan.struct.result_factor
        exact, off = [], []
        for x in (q.double().numpy(), k.double().numpy()):
            y = x.copy()
            a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
            z = (a + 1j * b) * (m * np.exp(2j * np.pi * turns))[:, None, :]
            if inter:
                y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
            else:
                y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
            exact.append(y)
            off.append(2.0 ** -20 * partners(x, rot, inter))
        half = torch.finfo(dtype).eps / 2
        err = np.abs(got.double().cpu().numpy() - exact[0])
        assert (err <= off[0] + half * (np.abs(exact[0]) + off[0])).all()
        assert theta.max() <= 1 / (2 * np.pi) * (1 + 2.0 ** -40)
        check_cached_near(p, exact[1], off[1], v.double().numpy(), cu, lens)


def test_append_rope_does_not_depend_on_how_rows_are_read():
    """The same codes and queries from fp32 as from the bf16 numbers that they are, and from any alignment of q."""
    n, held, heads, dim = [70, 9], [10, 100], 2, 64
    lens, cu, T = [a + b for a, b in zip(n, held)], cu_of(n), sum(n)
    for rot, inter in ((64, False), (20, False), (48, True), (6, True)):
        plan = api.attn_rope_plan(rot, interleaved=inter)
        q, k, v = (randn(T, h, dim, seed=i).cuda() for i, h in enumerate((4, heads, heads)))
        first = None
        for shift, dtype in ((0, torch.float32), (1, torch.float32), (2, torch.float32), (0, torch.bfloat16), (1, torch.bfloat16),
                             (2, torch.bfloat16), (4, torch.bfloat16)):
            p = Pair(lens, heads, dim, 32, seed=5)
            room = torch.zeros(T * 4 * dim + 8, dtype=dtype, device="cuda")[shift:shift + T * 4 * dim].view(T, 4, dim)
            room.copy_(q)
            got = api.attn_cache_append_rope(room, k.to(dtype), v.to(dtype), plan, p.dev, dev(cu), dev(lens), max(n))
            now = [p.dev.k_pages, p.dev.k_scale, p.dev.v_pages, p.dev.v_scale, got.to(torch.bfloat16)]
            first = now if first is None else first
            assert all(torch.equal(a, b) for a, b in zip(now, first)), (rot, inter, shift, dtype)


def test_append_rope_strided_in_place_and_rows_behind():
    """Slices of one projection, q rotated in place, rows of no sequence left as they are."""
    heads, group, dim, n, held = 2, 4, 64, [30, 9], [10, 100]
    lens, cu = [a + b for a, b in zip(n, held)], cu_of(n)
    one, two = (Pair(lens, heads, dim, 32, seed=5) for _ in range(2))
    plan = api.attn_rope_plan(dim)
    wide = randn(45, (heads * group + 2 * heads) * dim + 16, seed=3).cuda()
    part = lambda w, a, h: w[:, a * dim:(a + h) * dim].unflatten(1, (h, dim))  # noqa: E731
    before = wide.clone()
    q, k, v = part(wide, 0, 8), part(wide, 8, 2), part(wide, 10, 2)
    want = api.attn_cache_append_rope(q.contiguous(), k.contiguous(), v.contiguous(), plan, two.dev, dev(cu), dev(lens), 30,
                                      q_out=q.contiguous())
    assert api.attn_cache_append_rope(q, k, v, plan, one.dev, dev(cu), dev(lens), 30, q_out=q) is q
    assert torch.equal(q, want) and torch.equal(wide[:, 8 * dim:], before[:, 8 * dim:])
    assert torch.equal(wide[39:], before[39:]) and not torch.equal(q[:39], part(before, 0, 8)[:39])
    for name in ("k_pages", "k_scale", "v_pages", "v_scale"):
        assert torch.equal(getattr(one.dev, name), getattr(two.dev, name)), name
    # positions given: rows behind the last sequence have one too, and are left as well
    positions = torch.arange(45, dtype=torch.int32, device="cuda")
    out = torch.full((45, 8, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    api.attn_cache_append_rope(q, k, v, plan, one.dev, dev(cu), dev(lens), 30, positions=positions, q_out=out)
    assert (out[39:] == 3).all() and not (out[:39] == 3).all(2).all(1).any()
    assert api.attn_cache_get_status(one.dev) == api.ATTN_OK


# ------------------------------------------------------------------ attention

def check_tree(p, q, cu, lens, masks, scale=0.0, max_new=None, max_seqlen=None, words=None, **kw):
    n = int(np.diff(cu).max()) if max_new is None else max_new
    words = max(1, -(-n // 32)) if words is None else words
    T = int(cu[-1])
    bits = np.full((len(q), words), 0xDEADBEEF, np.uint32)
    bits[:T] = R.to_bits(masks, words)
    for b, m in enumerate(masks):  # bits of nodes that there are not are ignored
        for j in range(len(m), 32 * words):
            bits[cu[b]:cu[b + 1]:2, j // 32] |= np.uint32(1 << (j % 32))
    o, lse = api.attn_cache_tree_fwd(q.cuda(), p.dev, device_bits(bits), dev(cu), dev(lens), n,
                                     int(max(lens)) if max_seqlen is None else max_seqlen, scale=scale, **kw)
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
    q = q[:T]
    O, L, terms, spread = R.attend(p.ref, q.double().numpy(), cu, lens, masks, scale)
    tol, slack = attend_bounds(p.ref, O, spread, terms, cu, lens, q.shape[2])
    err = np.abs(o.double().cpu().numpy()[:T] - O)
    assert (err <= tol).all(), f"O: max err {err.max()}, worst ratio {(err / np.maximum(tol, 1e-300)).max()}"
    gl = lse.double().cpu().numpy()[:, :T]
    for b in range(len(lens)):
        s = slice(cu[b], cu[b + 1])
        seen = np.isfinite(L[:, s])
        assert np.array_equal(np.isneginf(gl[:, s]), ~seen)
        d = np.abs(gl[:, s][seen] - L[:, s][seen])
        assert (d <= slack[b] + 2.0 ** -22 * np.abs(L[:, s][seen])).all(), f"LSE: {d.max()} vs {slack[b]}"
    return o, lse


def trees(n, shape="random", seed=0):
    rng = np.random.default_rng(seed)
    return [R.ancestors(TREES[shape](x, rng)) for x in n]


@pytest.mark.parametrize("shape", TREES)
@pytest.mark.parametrize("dim,page_size,heads,group", [(128, 64, 2, 4), (64, 16, 1, 8), (32, 128, 3, 1), (128, 32, 1, 16),
                                                       (64, 128, 2, 5), (32, 16, 2, 3)])
def test_ragged_trees(dim, page_size, heads, group, shape):
    """Trees of one node to some, none, texts from none to several tiles, pages that end inside."""
    n, held = [5, 16, 1, 0, 33, 7, 20], [700, 0, 129, 50, 95, 1, 128]
    lens, cu = [a + b for a, b in zip(n, held)], cu_of(n)
    p = filled(lens, heads, dim, page_size, seed=dim + group)
    check_tree(p, randn(int(cu[-1]), heads * group, dim, seed=6), cu, lens, trees(n, shape))


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129, 200, 256, 257, 300, 513])
def test_numbers_of_rows(rows):
    """Every number of nodes around the sizes of tiles, one query head each."""
    n = [rows, max(1, rows - 3)]
    lens, cu = [rows + 260, n[1] + 31], cu_of(n)
    p = filled(lens, 1, 64, 32, seed=rows)
    check_tree(p, randn(sum(n), 1, 64, seed=rows), cu, lens, trees(n))


@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("n,group", [(4, 4), (8, 4), (16, 4), (32, 4), (33, 4), (64, 8), (1, 1), (1, 5)])
def test_lengths_around_tiles(n, group, dim):
    lens = [n + x for x in (0, 1, 15, 16, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000)]
    cu = cu_of([n] * len(lens))
    p = filled(lens, 1, dim, 16, seed=n)
    check_tree(p, randn(n * len(lens), group, dim, seed=n), cu, lens, trees([n] * len(lens)))


def test_masks_that_are_no_trees():
    """Any bits: nodes that see later ones, that do not see themselves, that see nothing at
    all (an empty row where there is no text)."""
    rng = np.random.default_rng(1)
    n, held = [40, 9, 70, 3], [0, 200, 64, 0]
    masks = [rng.random((x, x)) < 0.3 for x in n]
    masks[0][5] = False
    masks[0][39] = False
    masks[1][:] = False
    masks[3][:] = False
    lens, cu = [a + b for a, b in zip(n, held)], cu_of(n)
    for group, dim in ((1, 64), (4, 128)):
        p = filled(lens, 2, dim, 32, seed=2)
        o, lse = check_tree(p, randn(sum(n), 2 * group, dim, seed=4), cu, lens, masks)
        assert (o[5] == 0).all() and torch.isneginf(lse[:, 5]).all() and (o[-3:] == 0).all()


def test_a_chain_is_causal_attention():
    n, lens = [17, 40], [400, 40]
    cu = cu_of(n)
    p = filled(lens, 2, 64, 32, seed=3)
    q = randn(57, 4, 64, seed=5)
    O, L, _, _ = p.ref.attend(q.double().numpy(), cu, lens)
    o, _, _, _ = R.attend(p.ref, q.double().numpy(), cu, lens, trees(n, "chain"))
    assert np.abs(O - o).max() < 1e-12
    check_tree(p, q, cu, lens, trees(n, "chain"))


@pytest.mark.parametrize("n,heads,group,lens", [(8, 1, 4, [9001]), (12, 2, 1, [12000, 40]), (64, 1, 8, [6000, 9000]),
                                               (4, 8, 4, [5000] * 3), (1, 4, 8, [7000]), (32, 2, 4, [3000, 1, 4095])])
def test_long_texts(n, heads, group, lens):
    """One sequence over many CTAs, and their joins."""
    k = [min(n, x) for x in lens]
    p = filled(lens, heads, 64, 64, seed=n)
    check_tree(p, randn(sum(k), heads * group, 64, seed=n), cu_of(k), lens, trees(k))


def test_many_sequences():
    """More (sequence, head)s than SMs, of very different lengths, some without nodes."""
    n = [(7 * i) % 23 if i % 7 else 0 for i in range(90)]
    lens = [x + (97 * i) % 900 for i, x in enumerate(n)]
    p = filled(lens, 4, 64, 32, seed=9)
    check_tree(p, randn(sum(n), 8, 64, seed=3), cu_of(n), lens, trees(n))


def test_rows_behind_the_last_sequence_and_wide_bounds():
    n, lens = [3, 2], [100, 40]
    p = filled(lens, 1, 128, 64, seed=41)
    q = randn(9, 4, 128, seed=8)
    q[5:] = float("nan")
    for max_new, words in ((9, 1), (9, 4), (300, 10)):
        o, lse = torch.full((9, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, 9), 5.0, device="cuda")
        check_tree(p, q, cu_of(n), lens, trees(n), max_new=max_new, max_seqlen=128, words=words, out=o, lse=lse)
        assert (o[5:] == 5).all() and (lse[:, 5:] == 5).all()


def test_large_scores_and_scales():
    lens, n = [333, 80], [6, 20]
    p = filled(lens, 2, 64, 32, seed=33)
    for size, scale in ((60.0, 0.0), (1.0, 3.0), (1e-30, 0.0), (1e30, 1e-30)):
        check_tree(p, randn(26, 4, 64, seed=7, scale=size), cu_of(n), lens, trees(n), scale=scale)


# ------------------------------------------------------------------ the path

@pytest.mark.parametrize("page_size,dim", [(16, 64), (32, 128), (64, 32), (128, 128), (128, 64), (16, 32)])
def test_keep(page_size, dim):
    """Paths of none, of all and of some nodes, over several pages whose scales differ."""
    rng = np.random.default_rng(page_size)
    n, held = [40, 7, 0, 64, 200, 5, 33, 1], [100, 0, 30, 64, 17, 60, 15, 128]
    lens, cu = [a + b for a, b in zip(n, held)], cu_of(n)
    p = filled(lens, 3, dim, page_size, seed=7)
    counts = [9, 7, 0, 1, 70, 0, 20, 1]
    paths = [sorted(rng.choice(x, c, replace=False).tolist()) for x, c in zip(n, counts)]
    path = np.full((len(n), 80), 1 << 28, np.int32)
    for b, x in enumerate(paths):
        path[b, :len(x)] = x
    got = api.attn_cache_tree_keep(dev(path), dev(counts), p.dev, dev(cu), dev(lens), 200)
    want = R.keep(p.ref, paths, cu, lens)
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
    assert got.tolist() == want.tolist()
    p.check_codes()


@pytest.mark.parametrize("path,count", [([3, 2], 2), ([2, 2], 2), ([-1, 0], 2), ([0, 8], 2), ([0, 1], -1), ([0, 1], 3)], ids=str)
def test_keep_leaves_out_a_sequence_of_a_wrong_path(path, count):
    p = filled([30, 30], 2, 64, 16, seed=1)
    new = torch.full((2,), 99, dtype=torch.int32, device="cuda")
    api.attn_cache_tree_keep(dev([path, [1, 3]]), dev([count, 2]), p.dev, dev([0, 8, 16]), dev([30, 30]), 8, new_lens=new)
    assert api.attn_cache_get_status(p.dev) == api.ATTN_ERR_DEVICE_INVALID_INPUT
    q = C.Cache(*p.ref.codes, *p.ref.scale, p.table[1:])
    R.keep(q, [[1, 3]], [0, 8], [30])
    p.ref = q
    p.check_codes()
    assert new.tolist() == [99, 24]


# ------------------------------------------------------------------ together

def test_a_step_of_speculative_decoding():
    """Prompt, then twice: a drafted tree (build -> append_rope -> tree_fwd), its path
    kept, and at last a plain step of one token, each against the oracle."""
    heads, group, dim, ps = 2, 3, 64, 32
    rng = np.random.default_rng(3)
    prompt, most = np.array([37, 64, 1]), 60
    p = Pair(list(prompt + most), heads, dim, ps, seed=61)
    plan = api.attn_rope_plan(dim, interleaved=True)
    text = prompt.copy()
    cu = cu_of(text)
    q, k, v = (randn(int(cu[-1]), h, dim, seed=i).cuda() for i, h in enumerate((heads * group, heads, heads)))
    api.attn_cache_append_rope(q, k, v, plan, p.dev, dev(cu), dev(text), int(max(text)))
    mirror(p)
    for step in range(2):
        n = np.array([13, 20, 6])
        parents = [random_parents(int(x), rng) for x in n]
        masks = [R.ancestors(x) for x in parents]
        cu, lens, T = cu_of(n), text + n, int(n.sum())
        q, k, v = (randn(T, h, dim, seed=10 * step + 5 + i).cuda() for i, h in enumerate((heads * group, heads, heads)))
        bits, positions = api.attn_cache_tree_build(dev(sum(parents, [])), p.dev, dev(cu), dev(lens), int(n.max()))
        turned = api.attn_cache_append_rope(q, k, v, plan, p.dev, dev(cu), dev(lens), int(n.max()), positions=positions)
        want, _ = api.attn_rope(q, None, plan, positions=positions)  # (a rounding of fp32 may be another: one step of bf16)
        assert ((turned.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -20).all()
        mirror(p)
        check_tree(p, turned.cpu(), cu, lens, masks)
        # the longest path of each tree
        paths = [np.flatnonzero(m[m.sum(1).argmax()]).tolist() for m in masks]
        path = np.zeros((3, max(map(len, paths))), np.int32)
        for b, x in enumerate(paths):
            path[b, :len(x)] = x
        new = api.attn_cache_tree_keep(dev(path), dev([len(x) for x in paths]), p.dev, dev(cu), dev(lens), int(n.max()))
        text = R.keep(p.ref, paths, cu, lens)
        p.check_codes()
        assert new.tolist() == text.tolist() and api.attn_cache_get_status(p.dev) == api.ATTN_OK
    lens = text + 1
    q, k, v = (randn(3, h, dim, seed=90 + i).cuda() for i, h in enumerate((heads * group, heads, heads)))
    turned = api.attn_cache_append_rope(q, k, v, plan, p.dev, dev([0, 1, 2, 3]), dev(lens), 1)
    mirror(p)
    check_tree(p, turned.cpu(), cu_of([1, 1, 1]), lens, trees([1, 1, 1]))


def mirror(p):
    """The oracle's cache takes what the device's holds (its rotated keys have tests of their own)."""
    p.ref.codes = [p.dev.k_pages.cpu().numpy().copy(), p.dev.v_pages.cpu().numpy().copy()]
    p.ref.scale = [p.dev.k_scale.cpu().double().numpy(), p.dev.v_scale.cpu().double().numpy()]
