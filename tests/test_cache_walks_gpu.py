"""The cache and rotary kernels in the steady state of their walks: queues, rings and look-ups
ahead that turn many times, joins of many pieces, keys that no longer fit shared
memory.  Sequences share read-only pages, so that a long line of tokens needs little
memory.  Bounds are those of test_cache_gpu and test_cache_edges_gpu."""
import numpy as np
import pytest
import torch

from block_sparse_masked_mask_gb300 import api
from oracle import cache as C
from test_cache_gpu import Pair, check_attend, cu_of, dev, filled, randn
from test_rope_gpu import check as check_rotation, rows

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def shared(lens, heads, dim, page_size, pages=150, seed=0):
    """Sequences over random pages of one pool of appended tokens."""
    p = filled([pages * page_size], heads, dim, page_size, seed=seed, spread=False)
    rng = np.random.default_rng(seed)
    pool = p.table[0, :pages]
    p.table = pool[rng.integers(0, pages, (len(lens), -(-max(lens) // page_size)))].astype(np.int32)
    p.ref.table = p.table
    d = p.dev
    p.dev = api.KVCache(d.k_pages, d.v_pages, d.k_scale, d.v_scale, dev(p.table))
    return p


def lengths(n, low, high, seed):
    return [int(x) for x in np.random.default_rng(seed).integers(low, high, n)]


def check_weights(p, q, cu, lens, lse, causal=True):
    """test_weights_of_many_rows' bound: with more than 24 rows scale 2^-17 m sum |k| more."""
    heads, dim = p.dev.num_kv_heads, q.shape[2]
    group, most = q.shape[1] // heads, int(np.diff(cu).max())
    before = torch.rand((len(lens), heads, max(lens) + 1), generator=torch.Generator().manual_seed(2))
    got = api.attn_cache_weights(q.cuda(), lse, p.dev, dev(cu), dev(lens), most, max(lens), prev=before.cuda(),
                                 out=torch.full(before.shape, 3.0, device="cuda"), kind="causal" if causal else "none")
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
    got = got.cpu()
    ref, terms = p.ref.weights(q.double().numpy(), lse.cpu().numpy(), cu, lens, causal)
    for b, L in enumerate(lens):
        A, rows = terms[b].max(initial=0), (cu[b + 1] - cu[b]) * group
        m = np.abs(q[cu[b]:cu[b + 1]].double().numpy()).max(initial=0)
        off = 2.0 ** (-17 if most * group > 24 else -25) * m * np.abs(p.ref.numbers(0, b, L)).sum(-1).max() / np.sqrt(dim)
        rel = 2 * (dim + 4) * 2.0 ** -24 * A + 2.0 ** -22 + 2.0 ** -22 * (2 * A + 16) + rows * 2.0 ** -24
        w = before[b, :, :L].double().numpy()
        err = np.abs(got[b, :, :L].double().numpy() - (w + ref[b]))
        tol = (rel + np.expm1(off)) * ref[b] + (-(-rows // 128) + 1) * 2.0 ** -24 * (w + ref[b]) + 1e-37
        assert (err <= tol).all(), f"sequence {b}: worst ratio {(err / tol).max()}"
        assert (got[b, :, L:] == 3).all()


@pytest.mark.parametrize("new,group,seqs", [(1, 2, 64), (1, 16, 40), (8, 3, 40), (40, 1, 30), (70, 2, 24), (150, 2, 24)])
def test_long_pieces_of_the_line(new, group, seqs):
    """Decode steps, drafts and chunks over a line of tokens that gives every CTA
    thousands: attention (queue of groups, pages 32 groups at a time; tiles and their
    rings) and weights (blocks, pages 16 at a time; rings of three and eight tiles)."""
    lens = lengths(seqs, 5600, 6500, seqs + new)
    p = shared(lens, 8, 32, 32, seed=new)
    # per CTA: 3 and 4 per SM of the kernels of few rows, 2 per SM of the weights of many
    assert sum(lens) * 8 / (4 * sms()) > 4 * 16 * 32 or new * group > 24
    assert sum(lens) * 8 / (2 * sms()) > 24 * 128
    cu = cu_of([new] * seqs)
    q = randn(int(cu[-1]), 8 * group, 32, seed=3)
    _, lse = check_attend(p, q, cu, lens)
    check_weights(p, q, cu, lens, lse)


def test_wide_heads_on_the_line():
    """The same with D = 128 and 64, pages of 16 and 128 tokens."""
    for dim, page_size, new in ((128, 16, 1), (64, 128, 30)):
        lens = lengths(24, 5600, 6500, dim)
        p = shared(lens, 8, dim, page_size, pages=60, seed=dim)
        cu = cu_of([new] * 24)
        q = randn(24 * new, 16, dim, seed=5)
        _, lse = check_attend(p, q, cu, lens)
        check_weights(p, q, cu, lens, lse)


@pytest.mark.parametrize("others,new", [(0, 1), (0, 10), (64, 1), (64, 12), (0, 40), (3, 200)])
def test_joins_of_many_pieces(others, new):
    """One sequence of 65000 tokens alone and beside short ones: its results lie in
    hundreds of pieces (more than 32 per warp of the join)."""
    lens = [100] * others + [65000]
    p = shared(lens, 1, 32, 64, seed=new)
    cu = cu_of([new] * len(lens))
    check_attend(p, randn(int(cu[-1]), 1, 32, seed=6), cu, lens)


def check_evict(p, dst, w, lens, budgets, recent):
    """An eviction against its definition, the copies of each page all at once."""
    heads, ps = p.dev.num_kv_heads, p.dev.page_size
    keep = [min(a, b) for a, b in zip(lens, budgets)]
    kept, nw, nl = api.attn_cache_evict(w.cuda(), p.dev, dst.dev, dev(lens), dev(budgets), recent, max(lens), max(keep))
    assert api.attn_cache_get_status(p.dev) == api.ATTN_OK and nl.cpu().tolist() == keep
    kept, nw = kept.cpu().numpy(), nw.cpu().numpy()
    h = np.arange(heads)[:, None]
    for b, (L, n) in enumerate(zip(lens, keep)):
        tail = min(recent, n)
        best = np.argsort(-w[b, :, :L - tail].numpy(), axis=-1, kind="stable")[:, :n - tail]
        want = np.concatenate([np.sort(best, -1), np.broadcast_to(np.arange(L - tail, L), (heads, tail))], 1)
        assert np.array_equal(kept[b, :, :n], want) and (kept[b, :, n:] == -1).all()
        assert np.array_equal(nw[b, :, :n], np.take_along_axis(w[b].numpy(), want, 1)) and (nw[b, :, n:] == 0).all()
        pages = p.table[b][want // ps]                      # [heads, n]
        for side in (0, 1):
            codes = p.ref.codes[side][pages, h, want % ps]  # [heads, n, dim]
            unit = p.ref.scale[side][pages, h]
            for i in range(-(-n // ps)):
                part = slice(i * ps, min(n, (i + 1) * ps))
                top, to = unit[:, part].max(1), dst.table[b, i]
                x = C.e4m3_decode(codes[:, part]) * (unit[:, part] / top[:, None])[..., None]
                dst.ref.scale[side][to] = top
                dst.ref.codes[side][to, :, :x.shape[1]] = C.e4m3_encode(x)
    dst.check_codes()


@pytest.mark.parametrize("recent", [0, 300, 11000])
@pytest.mark.parametrize("length", [49151, 49152, 49153, 60000])
def test_evict_more_tokens_than_keys_fit(length, recent):
    """Keys behind the 49152 that shared memory holds are read again.  Few distinct
    weights, so that ties at the border lie on both sides, and many different ones."""
    p = filled([length, 700], 1, 32, 64, seed=1)
    g = torch.Generator().manual_seed(recent)
    few = torch.randint(0, 5, (2, 1, length), generator=g).float()
    spread = torch.randn((2, 1, length), generator=g)
    spread[..., ::7] = float("-inf")
    for w, keep in ((few, length // 2), (few, length - 5), (spread, 12000)):
        budgets = [keep, 600]
        check_evict(p, Pair(budgets, 1, 32, 64, seed=2), w, [length, 700], budgets, recent)


@pytest.mark.parametrize("dim,page_size", [(32, 16), (128, 16), (64, 32)])
def test_evict_copies_page_after_page(dim, page_size):
    """Several pages per copying CTA; ragged last pages, sequences that keep nothing."""
    heads, seqs = 8, 96
    lens = lengths(seqs, 600, 1500, dim)
    budgets = [0 if b % 11 == 0 else int(L * 0.9) for b, L in enumerate(lens)]
    if page_size == 16:
        assert sum(-(-n // page_size) for n in budgets) * heads > 3 * 64 * sms()
    p = shared(lens, heads, dim, page_size, seed=3)
    # scales of pages far enough apart that codes are rounded again
    scale = 2.0 ** np.random.default_rng(4).integers(-6, 7, p.ref.scale[0].shape).astype(np.float64)
    for buf, side in ((p.dev.k_scale, 0), (p.dev.v_scale, 1)):
        p.ref.scale[side] = np.roll(scale, side, 0)
        buf.copy_(torch.from_numpy(p.ref.scale[side].astype(np.float32)))
    w = torch.rand((seqs, heads, max(lens)), generator=torch.Generator().manual_seed(6))
    check_evict(p, Pair(budgets, heads, dim, page_size, seed=5), w, lens, budgets, 50)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 52), (64, 62), (32, 16)])
def test_rotation_of_many_heads_by_one_warp(D, rot, interleaved, dtype):
    """Enough tokens that a warp takes all heads of one, several turns of its loads; the
    last turn ragged; in place too."""
    T, Hq, Hk = 32 * sms() + 37, 37, 4
    q, k = rows(T, Hq, D, dtype, 1), rows(T, Hk, D, dtype, 2)
    pos = torch.arange(T, dtype=torch.int32) * 13
    plan = api.attn_rope_plan(rot, interleaved=interleaved)
    yq, yk = api.attn_rope(q, k, plan, positions=pos.cuda())
    at = torch.randperm(T, generator=torch.Generator().manual_seed(3))[:150]
    at[0], at[1] = 0, T - 1
    for x, y in ((q, yq), (k, yk)):
        check_rotation(x[at.cuda()], y[at.cuda()], pos[at].numpy(), dict(rotary_dim=rot, interleaved=interleaved))
    want = yq.clone(), yk.clone()
    api.attn_rope(q, k, plan, positions=pos.cuda(), q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
