"""Measured cases of the operators that serve trees of drafted tokens over the 8-bit key/value cache: the
tree's ancestor masks and positions, new keys and values rotated on their way into the cache, attention of a
tree's nodes, and the accepted path moved together.

Every case is a dict of plain values; ``prepare`` makes its inputs from a seed, ``run`` makes one pass
(the framework's calls where ``own`` is true, elementary torch operations where it is not) and ``exact``
gives the same outputs from the definitions in 64 bits.  The cache's codes are returned as float8 numbers
next to their power-of-two scales.
"""
import math
import random

import torch

own = False

F8_MAX = 448.0          # largest finite e4m3 number
SCALE_EXP = (-80, 120)  # exponents a page's scale may take
FACTOR, CONTEXT, BASE, ALPHA, BETA = 8.0, 8192, 10000.0, 1.0, 32.0  # of the rotations


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # a step of 64 requests turns its drafted trees into masks and positions, once for all layers
        dict(name="tree_build_64", op="build", seqs=64, new_lo=16, new_hi=64, hk=8, d=128, page=64, lo=1024, hi=16384, lens=11),
        # a large batch of wide trees
        dict(name="tree_build_wide", op="build", seqs=512, new_lo=128, new_hi=256, hk=1, d=32, page=128, lo=64, hi=1024, lens=12),
        # a plain decode step of 64 requests: one token each is rotated and goes in
        dict(name="append_rope_decode_64", op="append", seqs=64, new_lo=1, new_hi=1, hq=32, hk=8, d=128, page=64, rot=128,
             interleaved=False, scaling="none", dtype="bf16", lo=1024, hi=16384, tree=False, lens=21),
        # the drafted trees of 32 requests, siblings at one position
        dict(name="append_rope_trees_32", op="append", seqs=32, new_lo=17, new_hi=64, hq=32, hk=8, d=128, page=64, rot=128,
             interleaved=False, scaling="none", dtype="bf16", lo=1024, hi=8192, tree=True, lens=22),
        # ragged prompts, most behind tokens that are there already; half of each head is rotated, for a long context
        dict(name="append_rope_prompts", op="append", seqs=12, new_lo=257, new_hi=2048, hq=32, hk=8, d=128, page=32, rot=64,
             interleaved=True, scaling="ramp", dtype="bf16", lo=0, hi=700, tree=False, lens=23),
        # prompts in 32 bits, every head with keys of its own, positions interpolated
        dict(name="append_rope_fp32", op="append", seqs=5, new_lo=900, new_hi=4001, hq=16, hk=16, d=64, page=128, rot=32,
             interleaved=True, scaling="linear", dtype="fp32", lo=0, hi=0, tree=False, lens=24),
        # a single request with a small tree: the smallest attention, where latency counts
        dict(name="attend_tree_single", op="attend", seqs=1, new_lo=16, new_hi=16, hq=32, hk=8, d=128, page=64, lo=2049,
             hi=2049, lens=31),
        # small trees behind 1k to 16k tokens: many requests, the cache's bytes count
        dict(name="attend_tree_batch_64", op="attend", seqs=64, new_lo=4, new_hi=8, hq=32, hk=8, d=128, page=64, lo=1024,
             hi=16384, lens=32),
        # ordinary trees of 17 to 32 nodes
        dict(name="attend_tree_batch_32", op="attend", seqs=32, new_lo=17, new_hi=32, hq=32, hk=8, d=128, page=64, lo=1024,
             hi=16384, lens=33),
        # wide trees of a model with eight query heads for each key / value head: the products count
        dict(name="attend_tree_wide", op="attend", seqs=8, new_lo=48, new_hi=64, hq=64, hk=8, d=128, page=128, lo=4096,
             hi=16384, lens=34),
        # the accepted paths of 64 requests
        dict(name="keep_path_64", op="keep", seqs=64, new_lo=32, new_hi=64, hk=8, d=128, page=64, lo=1024, hi=8192,
             keep_lo=1, keep_hi=8, lens=41),
        # long accepted paths of a large batch
        dict(name="keep_path_long", op="keep", seqs=256, new_lo=128, new_hi=256, hk=16, d=128, page=32, lo=64, hi=1024,
             keep_lo=16, keep_hi=64, lens=42),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, its logarithm spread evenly."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["build", "append", "append", "attend", "attend", "attend", "keep"])
    hk = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 4, 5, 8])
    d = rng.choice([32, 64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    case = dict(op=op, hk=hk, d=d, page=page, lens=rng.randrange(1 << 30))
    if op == "build":
        seqs = _spread(rng, 1, 512)
        new = _spread(rng, 1, 256)
        return dict(case, hk=1, d=32, seqs=seqs, new_lo=max(1, new // rng.choice([1, 2, 4])), new_hi=new, lo=0, hi=_spread(rng, 1, 1024))
    seqs = _spread(rng, 1, 64)
    case["seqs"] = seqs
    if op == "append":
        tree = rng.random() < 0.4
        per = _spread(rng, 1, max(1, (64 * 256 if tree else 16384) // seqs))
        per = min(per, 256) if tree else per
        return dict(case, hq=min(32, hk * group), new_lo=max(1, per // 3), new_hi=per, rot=2 * rng.randint(2, d // 2),
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "ramp"]),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), lo=0, hi=_spread(rng, 1, 4096), tree=tree)
    if op == "keep":
        new = _spread(rng, 2, 256)
        return dict(case, new_lo=max(2, new // 2), new_hi=new, lo=0, hi=_spread(rng, 1, 2048), keep_lo=0,
                    keep_hi=max(1, new // rng.choice([2, 4, 8])))
    # the tokens of a batch, times its heads, stay under those of the largest listed cases
    most = max(64, min(16384, (64 * 4096 * 8) // (seqs * hk)))
    hi = _spread(rng, 64, most)
    new = min(_spread(rng, 1, 256), max(1, (1 << 27) // (seqs * hk * group * (hi + 64))))  # ... and so do the scores
    return dict(case, hq=hk * group, lo=max(0, hi // rng.choice([1, 2, 16]) - 5), hi=hi, new_lo=max(1, new // 2), new_hi=new)


def _lens(case):
    """(tokens held after the call, tokens new in it, tokens kept of those) of each sequence, from the case alone."""
    rng = random.Random(case["lens"])
    n = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    had = [_spread(rng, case["lo"], case["hi"]) if case["hi"] else 0 for _ in range(case["seqs"])]
    kept = [min(rng.randint(case["keep_lo"], case["keep_hi"]), x) for x in n] if case["op"] == "keep" else [0] * len(n)
    return [a + b for a, b in zip(had, n)], n, kept


def _words(n):
    return -(-max(n) // 32)


def work(case):
    total, new, kept = _lens(case)
    T, d, hk = sum(new), case["d"], case["hk"]
    if case["op"] == "build":
        return {"bytes": T * 4 * (2 + _words(new)), "flops": T * _words(new)}
    if case["op"] == "append":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": T * d * (2 * case["hq"] * size + 2 * hk * (size + 1)), "flops": T * (3 * (case["hq"] + hk) * case["rot"] + 4 * hk * d)}
    if case["op"] == "keep":
        return {"bytes": sum(kept) * (hk * 2 * 2 * d + 4), "flops": sum(kept) * hk * 2 * d}
    cells = sum(n * (t - n) + n for t, n in zip(total, new))  # (a node sees itself at least)
    return {"bytes": sum(total) * hk * 2 * d + T * (case["hq"] * (4 * d + 4) + 4 * _words(new)), "flops": 4 * cells * case["hq"] * d}


# --------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(n):
    at = [0]
    for x in n:
        at.append(at[-1] + x)
    return _ints(at)


def _pow2(e):
    """2^e for whole numbers e, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _scale_exp(amax):
    """The least e with amax <= 448 2^e, in the range that scales have."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 7/8 2^9
    e = e - 9 + (m > 0.875)
    return torch.where(amax > 0, e, SCALE_EXP[0]).clamp(*SCALE_EXP)


def _codes(x):
    return x.clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn)


def _pages(case, total, g):
    """A cache that holds `total` tokens of each sequence: pages in shuffled order, keys with a few strong
    channels, page by page quantised."""
    ps, hk, d = case["page"], case["hk"], case["d"]
    width = max(1, max(-(-t // ps) for t in total))
    need = sum(-(-t // ps) for t in total)
    pool = need + 3
    order = torch.randperm(pool, generator=g, device="cuda")[:need].int()
    table = torch.zeros(len(total), width, dtype=torch.int32, device="cuda")
    at = 0
    for b, t in enumerate(total):
        n = -(-t // ps)
        table[b, :n] = order[at:at + n]
        at += n
    channel = 1 + 3 * (torch.rand(1, hk, 1, d, generator=g, device="cuda") > 0.95)
    out = {"table": table}
    for name, by in (("k", channel), ("v", 1.0)):
        x = torch.randn(pool, hk, ps, d, generator=g, device="cuda") * by
        e = _scale_exp(x.abs().amax((2, 3)))
        out[name + "_pages"] = _codes(x * _pow2(-e)[..., None, None]).view(torch.uint8)
        out[name + "_scale"] = _pow2(e)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    total, new, kept = _lens(case)
    T, hk, d = sum(new), case["hk"], case["d"]
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s = {"case": dict(case), "total": _ints(total), "cu": _cu(new), "max_new": max(new), "max_total": max(total)}
    s |= _pages(case, total, g)
    # a drafted tree: every node hangs on one of those before it, some on the last token of the text (-1)
    row = torch.arange(T, device="cuda") - s["cu"].long()[_owner(s["cu"], T)]
    s["parents"] = ((torch.rand(T, generator=g, device="cuda") * (row + 1)).int() - 1).clamp(min=-1).minimum(row.int() - 1)
    if case["op"] == "append":
        s["positions"] = _plain_build(s)["positions"] if case["tree"] else None
        s["q"] = randn(T, case["hq"], d).to(_dtype(case))
        s["k"], s["v"] = (1.35 * randn(T, hk, d)).to(_dtype(case)), (2 * randn(T, hk, d)).to(_dtype(case))
        s["touched"] = max((t - 1) // case["page"] - (t - n) // case["page"] + 1 for t, n in zip(total, new))
    if case["op"] == "attend":
        s["bits"] = _plain_build(s)["bits"]
        s["q"] = randn(T, case["hq"], d).to(torch.bfloat16)
        s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(case["hq"], T, device="cuda")
    if case["op"] == "keep":
        # an accepted path: its nodes in the tree's order
        s["path"] = torch.full((len(new), max(1, max(kept))), -1, dtype=torch.int32, device="cuda")
        rng = random.Random(seed)
        for b, (n, m) in enumerate(zip(new, kept)):
            if m:
                s["path"][b, :m] = _ints(sorted(rng.sample(range(n), m)))
        s["counts"], s["new_total"] = _ints(kept), torch.zeros(len(new), dtype=torch.int32, device="cuda")
        s["touched"] = max((t - n + max(m, 1) - 1) // case["page"] - (t - n) // case["page"] + 1 for t, n, m in zip(total, new, kept))
    return s


# --------------------------------------------------------------------------- the plain forms
def _owner(cu, T):
    """The sequence of each packed token."""
    return torch.searchsorted(cu, torch.arange(T, device="cuda", dtype=torch.int32), right=True) - 1


def _plain_build(s):
    """Ancestors by squaring: who can be reached in 1, 2, 4, .. steps up."""
    cu, total, n = s["cu"].long(), s["total"].long(), s["max_new"]
    T, B = s["parents"].shape[0], s["total"].shape[0]
    owner = _owner(s["cu"], T)
    row = torch.arange(T, device="cuda") - cu[owner]
    reach = torch.eye(n, device="cuda").expand(B, n, n).clone()
    up = s["parents"] >= 0
    reach[owner[up], row[up], s["parents"][up].long()] = 1
    for _ in range(max(1, (n - 1).bit_length())):
        reach = ((reach @ reach) > 0).float()
    seen = reach[owner, row]                                              # [T, n]
    words = -(-n // 32)
    weight = (1 << torch.arange(32, device="cuda"))                       # 64-bit whole numbers
    bits = (torch.nn.functional.pad(seen, (0, 32 * words - n)).view(T, words, 32).long() * weight).sum(-1)
    bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).int()     # the same 32 bits, signed
    positions = total[owner] - (cu[1:] - cu[:-1])[owner] + seen.sum(-1).long() - 1
    return {"bits": bits, "positions": positions.int()}


def _positions(s, T):
    """Where each new token stands: as given, or behind what its sequence held before."""
    if s["positions"] is not None:
        return s["positions"].long()
    cu = s["cu"].long()
    b = _owner(s["cu"], T)
    new = cu[1:] - cu[:-1]
    return torch.arange(T, device="cuda") - cu[b] + s["total"].long()[b] - new[b]


def _frequencies(case):
    """(angle of one position for each pair, the factor on the result), in 64 bits."""
    rot, kind = case["rot"], case["scaling"]
    base = BASE * FACTOR ** (rot / (rot - 2)) if kind == "ntk" else BASE
    theta = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if kind == "linear":
        theta = theta / FACTOR
    if kind == "ramp":
        turns = CONTEXT * theta / (2 * math.pi)
        keep = ((turns - ALPHA) / (BETA - ALPHA)).clamp(0, 1)
        return theta * ((1 - keep) / FACTOR + keep), 0.1 * math.log(FACTOR) + 1
    return theta, 1.0


def _rotate(x, cos, sin, rot, interleaved):
    """In the type of x."""
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    c, s = cos[:, None].to(x.dtype), sin[:, None].to(x.dtype)
    y = (a * c - b * s, b * c + a * s)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat((y, x[..., rot:]), -1)


def _f8(s, *names):
    return {n: s[n].view(torch.float8_e4m3fn) if n.endswith("pages") else s[n] for n in names}


def _plain_append(s):
    case = s["case"]
    T = s["q"].shape[0]
    theta, m = _frequencies(case)
    angle = _positions(s, T).double()[:, None] * theta
    cos, sin = angle.cos() * m, angle.sin() * m
    q = _rotate(s["q"].float(), cos, sin, case["rot"], case["interleaved"]).to(s["q"].dtype)
    # keys in 64 bits: a page's scale turns on whether its largest passes a border
    _plain_store(s, "k", _rotate(s["k"].double(), cos, sin, case["rot"], case["interleaved"]))
    _plain_store(s, "v", s["v"].float())
    return {"q": q, **_f8(s, "k_pages", "k_scale", "v_pages", "v_scale")}


def _plain_store(s, name, values):
    case, table, ps = s["case"], s["table"].long(), s["case"]["page"]
    cu, total = s["cu"].long(), s["total"].long()
    held = total - (cu[1:] - cu[:-1])
    # pages that each sequence writes to, the first of them perhaps begun
    first = held // ps
    local = first[:, None] + torch.arange(s["touched"], device="cuda")
    used = local < (total[:, None] + ps - 1) // ps
    page = table.gather(1, local.clamp(max=table.shape[1] - 1))
    at = local[..., None] * ps + torch.arange(ps, device="cuda")          # [B, touched, ps] token numbers
    old = at < held[:, None, None]
    fresh = ~old & (at < total[:, None, None])
    src = (cu[:-1, None, None] + at - held[:, None, None]).clamp(0, values.shape[0] - 1)
    x = values[src].transpose(2, 3)                                       # [B, touched, hk, ps, d]
    x = torch.where(fresh[:, :, None, :, None], x, 0.0)
    e = _scale_exp(x.abs().amax((3, 4)))
    was = s[name + "_scale"][page]
    begun = old.any(2)[..., None]
    scale = torch.where(begun, torch.maximum(was, _pow2(e)), _pow2(e))
    codes = s[name + "_pages"][page].view(torch.float8_e4m3fn).to(x.dtype)
    codes = torch.where(old[:, :, None, :, None], codes * (was / scale)[..., None, None], codes)
    codes = torch.where(fresh[:, :, None, :, None], x / scale[..., None, None], codes)
    sel = page[used]
    s[name + "_pages"][sel] = _codes(codes[used]).view(torch.uint8)
    s[name + "_scale"][sel] = scale[used]


def _cached(s, name):
    """The cache's numbers of each sequence, [B, heads, tokens, d], in 32 bits."""
    x = s[name + "_pages"].view(torch.float8_e4m3fn).float() * s[name + "_scale"][..., None, None]
    x = x[s["table"].long()].transpose(1, 2)                              # [B, hk, pages, ps, d]
    return x.flatten(2, 3)[:, :, :s["max_total"]]


def _plain_attend(s):
    case = s["case"]
    q, hk, N = s["q"], case["hk"], s["max_new"]
    T, hq, d = q.shape
    B, g = case["seqs"], hq // hk
    cu, total = s["cu"].long(), s["total"].long()
    n = cu[1:] - cu[:-1]
    owner = _owner(s["cu"], T)
    row = torch.arange(T, device="cuda") - cu[owner]
    padded = torch.zeros(B, N, hq, d, device="cuda")
    padded[owner, row] = q.float()
    padded = padded.view(B, N, hk, g, d).transpose(1, 2)                  # [B, hk, new, g, d]
    score = (padded.flatten(2, 3) @ _cached(s, "k").transpose(2, 3)).view(B, hk, N, g, -1) / math.sqrt(d)
    # what each new token sees: the text before the tree, and of the tree what its bits say
    bits = torch.zeros(B, N, s["bits"].shape[1], dtype=torch.int32, device="cuda")
    bits[owner, row] = s["bits"]
    j = torch.arange(score.shape[-1], device="cuda") - (total - n)[:, None]  # [B, L]: number in the tree
    inside = (j >= 0) & (j < n[:, None])
    at = j.clamp(0, N - 1)[:, None].expand(B, N, -1)
    seen = ((bits.gather(2, at // 32) >> (at % 32).int()) & 1).bool() & inside[:, None] | (j < 0)[:, None]
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (score - top).exp_()
    sums = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ _cached(s, "v")).view(B, hk, N, g, -1) / sums.clamp(min=1e-30)
    lse = (top + sums.log())[..., 0]
    s["o"].copy_(o.transpose(1, 2).flatten(2, 3)[owner, row])
    s["lse"].copy_(lse.transpose(1, 2).flatten(2, 3)[owner, row].t())
    return {"o": s["o"], "lse": s["lse"]}


def _plain_keep(s):
    case, ps = s["case"], s["case"]["page"]
    cu, total, m = s["cu"].long(), s["total"].long(), s["counts"].long()
    base = total - (cu[1:] - cu[:-1])
    table = s["table"].long()
    local = (base // ps)[:, None] + torch.arange(s["touched"], device="cuda")
    used = (local * ps < (base + m)[:, None]) & (m > 0)[:, None]
    page = table.gather(1, local.clamp(max=table.shape[1] - 1))           # [B, touched]
    at = (local[..., None] * ps + torch.arange(ps, device="cuda")).flatten(1)   # token numbers of their slots
    j = at - base[:, None]                                                # number in the path
    moved = (j >= 0) & (j < m[:, None])
    src = torch.where(moved, base[:, None] + s["path"].long().gather(1, j.clamp(0, s["path"].shape[1] - 1)), at)
    src = src.minimum(total[:, None] - 1).clamp(min=0)
    held = moved | ((j < 0) & (at >= 0))                                  # slots that hold tokens of the result
    live = held | (at < total[:, None])                                   # ... or drafted ones still
    src_page = table.gather(1, src // ps)
    shape = (case["seqs"], s["touched"], ps)
    for name in ("k", "v"):
        scale = s[name + "_scale"][src_page]                              # [B, slots, hk]
        was = s[name + "_scale"][page]                                    # [B, touched, hk]
        top = torch.where(held[..., None], scale, 0.0).view(*shape, -1).amax(2).maximum(was)
        by = scale.view(*shape, -1) / top[:, :, None]                     # [B, touched, ps, hk]
        x = s[name + "_pages"][src_page, :, src % ps].view(torch.float8_e4m3fn).float()
        x = _codes(x.view(*shape, *x.shape[2:]) * by[..., None]).view(torch.uint8).transpose(2, 3)
        there = s[name + "_pages"][page]
        x = torch.where(live.view(shape)[:, :, None, :, None], x, there)
        s[name + "_pages"][page[used]] = x[used]
        s[name + "_scale"][page[used]] = top[used]
    s["new_total"].copy_(base + m)
    return _kept(s)


def _kept(s):
    return {"new_total": s["new_total"], **_f8(s, "k_pages", "k_scale", "v_pages", "v_scale")}


# --------------------------------------------------------------------------- the framework's calls
def _handles(s):
    """What a serving program makes once and keeps: the rotation's plan, the handle of the cache."""
    from block_sparse_masked_mask_gb300 import api
    if "handle" not in s:
        case = s["case"]
        s["handle"] = api.KVCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"])
        if case["op"] == "append":
            s["plan"] = api.attn_rope_plan(case["rot"], base=BASE, interleaved=case["interleaved"], scaling=case["scaling"],
                                           factor=FACTOR, original_context=CONTEXT, alpha=ALPHA, beta=BETA)
    return api, s["handle"]


def _own(s):
    api, handle = _handles(s)
    op = s["case"]["op"]
    if op == "build":
        bits, positions = api.attn_cache_tree_build(s["parents"], handle, s["cu"], s["total"], s["max_new"])
        return {"bits": bits, "positions": positions}
    if op == "append":
        q = api.attn_cache_append_rope(s["q"], s["k"], s["v"], s["plan"], handle, s["cu"], s["total"], s["max_new"],
                                       positions=s["positions"])
        return {"q": q, **_f8(s, "k_pages", "k_scale", "v_pages", "v_scale")}
    if op == "attend":
        api.attn_cache_tree_fwd(s["q"], handle, s["bits"], s["cu"], s["total"], s["max_new"], s["max_total"],
                                out=s["o"], lse=s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    api.attn_cache_tree_keep(s["path"], s["counts"], handle, s["cu"], s["total"], s["max_new"], new_lens=s["new_total"])
    return _kept(s)


def run(state):
    if own:
        return _own(state)
    return {"build": _plain_build, "append": _plain_append, "attend": _plain_attend, "keep": _plain_keep}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    if case["op"] == "build":
        return None  # whole numbers
    s = prepare(case, seed)
    total, new, kept = _lens(case)
    starts = [sum(new[:b]) for b in range(len(new))]
    if case["op"] == "append":
        return _exact_append(case, s, total, new, starts)
    if case["op"] == "attend":
        return _exact_attend(case, s, total, new, starts)
    return _exact_keep(case, s, total, new, kept)


def _turned(case, x, p):
    """Each pair as a complex number, times m e^(i p theta)."""
    rot = case["rot"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    theta = torch.exp(-2 * i / rot * math.log(BASE * (FACTOR ** (rot / (rot - 2)) if case["scaling"] == "ntk" else 1)))
    m = 1.0
    if case["scaling"] == "linear":
        theta = theta / FACTOR
    if case["scaling"] == "ramp":
        g = torch.clamp((CONTEXT / (2 * math.pi / theta) - ALPHA) / (BETA - ALPHA), 0, 1)
        theta, m = (1 - g) * theta / FACTOR + g * theta, 1 + math.log(FACTOR) / 10
    turn = torch.polar(torch.full((len(p), rot // 2), m, dtype=torch.float64, device="cuda"), torch.outer(p, theta))
    first = torch.arange(rot // 2, device="cuda")
    a, b = (2 * first, 2 * first + 1) if case["interleaved"] else (first, first + rot // 2)
    z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
    y = x.clone()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_append(case, s, total, new, starts):
    """The rotated numbers before they are rounded, those of the cache in units of their page's scale."""
    ps = case["page"]
    if s["positions"] is None:
        p = torch.cat([torch.arange(t - n, t, dtype=torch.float64, device="cuda") for t, n in zip(total, new)])
    else:
        p = s["positions"].double()
    out = {"q": _turned(case, s["q"].double(), p)}
    for name in ("k", "v"):
        fresh = s[name].double()
        if name == "k":
            fresh = _turned(case, fresh, p)
        codes = s[name + "_pages"].view(torch.float8_e4m3fn).double()
        scale = s[name + "_scale"].double()
        for b, (t, n, at) in enumerate(zip(total, new, starts)):
            for j in range((t - n) // ps, -(-t // ps)):
                page = int(s["table"][b, j])
                lo, hi = max(t - n, j * ps), min(t, (j + 1) * ps)
                x = fresh[at + lo - (t - n):at + hi - (t - n)].transpose(0, 1)
                big = x.abs().amax((1, 2)).clamp(min=1e-300)
                unit = torch.exp2(torch.ceil(torch.log2(big / F8_MAX)).clamp(*SCALE_EXP))
                unit = torch.where(big <= F8_MAX * unit / 2, unit / 2, unit)  # a logarithm rounded over a whole number
                held = lo - j * ps
                if held:
                    unit = torch.maximum(unit, scale[page])
                    codes[page, :, :held] *= (scale[page] / unit)[:, None, None]
                codes[page, :, held:hi - j * ps] = x / unit[:, None, None]
                scale[page] = unit
        out[name + "_pages"], out[name + "_scale"] = codes, scale
    return out


def _numbers(s, name, b, t):
    """[heads, t, d] of sequence b."""
    pages = s["table"][b, :-(-t // s["case"]["page"])].long()
    x = s[name + "_pages"][pages].view(torch.float8_e4m3fn).double() * s[name + "_scale"][pages].double()[..., None, None]
    return x.transpose(0, 1).flatten(1, 2)[:, :t]


def _exact_attend(case, s, total, new, starts):
    hk, d = case["hk"], case["d"]
    parents = s["parents"].tolist()
    o, lse = [], []
    for b, (t, n, at) in enumerate(zip(total, new, starts)):
        hidden = torch.ones(n, t, dtype=torch.bool)
        hidden[:, :t - n] = False
        for i in range(n):  # up from the node
            j = i
            while j >= 0:
                hidden[i, t - n + j] = False
                j = parents[at + j]
        q = s["q"][at:at + n].double().view(n, hk, -1, d).transpose(0, 1)
        x = torch.einsum("hngd,htd->hngt", q, _numbers(s, "k", b, t)) / math.sqrt(d)
        x.masked_fill_(hidden.cuda()[:, None], -math.inf)
        z = torch.logsumexp(x, -1)
        w = torch.einsum("hngt,htd->hngd", torch.exp(x - z[..., None]), _numbers(s, "v", b, t))
        o.append(w.transpose(0, 1).flatten(1, 2))
        lse.append(z.transpose(0, 1).flatten(1, 2).t())
    return {"o": torch.cat(o), "lse": torch.cat(lse, 1)}


def _exact_keep(case, s, total, new, kept):
    """The moved numbers before they are rounded, in units of their new page's scale."""
    ps, out = case["page"], {"new_total": None}
    paths = s["path"].tolist()
    for name in ("k", "v"):
        codes = s[name + "_pages"].view(torch.float8_e4m3fn).double()
        scale = s[name + "_scale"].double()
        for b, (t, n, m) in enumerate(zip(total, new, kept)):
            base = t - n
            table = s["table"][b].tolist()
            old = {}  # the pages as they were
            for p in range(base // ps, -(-t // ps)):
                old[p] = (codes[table[p]].clone(), scale[table[p]].clone())
            for p in range(base // ps, -(-(base + m) // ps) if m else 0):
                from_ = {a: base + paths[b][a - base] for a in range(max(base, p * ps), min(base + m, (p + 1) * ps))}
                unit = old[p][1]
                for a in from_.values():
                    unit = torch.maximum(unit, old[a // ps][1])
                for a in range(p * ps, min((p + 1) * ps, t)):
                    x, by = old[from_.get(a, a) // ps]
                    codes[table[p], :, a % ps] = x[:, from_.get(a, a) % ps] * (by / unit)[:, None]
                scale[table[p]] = unit
        out[name + "_pages"], out[name + "_scale"] = codes, scale
    return out
