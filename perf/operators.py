"""The serving operators' measured cases: rotary positions, the 8-bit key/value cache (append, attention,
attention weights received) and eviction from it.

Every case is a dict of plain values; ``prepare`` makes its inputs from a seed, ``run`` makes one pass
(the framework's calls where ``own`` is true, elementary torch operations in 32 bits where it is not) and
``exact`` gives the same outputs from the definitions in 64 bits.  The cache's codes are returned as
float8 numbers next to their power-of-two scales.
"""
import math
import random

import torch

own = False

F8_MAX = 448.0        # largest finite e4m3 number
SCALE_EXP = (-80, 120)  # exponents a page's scale may take


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 requests: the smallest rotation, half of each head, long contexts
        dict(name="rope_decode_64", op="rope", seqs=64, new_lo=1, new_hi=1, hq=32, hk=8, d=128, rot=64,
             interleaved=True, scaling="ramp", dtype="bf16", inverse=False, lo=64, hi=131072, explicit=False, lens=11),
        # the packed 32k training batch of documents, 32 heads for q and for k
        dict(name="rope_documents_32k", op="rope", seqs=12, new_lo=2731, new_hi=2731, hq=32, hk=32, d=128, rot=128,
             interleaved=False, scaling="none", dtype="bf16", inverse=False, lo=0, hi=0, explicit=True, lens=12),
        # its gradient in 32 bits at ragged lengths, part of each head, positions interpolated
        dict(name="rope_gradient_fp32", op="rope", seqs=5, new_lo=900, new_hi=4001, hq=16, hk=16, d=64, rot=32,
             interleaved=True, scaling="linear", dtype="fp32", inverse=True, lo=0, hi=0, explicit=False, lens=13),
        # one decode step of 64 requests puts its tokens into the cache
        dict(name="append_decode_64", op="append", seqs=64, new_lo=1, new_hi=1, hk=8, d=128, page=64, dtype="bf16",
             lo=1024, hi=16384, lens=21),
        # ragged prompts go in, most behind tokens that are there already
        dict(name="append_prompts", op="append", seqs=12, new_lo=257, new_hi=2048, hk=16, d=128, page=32, dtype="bf16",
             lo=0, hi=700, lens=22),
        # a single request's decode step: the smallest attention, where latency counts
        dict(name="attend_single", op="attend", seqs=1, new_lo=1, new_hi=1, hq=32, hk=8, d=128, page=64, causal=True,
             lo=2049, hi=2049, lens=31),
        # a decode step of 64 requests of 1k to 16k tokens: the largest pass over a cache
        dict(name="attend_batch_64", op="attend", seqs=64, new_lo=1, new_hi=1, hq=32, hk=8, d=128, page=64, causal=True,
             lo=1024, hi=16384, lens=32),
        # chunks of prompts attend to what is cached and to themselves
        dict(name="attend_chunks", op="attend", seqs=4, new_lo=300, new_hi=512, hq=32, hk=8, d=128, page=128, causal=True,
             lo=4096, hi=16384, lens=33),
        # the weights that a decode step's queries give to the cached tokens
        dict(name="weigh_batch_32", op="weigh", seqs=32, new_lo=1, new_hi=1, hq=32, hk=8, d=128, page=64, causal=True,
             lo=1024, hi=16384, lens=41),
        # a window of a prompt's last queries scores its tokens, every head with keys of its own
        dict(name="weigh_window", op="weigh", seqs=8, new_lo=32, new_hi=32, hq=16, hk=16, d=128, page=32, causal=True,
             lo=1000, hi=8192, lens=42),
        # one request's cache is cut to half
        dict(name="evict_single", op="evict", seqs=1, hk=8, d=128, page=64, lo=2049, hi=2049, keep=0.5, recent=64, lens=51),
        # a batch of caches is cut to half
        dict(name="evict_batch_32", op="evict", seqs=32, hk=8, d=128, page=64, lo=1024, hi=16384, keep=0.5, recent=256, lens=52),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, its logarithm spread evenly."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "weigh", "evict"])
    lens = rng.randrange(1 << 30)
    hk = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 4, 5, 8])
    d = rng.choice([32, 64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    seqs = _spread(rng, 1, 64)
    case = dict(op=op, seqs=seqs, hk=hk, d=d, lens=lens)
    if op == "rope":
        per = _spread(rng, 1, max(1, 32768 // seqs))
        return dict(case, hq=min(32, hk * group), new_lo=max(1, per // 3), new_hi=per, rot=2 * rng.randint(2, d // 2),
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "ramp"]),
                    dtype=rng.choice(["bf16", "fp32"]), inverse=rng.random() < 0.5, lo=0, hi=_spread(rng, 1, 131072),
                    explicit=rng.random() < 0.5)
    if op == "append":
        per = _spread(rng, 1, max(1, 16384 // seqs))
        return dict(case, page=page, new_lo=max(1, per // 3), new_hi=per, dtype=rng.choice(["bf16", "fp32"]), lo=0,
                    hi=_spread(rng, 1, 4096))
    # the tokens of a batch, times its heads, stay under those of the largest listed case
    most = max(64, min(16384, (64 * 4096 * 8) // (seqs * hk)))
    hi = _spread(rng, 64, most)
    case.update(page=page, lo=max(1, hi // rng.choice([1, 2, 16])), hi=hi)
    if op == "evict":
        return dict(case, keep=rng.choice([0.1, 0.25, 0.5, 0.9]), recent=_spread(rng, 1, 256))
    new = rng.choice([1, 1, 2, 5, 64, 300]) if op == "attend" else rng.choice([1, 1, 3, 16, 64])
    # ... and so do the scores
    new = max(1, min(new, (1 << 28) // (seqs * hk * group * hi)))
    return dict(case, hq=hk * group, new_lo=max(1, new // 2), new_hi=new, causal=rng.random() < 0.8)


def _lens(case):
    """(tokens held after the call, tokens new in it) of each sequence, from the case alone."""
    rng = random.Random(case["lens"])
    n = [rng.randint(case["new_lo"], case["new_hi"]) if case.get("new_hi") else 0 for _ in range(case["seqs"])]
    if case.get("name") == "rope_documents_32k":
        n[-1] += 32768 - sum(n)
    had = [_spread(rng, case["lo"], case["hi"]) if case["hi"] else 0 for _ in range(case["seqs"])]
    if case["op"] in ("attend", "weigh"):  # lo and hi count the new tokens in
        return [max(a, b) for a, b in zip(had, n)], n
    return [a + b for a, b in zip(had, n)], n


def work(case):
    total, new = _lens(case)
    T, d, hk = sum(new), case["d"], case["hk"]
    if case["op"] == "rope":
        values = T * (case["hq"] + hk) * d
        return {"bytes": 2 * values * (2 if case["dtype"] == "bf16" else 4), "flops": 3 * T * (case["hq"] + hk) * case["rot"]}
    if case["op"] == "append":
        return {"bytes": 2 * T * hk * d * ((2 if case["dtype"] == "bf16" else 4) + 1), "flops": 4 * T * hk * d}
    if case["op"] == "evict":
        kept = sum(_kept(case, x) for x in total)
        return {"bytes": hk * (sum(total) * 4 + kept * (2 * 2 * d + 8)), "flops": hk * sum(total)}
    cells = sum(n * (t if not case["causal"] else t - n) + (n * (n + 1) // 2 if case["causal"] else 0) for t, n in zip(total, new))
    if case["op"] == "attend":
        return {"bytes": sum(total) * hk * 2 * d + T * case["hq"] * (4 * d + 4), "flops": 4 * cells * case["hq"] * d}
    return {"bytes": sum(total) * hk * (d + 8) + T * case["hq"] * (2 * d + 4), "flops": 2 * cells * case["hq"] * d}


def _kept(case, total):
    return min(total, max(1, int(total * case["keep"])))


# --------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32


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
    total, new = _lens(case)
    T, hk, d = sum(new), case["hk"], case["d"]
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s = {"case": dict(case), "total": _ints(total), "cu": _cu(new), "max_new": max(new), "max_total": max(total)}
    if case["op"] == "rope":
        s["q"], s["k"] = randn(T, case["hq"], d).to(_dtype(case)), randn(T, hk, d).to(_dtype(case))
        s["positions"] = _positions(s, T).int() if case["explicit"] else None
        return s
    if case["op"] == "append":
        held = [t - n for t, n in zip(total, new)]
        s |= _pages(case, total, g)
        s["k"], s["v"] = randn(T, hk, d).to(_dtype(case)), (2 * randn(T, hk, d)).to(_dtype(case))
        s["touched"] = max((t - 1) // case["page"] - h // case["page"] + 1 for t, h in zip(total, held))
        return s
    s |= _pages(case, total, g)
    if case["op"] == "evict":
        kept = [_kept(case, t) for t in total]
        ps = case["page"]
        # weights of many sizes, some tokens never looked at
        w = torch.exp(2 * randn(len(total), hk, max(total)))
        s["weights"] = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.05, 0.0, w)
        s["budgets"], s["most"] = _ints(kept), max(kept)
        pages = [-(-n // ps) for n in kept]
        s["dst_table"] = torch.zeros(len(total), max(pages), dtype=torch.int32, device="cuda")
        order = torch.randperm(sum(pages), generator=g, device="cuda").int()
        at = 0
        for b, n in enumerate(pages):
            s["dst_table"][b, :n] = order[at:at + n]
            at += n
        for name in ("k", "v"):
            s["dst_%s_pages" % name] = torch.zeros(sum(pages), hk, ps, d, dtype=torch.uint8, device="cuda")
            s["dst_%s_scale" % name] = torch.ones(sum(pages), hk, device="cuda")
        s["kept"] = torch.full((len(total), hk, max(kept)), -1, dtype=torch.int32, device="cuda")
        s["new_weights"] = torch.zeros(len(total), hk, max(kept), device="cuda")
        s["new_total"] = torch.zeros(len(total), dtype=torch.int32, device="cuda")
        return s
    s["q"] = randn(T, case["hq"], d).to(torch.bfloat16)
    s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(case["hq"], T, device="cuda")
    if case["op"] == "weigh":
        s["lse"] = _scores(s)[1]
        s["prev"] = torch.rand(len(total), hk, max(total), generator=g, device="cuda")
        s["weights"] = s["prev"].clone()
    return s


# --------------------------------------------------------------------------- the plain forms
def _owner(cu, T):
    """The sequence of each packed token."""
    return torch.searchsorted(cu, torch.arange(T, device="cuda", dtype=torch.int32), right=True) - 1


def _positions(s, T):
    """Where each new token stands in its sequence: behind what the sequence held before."""
    cu = s["cu"].long()
    b = _owner(s["cu"], T)
    new = cu[1:] - cu[:-1]
    return torch.arange(T, device="cuda") - cu[b] + s["total"].long()[b] - new[b]


FACTOR, CONTEXT, BASE, ALPHA, BETA = 8.0, 8192, 10000.0, 1.0, 32.0


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
    x32 = x.float()
    if interleaved:
        a, b = x32[..., 0:rot:2], x32[..., 1:rot:2]
    else:
        a, b = x32[..., :rot // 2], x32[..., rot // 2:rot]
    c, s = cos[:, None], sin[:, None]
    y = (a * c - b * s, b * c + a * s)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat((y, x32[..., rot:]), -1).to(x.dtype)


def _plain_rope(s):
    case = s["case"]
    T = s["q"].shape[0]
    p = _positions(s, T) if s["positions"] is None else s["positions"]
    theta, m = _frequencies(case)
    angle = p.double()[:, None] * theta
    cos, sin = (angle.cos() * m).float(), (angle.sin() * (-m if case["inverse"] else m)).float()
    return {n: _rotate(s[n], cos, sin, case["rot"], case["interleaved"]) for n in ("q", "k")}


def _f8(s, *names):
    return {n: s[n].view(torch.float8_e4m3fn) if n.endswith("pages") else s[n] for n in names}


def _plain_append(s):
    case, table, ps = s["case"], s["table"].long(), s["case"]["page"]
    T = s["k"].shape[0]
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
    src = (cu[:-1, None, None] + at - held[:, None, None]).clamp(0, T - 1)
    out = {}
    for name in ("k", "v"):
        x = s[name][src].float().transpose(2, 3)                          # [B, touched, hk, ps, d]
        x = torch.where(fresh[:, :, None, :, None], x, 0.0)
        e = _scale_exp(x.abs().amax((3, 4)))
        was = s[name + "_scale"][page]
        begun = old.any(2)[..., None]
        scale = torch.where(begun, torch.maximum(was, _pow2(e)), _pow2(e))
        codes = s[name + "_pages"][page].view(torch.float8_e4m3fn).float()
        codes = torch.where(old[:, :, None, :, None], codes * (was / scale)[..., None, None], codes)
        codes = torch.where(fresh[:, :, None, :, None], x / scale[..., None, None], codes)
        sel = page[used]
        s[name + "_pages"][sel] = _codes(codes[used]).view(torch.uint8)
        s[name + "_scale"][sel] = scale[used]
    return _f8(s, "k_pages", "k_scale", "v_pages", "v_scale")


def _cached(s, name):
    """The cache's numbers of each sequence, [B, heads, tokens, d], in 32 bits."""
    x = s[name + "_pages"].view(torch.float8_e4m3fn).float() * s[name + "_scale"][..., None, None]
    x = x[s["table"].long()].transpose(1, 2)                              # [B, hk, pages, ps, d]
    return x.flatten(2, 3)[:, :, :s["max_total"]]


def _scores(s):
    """(scores with what is hidden at -inf [B, hk, new, group, tokens], lse [hq, T], owner, place of each row)."""
    case = s["case"]
    q, hk = s["q"], case["hk"]
    T, hq, d = q.shape
    B, g = case["seqs"], hq // hk
    owner = _owner(s["cu"], T)
    row = torch.arange(T, device="cuda") - s["cu"].long()[owner]
    padded = torch.zeros(B, s["max_new"], hq, d, device="cuda")
    padded[owner, row] = q.float()
    padded = padded.view(B, s["max_new"], hk, g, d).transpose(1, 2)       # [B, hk, new, g, d]
    score = (padded.flatten(2, 3) @ _cached(s, "k").transpose(2, 3)).view(B, hk, s["max_new"], g, -1) / math.sqrt(d)
    cu, total = s["cu"].long(), s["total"].long()
    n = cu[1:] - cu[:-1]
    j = torch.arange(score.shape[-1], device="cuda")
    i = torch.arange(s["max_new"], device="cuda")
    last = total[:, None] - n[:, None] + i if case["causal"] else (total[:, None] - 1).expand(B, s["max_new"])
    seen = (j <= last[..., None]) & (j < total[:, None, None]) & (i < n[:, None])[..., None]
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1).clamp(min=-1e30)
    lse = top + (score - top[..., None]).exp_().sum(-1).log()             # [B, hk, new, g]
    return score, lse.transpose(1, 2).flatten(2, 3)[owner, row].t().contiguous(), owner, row


def _plain_attend(s):
    score, lse, owner, row = _scores(s)
    B, hk, n, g, L = score.shape
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (score - top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ _cached(s, "v")).view(B, hk, n, g, -1) / total.clamp(min=1e-30)
    s["o"].copy_(o.transpose(1, 2).flatten(2, 3)[owner, row])
    s["lse"].copy_(lse)
    return {"o": s["o"], "lse": s["lse"]}


def _plain_weigh(s):
    score, _, owner, row = _scores(s)
    B, hk, n, g, L = score.shape
    lse = torch.zeros(B, n, hk * g, device="cuda")
    lse[owner, row] = s["lse"].t()
    lse = lse.view(B, n, hk, g).transpose(1, 2)
    got = (score - lse[..., None]).exp_().sum((2, 3))
    held = torch.arange(L, device="cuda") < s["total"][:, None, None]
    s["weights"].copy_(torch.where(held, s["prev"] + got, s["prev"]))
    return {"weights": s["weights"]}


def _plain_evict(s):
    case, ps = s["case"], s["case"]["page"]
    B, hk, W = s["weights"].shape
    total, budget = s["total"].long(), torch.minimum(s["budgets"], s["total"]).long()
    j = torch.arange(W, device="cuda")
    recent = torch.minimum(budget, torch.tensor(case["recent"], device="cuda"))
    rank = torch.where(j >= (total - recent)[:, None, None], math.inf, s["weights"])
    rank = torch.where(j < total[:, None, None], rank, -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True).indices            # ties: lowest index first
    chosen = torch.where(torch.arange(W, device="cuda") < budget[:, None, None], order, W)
    kept = chosen.sort(-1).values[..., :s["most"]]                         # [B, hk, most], W behind the last
    there = kept < W
    at = kept.clamp(max=W - 1)
    s["kept"].copy_(torch.where(there, kept, -1))
    s["new_weights"].copy_(torch.where(there, s["weights"].gather(2, at), 0.0))
    s["new_total"].copy_(budget)
    pages = s["dst_table"].shape[1]
    pad = pages * ps - s["most"]
    at, there = (torch.nn.functional.pad(x, (0, pad)) for x in (at, there))
    page = s["table"].long().gather(1, (at // ps).flatten(1)).view(at.shape)
    h = torch.arange(hk, device="cuda")[None, :, None]
    used = (torch.arange(pages, device="cuda") * ps < budget[:, None])     # [B, pages]
    dst = s["dst_table"].long()[used]
    slot = there.view(B, hk, pages, ps).transpose(1, 2)[used]              # [used pages, hk, ps]
    for name in ("k", "v"):
        scale = torch.where(there, s[name + "_scale"][page, h], 0.0)
        x = s[name + "_pages"][page, h, at % ps].view(torch.float8_e4m3fn).float()
        top = scale.view(B, hk, pages, ps).amax(-1, keepdim=True)
        x = x * (scale.view(B, hk, pages, ps) / top.clamp(min=1e-30)).flatten(2)[..., None]
        x = _codes(x.view(B, hk, pages, ps, -1).transpose(1, 2)[used]).view(torch.uint8)
        s["dst_%s_pages" % name][dst] = torch.where(slot[..., None], x, s["dst_%s_pages" % name][dst])
        s["dst_%s_scale" % name][dst] = top[..., 0].transpose(1, 2)[used]
    return _evicted(s)


def _evicted(s):
    return _f8(s, "kept", "new_weights", "new_total", "dst_k_pages", "dst_k_scale", "dst_v_pages", "dst_v_scale")


# --------------------------------------------------------------------------- the framework's calls
def _handles(s):
    """What a serving program makes once and keeps: the rotation's plan, the handle of the cache."""
    from block_sparse_masked_mask_gb300 import api
    if "handle" not in s:
        case = s["case"]
        if case["op"] == "rope":
            s["handle"] = api.attn_rope_plan(case["rot"], base=BASE, interleaved=case["interleaved"], scaling=case["scaling"],
                                             factor=FACTOR, original_context=CONTEXT, alpha=ALPHA, beta=BETA)
        else:
            s["handle"] = api.KVCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"])
        if case["op"] == "evict":
            s["dst"] = api.KVCache(s["dst_k_pages"], s["dst_v_pages"], s["dst_k_scale"], s["dst_v_scale"], s["dst_table"])
    return api, s["handle"]


def _own(s):
    api, handle = _handles(s)
    case = s["case"]
    if case["op"] == "rope":
        where = {"cu_seqlens": s["cu"], "seq_lens": s["total"]} if s["positions"] is None else {"positions": s["positions"]}
        q, k = api.attn_rope(s["q"], s["k"], handle, inverse=case["inverse"], **where)
        return {"q": q, "k": k}
    if case["op"] == "append":
        api.attn_cache_append(s["k"], s["v"], handle, s["cu"], s["total"], s["max_new"])
        return _f8(s, "k_pages", "k_scale", "v_pages", "v_scale")
    if case["op"] == "evict":
        api.attn_cache_evict(s["weights"], handle, s["dst"], s["total"], s["budgets"], case["recent"], s["max_total"],
                             s["most"], kept=s["kept"], new_weights=s["new_weights"], new_lens=s["new_total"])
        return _evicted(s)
    kind = "causal" if case["causal"] else "none"
    if case["op"] == "attend":
        api.attn_cache_fwd(s["q"], handle, s["cu"], s["total"], s["max_new"], s["max_total"], kind=kind, out=s["o"], lse=s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    api.attn_cache_weights(s["q"], s["lse"], handle, s["cu"], s["total"], s["max_new"], s["max_total"], kind=kind,
                           prev=s["prev"], out=s["weights"])
    return {"weights": s["weights"]}


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "weigh": _plain_weigh,
            "evict": _plain_evict}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    total, new = _lens(case)
    starts = [sum(new[:b]) for b in range(len(new))]
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend, "weigh": _exact_weigh,
            "evict": _exact_evict}[case["op"]](case, s, total, new, starts)


def _exact_rope(case, s, total, new, starts):
    """Each pair as a complex number, times m e^(i p theta) (its conjugate for the gradient)."""
    rot = case["rot"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    theta = torch.exp(-2 * i / rot * math.log(BASE * (FACTOR ** (rot / (rot - 2)) if case["scaling"] == "ntk" else 1)))
    m = 1.0
    if case["scaling"] == "linear":
        theta = theta / FACTOR
    if case["scaling"] == "ramp":
        g = torch.clamp((CONTEXT / (2 * math.pi / theta) - ALPHA) / (BETA - ALPHA), 0, 1)
        theta, m = (1 - g) * theta / FACTOR + g * theta, 1 + math.log(FACTOR) / 10
    p = torch.cat([torch.arange(t - n, t, dtype=torch.float64, device="cuda") for t, n in zip(total, new)])
    turn = torch.polar(torch.full((len(p), rot // 2), m, dtype=torch.float64, device="cuda"), torch.outer(p, theta))
    turn = turn.conj() if case["inverse"] else turn
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        first = torch.arange(rot // 2, device="cuda")
        a, b = (2 * first, 2 * first + 1) if case["interleaved"] else (first, first + rot // 2)
        z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
        y = x.clone()
        y[..., a], y[..., b] = z.real, z.imag
        out[name] = y
    return out


def _numbers(s, name):
    return s[name + "_pages"].view(torch.float8_e4m3fn).double() * s[name + "_scale"].double()[..., None, None]


def _sequence(s, numbers, b, t):
    """[heads, t, d] of sequence b."""
    ps = s["case"]["page"]
    pages = s["table"][b, :-(-t // ps)].long()
    return numbers[pages].transpose(0, 1).flatten(1, 2)[:, :t]


def _exact_append(case, s, total, new, starts):
    """The numbers before they are rounded, in units of their page's scale."""
    ps, out = case["page"], {}
    for name in ("k", "v"):
        codes = s[name + "_pages"].view(torch.float8_e4m3fn).double()
        scale = s[name + "_scale"].double()
        for b, (t, n, at) in enumerate(zip(total, new, starts)):
            for j in range((t - n) // ps, -(-t // ps)):
                page = int(s["table"][b, j])
                lo, hi = max(t - n, j * ps), min(t, (j + 1) * ps)
                x = s[name][at + lo - (t - n):at + hi - (t - n)].double().transpose(0, 1)
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


def _logits(case, s, numbers, b, t, n, at):
    """Scores [heads, n, group, t] of sequence b, what is hidden at -inf."""
    hk, d = case["hk"], case["d"]
    K = _sequence(s, numbers, b, t)
    q = s["q"][at:at + n].double().view(n, hk, -1, d).transpose(0, 1)
    x = torch.einsum("hngd,htd->hngt", q, K) / math.sqrt(d)
    if case["causal"]:
        hidden = torch.ones(n, t, dtype=torch.bool, device="cuda").triu(t - n + 1)
        x.masked_fill_(hidden[:, None], -math.inf)
    return x


def _exact_attend(case, s, total, new, starts):
    K, V = _numbers(s, "k"), _numbers(s, "v")
    o, lse = [], []
    for b, (t, n, at) in enumerate(zip(total, new, starts)):
        x = _logits(case, s, K, b, t, n, at)
        z = torch.logsumexp(x, -1)
        w = torch.einsum("hngt,htd->hngd", torch.exp(x - z[..., None]), _sequence(s, V, b, t))
        o.append(w.transpose(0, 1).flatten(1, 2))
        lse.append(z.transpose(0, 1).flatten(1, 2).t())
    return {"o": torch.cat(o), "lse": torch.cat(lse, 1)}


def _exact_weigh(case, s, total, new, starts):
    K = _numbers(s, "k")
    out = s["prev"].double()
    for b, (t, n, at) in enumerate(zip(total, new, starts)):
        x = _logits(case, s, K, b, t, n, at)
        z = s["lse"][:, at:at + n].double().t().view(n, case["hk"], -1).transpose(0, 1)
        out[b, :, :t] += torch.exp(x - z[..., None]).sum((1, 2))
    return {"weights": out}


def _exact_evict(case, s, total, new, starts):
    """Which are kept has no other value in 64 bits; the moved numbers before they are rounded have."""
    ps, hk = case["page"], case["hk"]
    lists = []
    for b, t in enumerate(total):
        keep = _kept(case, t)
        tail = min(case["recent"], keep)
        w = s["weights"][b, :, :t - tail].double().cpu().numpy()
        by = (-w).argsort(axis=-1, kind="stable")[:, :keep - tail]
        old = torch.from_numpy(by.copy()).sort(-1).values
        lists.append(torch.cat((old, torch.arange(t - tail, t).expand(hk, tail)), 1).cuda())
    h = torch.arange(hk, device="cuda")[:, None]
    weights = torch.zeros(s["new_weights"].shape, dtype=torch.float64, device="cuda")
    out = {"kept": None, "new_total": None, "new_weights": weights}
    for b, at in enumerate(lists):
        weights[b, :, :at.shape[1]] = s["weights"][b].double()[h, at]
    for name in ("k", "v"):
        codes = s["dst_%s_pages" % name].view(torch.float8_e4m3fn).double()
        scale = s["dst_%s_scale" % name].double()
        numbers, was = _numbers(s, name), s[name + "_scale"].double()
        for b, at in enumerate(lists):
            page = s["table"][b].long()[at // ps]
            for j in range(-(-at.shape[1] // ps)):
                part, here = at[:, j * ps:(j + 1) * ps], page[:, j * ps:(j + 1) * ps]
                unit = was[here, h].amax(1)
                dst = int(s["dst_table"][b, j])
                codes[dst, :, :part.shape[1]] = numbers[here, h, part % ps] / unit[:, None, None]
                scale[dst] = unit
        out["dst_%s_pages" % name], out["dst_%s_scale" % name] = codes, scale
    return out
