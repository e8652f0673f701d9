"""Rotary positions on the GPU against the fp64 oracle.

Tolerance.  The turn is exact to 2^-33; its fp32 value (at most 1/2) is off by
2^-26 at most, so the angle by 2 pi 2^-26 < 1e-7; sine and cosine add 2 ulp
(2^-23), each product and the sum one rounding of 2^-24.  So each result is within
m (|x| + |y|) (1e-7 + 2^-22 + 2^-23) < 5e-7 m (|x| + |y|) of the exact one, m the
result factor; a bf16 result is rounded once more, by at most 2^-8 of its value.
"""
import numpy as np
import pytest
import torch

from block_sparse_masked_mask_gb300 import api
from oracle import cache as C

pytestmark = pytest.mark.gpu

SCALINGS = {"none": {}, "linear": dict(scaling="linear", factor=4.0), "ntk": dict(scaling="ntk", factor=8.0),
            "ramp": dict(scaling="ramp", factor=16.0, original_context=4096, alpha=1.0, beta=32.0)}


def bound(x, y, theta, interleaved, m, dtype):
    """Elementwise tolerance for y = rotation of x (fp64 arrays)."""
    n = len(theta)
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    tol = np.zeros(x.shape)
    both = 5e-7 * m * (np.abs(x[..., a]) + np.abs(x[..., b]))
    tol[..., a], tol[..., b] = both, both
    if dtype == torch.bfloat16:
        turned = np.zeros(x.shape[-1], bool)
        turned[a], turned[b] = True, True
        tol = np.where(turned, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(y), 0)
    return tol


def check(x, got, positions, plan_args, inverse=False):
    kw = dict(plan_args)
    rot, base, inter = kw.pop("rotary_dim"), kw.pop("base", 10000.0), kw.pop("interleaved", False)
    theta, m = C.rope_angles(rot, base, **kw)
    ref = C.rope(x.double().cpu().numpy(), positions, theta, inter, m, inverse)
    tol = bound(x.double().cpu().numpy(), ref, theta, inter, m, x.dtype)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), f"max err {err.max()}, worst ratio {(err / np.maximum(tol, 1e-300)).max()}"


def rows(T, H, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, H, D), generator=g).to(dtype).cuda()


@pytest.mark.parametrize("scaling", sorted(SCALINGS))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot", [(32, 2), (32, 32), (64, 6), (64, 40), (128, 128), (128, 20), (128, 64), (128, 126)])
def test_rotation_and_its_inverse(D, rot, dtype, interleaved, scaling):
    if scaling == "ntk" and rot == 2:
        pytest.skip("the raised base needs more than one pair")
    T, Hq, Hk = 37, 5, 2
    args = dict(rotary_dim=rot, interleaved=interleaved, **SCALINGS[scaling])
    plan = api.attn_rope_plan(**args)
    q, k = rows(T, Hq, D, dtype, 1), rows(T, Hk, D, dtype, 2)
    pos = torch.randint(0, 1 << 17, (T,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    pos[:4] = torch.tensor([0, 2 ** 31 - 1, -2 ** 31, -5], dtype=torch.int32)
    for inverse in (False, True):
        yq, yk = api.attn_rope(q, k, plan, positions=pos.cuda(), inverse=inverse)
        check(q, yq, pos.numpy(), args, inverse)
        check(k, yk, pos.numpy(), args, inverse)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 0), (1, 32, 8), (2, 1, 1), (700, 3, 1), (4099, 32, 32), (3000, 1, 0)])
def test_sizes_and_positions_from_the_sequences(T, Hq, Hk):
    """Positions by cu_seqlens and by lengths, empty sequences among them; the
    rows behind the last sequence keep what they held."""
    D, args = 64, dict(rotary_dim=64)
    plan = api.attn_rope_plan(**args)
    q = rows(T + 3, Hq, D, torch.float32, 4)
    k = rows(T + 3, Hk, D, torch.float32, 5) if Hk else None
    cuts = sorted([0, 0, T // 3, T // 3, T // 2, T])
    cu = torch.tensor(cuts, dtype=torch.int32)
    n = np.diff(cuts)
    lens = torch.tensor([int(x) + 1000 * i for i, x in enumerate(n)], dtype=torch.int32)
    owner = np.repeat(np.arange(len(n)), n)
    place = np.arange(T) - np.asarray(cuts)[owner]
    for seq_lens, pos in ((None, place), (lens.cuda(), place + 1000 * owner)):
        qo = torch.full_like(q, 7.0)
        ko = None if k is None else torch.full_like(k, 7.0)
        yq, yk = api.attn_rope(q, k, plan, cu_seqlens=cu.cuda(), seq_lens=seq_lens, q_out=qo, k_out=ko)
        assert yq is qo and yk is ko
        check(q[:T], yq[:T], pos, args)
        assert (yq[T:] == 7).all()
        if k is not None:
            check(k[:T], yk[:T], pos, args)
            assert (yk[T:] == 7).all()


@pytest.mark.parametrize("dtype,offset", [(torch.bfloat16, 0), (torch.bfloat16, 1), (torch.float32, 2)])
def test_slices_of_one_projection_and_in_place(dtype, offset):
    """q and k as slices of a wider projection, at any element offset, and
    rotated in place; what lies around them is left alone."""
    T, Hq, Hk, D = 65, 4, 2, 64
    plan_args = dict(rotary_dim=48, interleaved=True)
    plan = api.attn_rope_plan(**plan_args)
    wide = rows(T, 1, (Hq + 2 * Hk) * D + 8, dtype, 6)[:, 0]
    flat = wide[:, offset:offset + (Hq + 2 * Hk) * D]
    q, k = flat[:, :Hq * D].unflatten(1, (Hq, D)), flat[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    before, q0, k0 = wide.clone(), q.clone(), k.clone()
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 3
    yq, yk = api.attn_rope(q, k, plan, positions=pos)
    assert torch.equal(wide, before)
    api.attn_rope(q, k, plan, positions=pos, q_out=q, k_out=k)
    assert torch.equal(q, yq) and torch.equal(k, yk)
    check(q0, q, pos.cpu().numpy(), plan_args)
    check(k0, k, pos.cpu().numpy(), plan_args)
    rest = torch.ones_like(wide, dtype=torch.bool)
    rest[:, offset:offset + (Hq + Hk) * D] = False
    assert torch.equal(wide[rest], before[rest])


def test_gradient_by_differences():
    """The rotation is linear: L = <R x, g> changes by exactly <R e, g> h along e,
    which is (R^T g) e, the inverse rotation's output.  Each rotated number is off
    by 5e-7 m (|x| + |y|) <= 6e-6 here (values below 5, m < 1.14); two of them at
    two places, times |g| < 5: 1.2e-4."""
    T, D = 9, 32
    plan = api.attn_rope_plan(24, interleaved=True, scaling="ramp", factor=4.0, original_context=2048)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 977
    x, g = rows(T, 2, D, torch.float32, 7), rows(T, 2, D, torch.float32, 8)
    grad, _ = api.attn_rope(g, None, plan, positions=pos, inverse=True)
    for d in (0, 1, 10, 23, 24, 31):
        up, down = x.clone(), x.clone()
        up[..., d] += 0.5
        down[..., d] -= 0.5
        yu, yd = (api.attn_rope(z, None, plan, positions=pos)[0].double() for z in (up, down))
        diff = ((yu - yd) * g.double()).sum(-1)
        assert (diff - grad[..., d].double()).abs().max() <= 1.2e-4
    y, _ = api.attn_rope(x, None, plan, positions=pos)
    lhs, rhs = (y.double() * g.double()).sum(), (x.double() * grad.double()).sum()
    pair = lambda z: z.abs().double()[..., :24].unflatten(-1, (12, 2)).sum(-1)
    assert abs(lhs - rhs) <= 2 * 5e-7 * 1.14 * (pair(x) * pair(g)).sum()


def test_far_positions_are_reduced_exactly():
    """At 2^31 - 1 an fp32 angle would be off by many turns."""
    D, args = 128, dict(rotary_dim=128, base=500000.0)
    plan = api.attn_rope_plan(**args)
    pos = torch.tensor([2 ** 31 - 1, 2 ** 30 + 1, 10 ** 9 + 7, 123456789], dtype=torch.int32)
    q = rows(4, 2, D, torch.float32, 9)
    theta, m = C.rope_angles(128, 500000.0)
    ref = C.rope(q.double().cpu().numpy(), pos.numpy(), theta)
    got = api.attn_rope(q, None, plan, positions=pos.cuda())[0].double().cpu().numpy()
    # the fp64 angle itself is off by 2^31 2^-53 theta, and the plan's turn by 2^-53 of itself:
    # together under 2e-6 with theta <= 1
    x = q.double().cpu().numpy()
    tol = bound(x, ref, theta, False, m, torch.float32) + 2e-6 * (np.abs(x) + np.abs(np.roll(x, 64, -1)))
    assert (np.abs(got - ref) <= tol).all()


def test_training_step_with_rotated_queries_and_keys():
    """attn_rope -> attn_fwd -> attn_bwd -> inverse, against the fp64 oracle
    (the backward's bars: 2^-6 of the largest element, 2^-8 in the mean; the
    rotation's own rounding to bf16 on both ways adds one 2^-8 each, so twice those)."""
    import oracle
    from block_sparse_masked_mask_gb300 import workloads as W
    w = W.random_workload(5, "shared_prefix", [300, 129], num_heads=2, head_dim=64)
    dm = w.device_meta()
    # suffixes of a shared prefix continue its positions
    seg = torch.from_numpy(w.seg)
    pos = torch.arange(w.total_tokens, dtype=torch.int32) % 173
    plan = api.attn_rope_plan(64)
    theta, _ = C.rope_angles(64, 10000.0)
    kw = w.api_kwargs(dm)
    bm = api.attn_block_mask_build(w.kind, dm["cu_seqlens"], w.total_tokens, w.max_seqlen, **kw)
    q, k = api.attn_rope(w.q.cuda(), w.k.cuda(), plan, positions=pos.cuda())
    o, lse = api.attn_fwd(q, k, w.v.cuda(), bm, w.kind, dm["cu_seqlens"], w.max_seqlen, **kw)
    do = W.grad_output(w)
    dq, dk, dv = api.attn_bwd(q, k, w.v.cuda(), o, lse, do.cuda(), bm, w.kind, dm["cu_seqlens"], w.max_seqlen, **kw)
    dq, dk = api.attn_rope(dq, dk, plan, positions=pos.cuda(), inverse=True)
    assert api.attn_get_status(bm) == api.ATTN_OK
    # the oracle's q and k are the rotated ones as the library rounds them
    rq, rk = (torch.from_numpy(C.rope(x.double().numpy(), pos.numpy(), theta)).to(torch.bfloat16) for x in (w.q, w.k))
    ref = oracle.attention_backward(rq, rk, w.v, do, w.kind, w.cu_seqlens, w.meta())
    for got, r, turned in zip((dq, dk, dv), ref, (True, True, False)):
        r = C.rope(r, pos.numpy(), theta, inverse=True) if turned else r
        err = np.abs(got.double().cpu().numpy() - r)
        assert err.max() <= 2 * 2.0 ** -6 * np.abs(r).max()
        assert err.sum() <= 2 * 2.0 ** -8 * np.abs(r).sum()
    assert seg.numel() == w.total_tokens


def test_captured_replay_and_other_stream():
    T, D = 50, 64
    plan = api.attn_rope_plan(64)
    q, k = rows(T, 4, D, torch.bfloat16, 10), rows(T, 2, D, torch.bfloat16, 11)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    yq, yk = torch.empty_like(q), torch.empty_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    api.attn_rope(q, k, plan, positions=pos, q_out=yq, k_out=yk, stream=side)
    side.synchronize()
    first = yq.clone(), yk.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.attn_rope(q, k, plan, positions=pos, q_out=yq, k_out=yk)
    yq.zero_()
    yk.zero_()
    graph.replay()
    assert torch.equal(yq, first[0]) and torch.equal(yk, first[1])
    q.mul_(2)
    pos.add_(7)
    graph.replay()
    check(q, yq, pos.cpu().numpy(), dict(rotary_dim=64))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot", [(32, 2), (32, 30), (64, 34), (128, 4), (128, 52), (128, 102), (128, 126)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_rotated_widths_that_no_access_divides(D, rot, dtype, interleaved):
    """What lies behind the rotated dimensions is copied bit for bit, infinities and NaN too;
    in place as well."""
    T, H = 37, 3
    x = torch.randn((T, H, D), generator=torch.Generator().manual_seed(rot)).to(dtype)
    x[::3, :, rot:] = float("inf")
    x[1::3, :, rot:] = float("nan")
    positions = torch.arange(T, dtype=torch.int32) * 1000
    plan = api.attn_rope_plan(rot, interleaved=interleaved)
    y, _ = api.attn_rope(x.cuda(), None, plan, positions=positions.cuda())
    same = x.cuda()
    api.attn_rope(same, None, plan, positions=positions.cuda(), q_out=same)
    as_ints = torch.int16 if dtype == torch.bfloat16 else torch.int32
    assert torch.equal(same.view(as_ints), y.view(as_ints))
    y = y.cpu()
    assert torch.equal(y[..., rot:].contiguous().view(as_ints), x[..., rot:].contiguous().view(as_ints))
    part = x.clone()
    part[..., rot:] = 0
    z, _ = api.attn_rope(part.cuda(), None, plan, positions=positions.cuda())
    assert torch.equal(y[..., :rot], z.cpu()[..., :rot])
    back, _ = api.attn_rope(y.cuda(), None, plan, positions=positions.cuda(), inverse=True)
    # two rotations: per element two products and a sum, twice, on values up to sqrt(2) max |x|,
    # sines and cosines to 2^-22, each result rounded once
    half_step = torch.finfo(dtype).eps / 2
    bound = 2 * (half_step + 2 * 2.0 ** -22) * 2 * x[..., :rot].double().abs().max()
    assert (back.cpu()[..., :rot].double() - x[..., :rot].double()).abs().max() <= bound
