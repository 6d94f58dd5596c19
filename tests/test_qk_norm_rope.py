"""Norm and rotation of queries and keys against their definition in 64 bits.

Tolerances, u = 2^-24.  A row's sum of squares (256 terms in a tree of depth 8 over sums of 8),
its root, the scaling by r and w, the angle (2^-31 of a turn, rounded to fp32: pi u) and the
rotation's two products are each off by at most a few u of the pair's size: together below
32 u = 2^-19 of the larger value of the pair, which rows of unit scale bound by
max(RMS, |value|) times 8; 2^-16 of max(RMS, |value|) in all.  In the gradient the two terms
of dx can cancel; they are each at most the size of the gradient row, which the same bound
covers with twice the terms: 2^-15.  bf16 outputs add half a step, 2^-8 of the value.  A weight
gradient is an fp32 sum of n rows in runs: at most n u of its terms' sizes, sqrt(n) u for
random signs; with n <= 2^13 the bound 2^13 u = 2^-11 of the sum's root mean square holds.
"""
import ctypes
import math

import pytest
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def dr():
    import gated_delta_rule_15_gb300.dr as m
    return m


SCALINGS = [None, dict(kind="linear", factor=4.0),
            dict(kind="by_parts", factor=16.0, original=8192.0, low=1.0, high=32.0)]


def frequencies(rot, base, scaling):
    fs = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling and scaling["kind"] == "linear":
            f /= scaling["factor"]
        elif scaling:
            turns = scaling["original"] * f / (2 * math.pi)
            w = min(1.0, max(0.0, (turns - scaling["low"]) / (scaling["high"] - scaling["low"])))
            f = f * w + f * (1 - w) / scaling["factor"]
        fs.append(f)
    return torch.tensor(fs, dtype=torch.float64)


def define(x, w, pos, freq, norm, layout, eps, scale):
    """[rows, H, d] in 64 bits; differentiable."""
    d, rot = x.shape[-1], 2 * len(freq)
    if norm != "none":
        ss = (x * x).sum(-1, keepdim=True)
        x = x / torch.sqrt(ss / (d if norm == "rms" else 1) + eps)
    if w is not None:
        x = x * w
    ang = pos.double()[:, None] * freq
    c, s = scale * ang.cos()[:, None], scale * ang.sin()[:, None]
    i = torch.arange(rot // 2)
    a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def check(got, ref, tol, what, bf16):
    got = got.double().cpu().reshape(ref.shape)
    rms = ref.square().mean().sqrt().clamp(min=1e-30)
    bound = tol * torch.maximum(ref.abs(), rms) + (2.0 ** -8 * ref.abs() if bf16 else 0)
    worst = ((got - ref).abs() / bound).max().item()
    assert worst <= 1, f"{what}: {worst:.3f} of the bound"


def run_case(dr, n, Hq, Hk, d, rot, dtype, norm, layout, scaling, *, fused=False, far=False, weights=None, scale=1.0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    weights = norm == "rms" if weights is None else weights
    qkv = (torch.randn((n, Hq + 2 * Hk, d), generator=gen) * (0.25 + 3.75 * torch.rand((n, 1, 1), generator=gen))).to(dt)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=gen), 1 + 0.2 * torch.randn(d, generator=gen)) if weights else (None, None))
    pos = torch.randint(-(1 << 20), 1 << 31, (n,), generator=gen) if far else torch.arange(n) + 17
    base = 500000.0 if far else 10000.0
    dq, dk = (torch.randn((n, h, d), generator=gen).to(dt) for h in (Hq, Hk))
    leaves = [x.double().detach().clone().requires_grad_() for x in (q, k)]
    ws = [None if w is None else w.double().requires_grad_() for w in (wq, wk)]
    freq = frequencies(rot, base, scaling)
    ref = [define(x, w, pos, freq, norm, layout, 1e-6, scale) for x, w in zip(leaves, ws)]
    sum((r * g.double()).sum() for r, g in zip(ref, (dq, dk))).backward()
    cu = lambda x: None if x is None else x.cuda()
    c = qkv.cuda()
    qc, kc = (c[:, :Hq], c[:, Hq:Hq + Hk]) if fused else (c[:, :Hq].contiguous(), c[:, Hq:Hq + Hk].contiguous())
    table = dr.rope_table(rot, base=base, scaling=scaling)
    kw = dict(positions=pos.cuda() if far else None, offset=17, norm=norm, wq=cu(wq), wk=cu(wk), layout=layout, rot_scale=scale)
    if rot == 0:
        table = None
    yq, yk = dr.qk_norm_rope(qc, kc, table, **kw)
    bf = dtype == "bf16"
    check(yq, ref[0].detach(), 2.0 ** -16, "q", bf)
    check(yk, ref[1].detach(), 2.0 ** -16, "k", bf)
    gq, gk, gwq, gwk = dr.qk_norm_rope_bwd(qc, kc, table, dq.cuda(), dk.cuda(), **kw)
    check(gq, leaves[0].grad, 2.0 ** -15, "dq", bf)
    check(gk, leaves[1].grad, 2.0 ** -15, "dk", bf)
    if weights:
        check(gwq, ws[0].grad, 2.0 ** -11, "dwq", False)
        check(gwk, ws[1].grad, 2.0 ** -11, "dwk", False)
    else:
        assert gwq is None and gwk is None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("norm", ["none", "l2", "rms"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 32), (128, 0), (256, 256), (256, 112)])
def test_widths_and_layouts(dr, d, rot, layout, norm, dtype):
    run_case(dr, 37, 3, 2, d, rot, dtype, norm, layout, None, seed=d + rot)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions_and_scalings(dr, layout, scaling, dtype):
    """Any 64-bit position, negative ones among them: below 2^31 the 64-bit reference's own
    product is off by 2^31 2^-53 radians."""
    run_case(dr, 300, 2, 1, 128, 128, dtype, "rms", layout, scaling, far=True, scale=1.25, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("n,Hq,Hk", [(1, 1, 1), (1, 40, 8), (5, 3, 3), (64, 32, 8), (1000, 6, 2), (8000, 1, 1)])
def test_rows_and_heads(dr, n, Hq, Hk):
    """One token, few tokens (heads are split over the GPU), many; parts of a fused row."""
    run_case(dr, n, Hq, Hk, 128, 128, "bf16", "rms", "half", None, fused=True, seed=n)
    run_case(dr, n, Hq, Hk, 64, 32, "f32", "l2", "interleaved", None, fused=True, weights=True, seed=n)


@pytest.mark.gpu
def test_rows_of_zeros_and_huge_rows(dr):
    """eps keeps a zero row zero and its gradient finite; a row of 1e18 still normalises in the
    L2 sense (its squares sum below the largest fp32 number)."""
    x = torch.zeros(4, 2, 64).cuda()
    x[2:] = 1e17
    t = dr.rope_table(64)
    for norm in ("l2", "rms"):
        y, _ = dr.qk_norm_rope(x, None, t, norm=norm)
        assert (y[:2] == 0).all() and torch.isfinite(y).all() and (y[2:].norm(dim=-1) > 0.9).all()
        g, _, _, _ = dr.qk_norm_rope_bwd(x, None, t, torch.ones_like(x), None, norm=norm)
        assert torch.isfinite(g[:2]).all()


@pytest.mark.gpu
def test_batched_positions_and_no_keys(dr):
    """[B, T, H, d] without positions: each sequence counts from the offset; k may be absent."""
    x = torch.randn(3, 50, 2, 128).cuda()
    t = dr.rope_table(128)
    a, none = dr.qk_norm_rope(x, None, t, offset=1000, norm="none")
    assert none is None
    pos = (torch.arange(50) + 1000).cuda()
    for b in range(3):
        want, _ = dr.qk_norm_rope(x[b], None, t, positions=pos, norm="none")
        assert torch.equal(a[b], want)


@pytest.mark.gpu
def test_in_place_and_into_a_fused_row(dr):
    n, Hq, Hk, d = 70, 4, 2, 128
    qkv = torch.randn(n, Hq + 2 * Hk, d).cuda().bfloat16()
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    t = dr.rope_table(d)
    kw = dict(norm="rms", wq=torch.rand(d).cuda(), wk=torch.rand(d).cuda())
    yq, yk = dr.qk_norm_rope(q, k, t, **kw)
    gq, gk, gwq, gwk = dr.qk_norm_rope_bwd(q, k, t, yq, yk, **kw)
    dqkv = torch.full_like(qkv, 5.0)
    a = dr.qk_norm_rope_bwd(q, k, t, yq, yk, dq=dqkv[:, :Hq], dk=dqkv[:, Hq:Hq + Hk], **kw)
    assert torch.equal(dqkv[:, :Hq], gq) and torch.equal(dqkv[:, Hq:Hq + Hk], gk) and (dqkv[:, Hq + Hk:] == 5).all()
    assert torch.equal(a[2], gwq) and torch.equal(a[3], gwk)
    v = qkv[:, Hq + Hk:].clone()
    dr.qk_norm_rope(q, k, t, q_out=q, k_out=k, **kw)
    assert torch.equal(q, yq) and torch.equal(k, yk) and torch.equal(qkv[:, Hq + Hk:], v)


@pytest.mark.gpu
def test_nan_stays_in_its_row(dr):
    q = torch.randn(9, 3, 64).cuda()
    q[4, 1, 7] = float("nan")
    y, _ = dr.qk_norm_rope(q, None, dr.rope_table(64))
    bad = torch.isnan(y).any(-1)
    assert bad[4, 1] and bad.sum() == 1


@pytest.mark.gpu
def test_streams_and_graph(dr):
    q, k = torch.randn(200, 8, 128).cuda().bfloat16(), torch.randn(200, 4, 128).cuda().bfloat16()
    t, w = dr.rope_table(128), torch.rand(128).cuda()
    run = lambda **o: (*dr.qk_norm_rope(q, k, t, wq=w, wk=w, **o), *dr.qk_norm_rope_bwd(q, k, t, q, k, wq=w, wk=w, **o))
    want = run()
    torch.cuda.synchronize()
    got = [run(stream=s) for s in (torch.cuda.Stream(), torch.cuda.Stream())]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = run()
    q.copy_(torch.randn(200, 8, 128).cuda())
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(run(), res))


@pytest.mark.gpu
@pytest.mark.parametrize("norm", ["l2", "rms"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,Hq,Hk,d", [(37, 3, 2, 128), (37, 3, 2, 64), (1, 5, 3, 128), (1003, 5, 3, 64), (5000, 7, 1, 128), (3, 1, 1, 256)])
def test_weight_gradients_without_eps(dr, n, Hq, Hk, d, dtype, norm):
    """eps = 0 with rows that are not zero: lanes without a row of their own (odd numbers of rows,
    uneven runs of heads) add nothing to the weights' gradients."""
    gen = torch.Generator().manual_seed(n + d)
    x = [torch.randn((n, h, d), generator=gen).to(DT[dtype]) for h in (Hq, Hk)]
    g = [torch.randn((n, h, d), generator=gen).to(DT[dtype]) for h in (Hq, Hk)]
    w = [1 + 0.2 * torch.randn(d, generator=gen) for _ in range(2)]
    leaves, ws = ([t.double().requires_grad_() for t in ts] for ts in (x, w))
    freq = frequencies(d // 2, 10000.0, None)
    ref = [define(a, b, torch.arange(n), freq, norm, "half", 0.0, 1.0) for a, b in zip(leaves, ws)]
    sum((r * t.double()).sum() for r, t in zip(ref, g)).backward()
    table = dr.rope_table(d // 2)
    cu = [[t.cuda() for t in ts] for ts in (x, g, w)]
    kw = dict(norm=norm, wq=cu[2][0], wk=cu[2][1], eps=0.0)
    y = dr.qk_norm_rope(*cu[0], table, **kw)
    got = dr.qk_norm_rope_bwd(*cu[0], table, *cu[1], **kw)
    bf = dtype == "bf16"
    for i, s in enumerate("qk"):
        check(y[i], ref[i].detach(), 2.0 ** -16, s, bf)
        check(got[i], leaves[i].grad, 2.0 ** -15, "d" + s, bf)
        check(got[2 + i], ws[i].grad, 2.0 ** -11, "dw" + s, False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(64, 0), (64, 16), (128, 48), (256, 128)])
def test_values_behind_the_rotated_part_pass_through(dr, d, rot, layout, dtype):
    """Without a norm they are handed on as they are, infinities and NaN among them, and touch no
    other value; forwards and back."""
    gen = torch.Generator().manual_seed(d + rot)
    x = torch.randn((9, 3, d), generator=gen).to(DT[dtype])
    clean = x.clone().cuda()
    inf = float("inf")
    for i, v in enumerate((inf, -inf, float("nan"), 0.0, inf)):
        x[i, i % 3, rot + (7 * i + 1) % (d - rot)] = v
    x, table = x.cuda(), dr.rope_table(rot) if rot else None
    kw = dict(norm="none", layout=layout, offset=5)
    for run in (lambda t: dr.qk_norm_rope(t, None, table, **kw)[0],
                lambda t: dr.qk_norm_rope_bwd(clean, None, table, t, None, **kw)[0]):
        y, want = run(x), run(clean)
        assert torch.equal(torch.isnan(y), torch.isnan(x))
        assert torch.equal(y[..., rot:].nan_to_num(nan=3.0), x[..., rot:].nan_to_num(nan=3.0))
        assert torch.equal(y[..., :rot], want[..., :rot])


@pytest.mark.gpu
@pytest.mark.parametrize("top", [1 << 20, 1 << 31, 1 << 44, (1 << 63) - 1])
def test_angles_are_the_table_times_the_position(dr, top):
    """The angle is the 64-bit product of position and table entry, whatever the position.  It is
    cut to 2^-32 of a turn and rounded to fp32 (half a turn at most: 2^-26 of a turn), 2 pi
    (2^-26 + 2^-32) < 1e-7; sine and cosine add an ulp or two and the products a rounding
    each, 3 * 2^-23: 2^-21 in all."""
    gen = torch.Generator().manual_seed(top % 1009)
    pos = torch.cat([torch.randint(-top, top, (61,), generator=gen), torch.tensor([-top, -1, 0, 1, top])])
    table = dr.rope_table(64, base=500000.0, device="cpu")
    x = torch.zeros(len(pos), 1, 64)
    x[..., :32] = 1
    y, _ = dr.qk_norm_rope(x.cuda(), None, table.cuda(), positions=pos.cuda(), norm="none")
    turns = torch.tensor([[(p * t) % (1 << 64) / 2.0 ** 64 for t in table.tolist()] for p in pos.tolist()], dtype=torch.float64)
    want = torch.cat([(2 * math.pi * turns).cos(), (2 * math.pi * turns).sin()], -1)[:, None]
    assert (y.double().cpu() - want).abs().max() <= 2.0 ** -21


# ---------------------------------------------------------------- without a GPU
@pytest.mark.parametrize("rot", [0, 16, 64, 128, 256])
@pytest.mark.parametrize("scaling", SCALINGS)
def test_table(dr, rot, scaling):
    """Turns a position in units of 2^-64: the double's 53 bits (pow is off by an ulp or two),
    rounded to a whole number of units (by half of one at most)."""
    t = dr.rope_table(rot, base=10000.0, scaling=scaling, device="cpu")
    want = frequencies(rot, 10000.0, scaling) / (2 * math.pi) * 2.0 ** 64
    assert t.shape == (rot // 2,)
    for a, b in zip(t.tolist(), want.tolist()):
        assert abs((a % (1 << 64)) - b) <= 0.5 + 8 * 2.0 ** -53 * b


@pytest.mark.parametrize("rot,base", [(64, 10000.0), (128, 500000.0), (256, 1.0000001), (16, 1e12)])
@pytest.mark.parametrize("scaling", SCALINGS)
def test_table_against_fifty_digits(dr, rot, base, scaling):
    """Every frequency within 2^-50 of itself and half a unit of 2^-64 turns."""
    from decimal import Decimal as D, localcontext
    with localcontext() as ctx:
        ctx.prec = 50
        pi = D("3.14159265358979323846264338327950288419716939937511")
        got = dr.rope_table(rot, base=base, scaling=scaling, device="cpu").tolist()
        for i, t in enumerate(got):
            f = (D(base).ln() * D(-2 * i) / D(rot)).exp()
            if scaling and scaling["kind"] == "linear":
                f /= D(scaling["factor"])
            elif scaling:
                w = (D(scaling["original"]) * f / (2 * pi) - D(scaling["low"])) / (D(scaling["high"]) - D(scaling["low"]))
                w = min(D(1), max(D(0), w))
                f *= w + (1 - w) / D(scaling["factor"])
            want = f / (2 * pi) * D(2) ** 64
            assert abs(D(t % (1 << 64)) - want) <= D("0.5") + want / D(2) ** 50


@pytest.mark.parametrize("args,status", [
    ((24, 1e4, 0, 0, 0, 0, 0), -2), ((-16, 1e4, 0, 0, 0, 0, 0), -1), ((512, 1e4, 0, 0, 0, 0, 0), -1),
    ((64, 1.0, 0, 0, 0, 0, 0), -1), ((64, float("nan"), 0, 0, 0, 0, 0), -1), ((64, 1e4, 3, 1, 1, 1, 2), -1),
    ((64, 1e4, 1, 0.5, 0, 0, 0), -1), ((64, 1e4, 2, 2, 0, 1, 32), -1), ((64, 1e4, 2, 2, 8192, 32, 32), -1)])
def test_table_refusals(dr, args, status):
    buf = (ctypes.c_uint64 * 128)()
    assert dr.lib().dr_rope_table(*args, ctypes.cast(buf, ctypes.c_void_p)) == status


def _desc(dr, **kw):
    d = dict(n_tok=10, seq_len=0, pos0=0, Hq=4, Hk=2, d=128, rot=64, q_stride=0, k_stride=0, q_out_stride=0,
             k_out_stride=0, dtype=dr.DR_BF16, norm=dr.DR_NORM_RMS, layout=0, reserved=0, eps=1e-6, rot_scale=1.0)
    d.update(kw)
    return dr.QkNormRopeDesc(**d)


@pytest.mark.parametrize("bad,status", [
    (dict(d=96), -2), (dict(rot=24), -2), (dict(rot=144), -1), (dict(rot=-16), -1), (dict(Hq=0), -1), (dict(Hk=-1), -1),
    (dict(n_tok=-1), -1), (dict(dtype=3), -1), (dict(norm=3), -1), (dict(layout=2), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(rot_scale=float("nan")), -1), (dict(reserved=2), -1), (dict(q_stride=511), -1),
    (dict(q_stride=516), -1), (dict(k_out_stride=128), -1), (dict(n_tok=1 << 40), -2)])
def test_bad_descriptors(dr, bad, status):
    n = ctypes.c_size_t(0)
    f = dr.lib().dr_qk_norm_rope_bwd_workspace_bytes
    assert f(ctypes.byref(_desc(dr)), ctypes.byref(n)) == 0 and n.value > 0
    assert f(ctypes.byref(_desc(dr, **bad)), ctypes.byref(n)) == status


no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only without a GPU")


@no_gpu_only
def test_host_side_errors(dr):
    vp = ctypes.c_void_p
    names = ("q", "k", "wq", "wk", "table", "pos", "yq", "yk", "gq", "gk", "dq", "dk", "dwq", "dwk", "ws")
    far = {n: (i + 1) << 36 for i, n in enumerate(names)}
    ptr = lambda o, n: vp(o[n]) if n in o and o[n] is not None else None if n in o else vp(far[n])

    def fwd(desc, **o):
        return dr.lib().dr_qk_norm_rope(ctypes.byref(desc), *[ptr(o, n) for n in names[:8]], None)

    def bwd(desc, wb=1 << 30, **o):
        return dr.lib().dr_qk_norm_rope_bwd(ctypes.byref(desc), *[ptr(o, n) for n in names[:6] + names[8:]], wb, None)

    d = _desc(dr)
    for n in ("q", "k", "table", "yq", "yk"):
        assert fwd(d, **{n: None}) == -1
        assert fwd(d, **{n: far[n] + 4}) == -1
    assert fwd(d, yq=far["k"]) == -1 and fwd(d, yq=far["yk"]) == -1 and fwd(d, yq=far["q"] + 16) == -1
    assert fwd(_desc(dr, q_stride=1024), yq=far["q"]) == -1          # another stride than its input's
    assert fwd(_desc(dr, norm=dr.DR_NORM_NONE)) == -1                # weights without a norm
    for n in ("q", "k", "table", "gq", "gk", "dq", "dk"):
        assert bwd(d, **{n: None}) == -1
    assert bwd(d, dq=far["gq"]) == -1 and bwd(d, dq=far["dk"]) == -1 and bwd(d, dk=far["q"]) == -1
    assert bwd(d, wq=None) == -1                                     # a gradient of no weights
    assert bwd(d, ws=None) == dr.DR_ERR_WORKSPACE and bwd(d, wb=8) == dr.DR_ERR_WORKSPACE
    # dq and dk as parts of one row of 4 + 2 + 2 heads: rows that meet are refused
    f = _desc(dr, q_out_stride=1024, k_out_stride=1024)
    assert bwd(f, dk=far["dq"] + 2 * 500) == -1 and bwd(f, dk=far["dq"] + 2 * 896) == -1
    assert bwd(f, dk=far["dq"] + 2 * 1024 * 3 + 2 * 256) == -1
    assert bwd(_desc(dr, q_out_stride=1024, k_out_stride=2048), dk=far["dq"] + 2 * 512) == -1


@pytest.mark.parametrize("make", [
    lambda x: x[:1].expand(6, 4, 64), lambda x: x[:1].unsqueeze(0).expand(2, 3, 4, 64),
    lambda x: x[:1].unsqueeze(0).expand(6, 1, 4, 64), lambda x: x.as_strided((6, 4, 64), (128, 64, 1)),
    lambda x: x[:3].unsqueeze(0).expand(2, 3, 4, 64)])
def test_rows_that_share_memory_are_refused(dr, make):
    """A broadcast row has stride 0, which the C ABI reads as contiguous rows: behind the tensor's end."""
    x = torch.zeros(6, 4, 64)
    assert dr._rows_of(x, "q") == (6, 4, 64, 256)
    assert dr._rows_of(x[:1].expand(1, 4, 64), "q")[:3] == (1, 4, 64)
    with pytest.raises(ValueError):
        dr._rows_of(make(x), "q")


@no_gpu_only
def test_operands_under_written_rows_are_refused(dr):
    """Weights, table and positions are read by every block; weight gradients and their partial sums
    are written beside the rows."""
    vp = ctypes.c_void_p
    names = ("q", "k", "wq", "wk", "table", "pos", "yq", "yk", "gq", "gk", "dq", "dk", "dwq", "dwk", "ws")
    far = {n: (i + 1) << 36 for i, n in enumerate(names)}

    def fwd(desc, **o):
        return dr.lib().dr_qk_norm_rope(ctypes.byref(desc), *[vp(o.get(n, far[n])) for n in names[:8]], None)

    def bwd(desc, **o):
        return dr.lib().dr_qk_norm_rope_bwd(ctypes.byref(desc), *[vp(o.get(n, far[n])) for n in names[:6] + names[8:]], 1 << 30, None)

    d, f = _desc(dr), _desc(dr, q_out_stride=1024, k_out_stride=1024)     # rows of 8 heads of 128, 4 + 2 of them written
    size = dict(wq=512, wk=512, table=256, pos=80, dwq=512, dwk=512)
    for n in ("wq", "wk", "table", "pos"):
        for y in ("yq", "yk"):
            assert fwd(d, **{n: far[y]}) == -1 and fwd(d, **{n: far[y] + 2 * 256}) == -1 and fwd(d, **{n: far[y] - size[n] + 8}) == -1
            assert fwd(f, **{n: far[y] + 2 * 1024 * 9}) == -1 and fwd(f, **{n: far[y] + 2 * 1024 * 9 - 16}) == -1
    for n in ("wq", "wk", "table", "pos", "dwq", "dwk"):
        for y in ("dq", "dk"):
            assert bwd(d, **{n: far[y]}) == -1 and bwd(d, **{n: far[y] - size[n] + 8}) == -1
            assert bwd(f, **{n: far[y] + 2 * 1024 * 9}) == -1
    assert bwd(d, dwq=far["dwk"]) == -1 and bwd(d, dwq=far["dwk"] + 256) == -1
    n = ctypes.c_size_t(0)
    assert dr.lib().dr_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 512
    for x in ("q", "k", "wq", "wk", "table", "pos", "gq", "gk", "dq", "dk", "dwq", "dwk"):
        assert bwd(d, ws=far[x]) == -1 and bwd(d, ws=far[x] - n.value // 16 * 16 + 16) == -1, x
