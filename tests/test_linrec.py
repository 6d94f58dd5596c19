"""The additive gated linear recurrence: forward, backward and single token against a plain
token loop in 64 bits.

Tolerances.  u = 2^-24 (fp32), 2^-8 = half a bf16 step.  A state or output is a sum of up to
n = min(T, memory) + dk products; fp32 sums of random-sign terms are off by about sqrt(n) u of
their root mean square, at most n u: with n <= 2^12 here the bound 2^12 u = 2.5e-4 of the RMS
holds for the worst element, taken relative to max(RMS, |value|).  A bf16 output adds its
rounding, 2^-8 of the value, and the kernels' bf16 operands (each rounded by at most 2^-8 of its
value, of random sign in sums of many: 3 of them at the worst element's six standard
deviations of 2^-8 / sqrt(3) each) at most 6 sqrt(3) / sqrt(3) 2^-8 = 2.4e-2 of the RMS.
The terms that are rounded are those of the element's own sum, sum_i q_i S_ij over the
row's token: with random signs the root of their squares' sum is the RMS of that token's
row, so the RMS of rows [.., d] is the row's own (tokens next to a large state are much
larger than the others where the decay is strong).
fp32 results of bf16 problems (states, the log-decay gradient) carry the fp32 bound.

The log-decay gradient is <a_t S_{t-1}, dS_t>, formed as <S, dS> at the end of a run of 256 tokens plus
the run's q.dq - k.dk behind t.  Each of those numbers is an fp32 sum of 128 products (off by
about 2 u of its size, random signs) and up to 2 * 256 of them are added: sqrt(512) 2 u < 64 u of
the largest.  Where the decay is so strong that the gradient is small against q.dq and k.dk, that
absolute error is the bound.
"""
import ctypes
import math

import pytest
import torch

F32_TOL = 2.5e-4
BF16_TOL = 2.4e-2
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def dr():
    import gated_delta_rule_15_gb300.dr as m
    return m


def reference(q, k, v, la, s0, cu=None, do=None, ds=None):
    """Token loop in 64 bits over each sequence: out, final state and, with d_out, the
    gradients.  Rows of no sequence are NaN."""
    q, k, v = (x.double().cpu() for x in (q, k, v))
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    a = torch.ones(B, T, H, dtype=torch.float64) if la is None else la.double().cpu().exp()
    spans = [(b, 0, T) for b in range(B)] if cu is None else \
        [(0, int(x), int(y)) for x, y in zip(cu[:-1], cu[1:])]
    N = len(spans)
    nan = float("nan")
    out = torch.full((B, T, H, dv), nan, dtype=torch.float64)
    fin = torch.zeros(N, H, dk, dv, dtype=torch.float64)
    g = None
    if do is not None:
        do = do.double().cpu()
        g = dict(dq=torch.full_like(q, nan), dk=torch.full_like(k, nan), dv=torch.full_like(v, nan),
                 dla=torch.full_like(a, nan), d0=torch.zeros_like(fin))
    for n, (b, lo, hi) in enumerate(spans):
        s = torch.zeros(H, dk, dv, dtype=torch.float64) if s0 is None else s0[n].double().cpu().clone()
        states = [s]
        for t in range(lo, hi):
            s = a[b, t, :, None, None] * s + k[b, t, :, :, None] * v[b, t, :, None, :]
            states.append(s)
            out[b, t] = torch.einsum("hij,hi->hj", s, q[b, t])
        fin[n] = s
        if g is None:
            continue
        d = torch.zeros(H, dk, dv, dtype=torch.float64) if ds is None else ds[n].double().cpu().clone()
        for t in range(hi - 1, lo - 1, -1):
            g["dq"][b, t] = torch.einsum("hij,hj->hi", states[t - lo + 1], do[b, t])
            d = d + q[b, t, :, :, None] * do[b, t, :, None, :]
            g["dk"][b, t] = torch.einsum("hij,hj->hi", d, v[b, t])
            g["dv"][b, t] = torch.einsum("hij,hi->hj", d, k[b, t])
            d = a[b, t, :, None, None] * d
            g["dla"][b, t] = (d * states[t - lo]).sum((-1, -2))
        g["d0"][n] = d
    return out, fin, g


def inputs(B, T, H, dk, dv, dtype, gate=True, N=0, init=True, strength=0.1, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)
    q, k, v, do = rn(B, T, H, dk), rn(B, T, H, dk), rn(B, T, H, dv), rn(B, T, H, dv)
    q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    la = -strength * torch.rand((B, T, H), generator=gen) if gate else None
    M = N or B
    s0, ds = (0.3 * rn(M, H, dk, dv), rn(M, H, dk, dv)) if init else (None, None)
    dt = DT[dtype]
    return dict(q=q.to(dt), k=k.to(dt), v=v.to(dt), la=la, s0=s0, do=do.to(dt), ds=ds)


def cuda(d):
    return {n: None if x is None else x.cuda() for n, x in d.items()}


def dla_slack(d, g):
    """64 u of the largest q.dq or k.dk (reference values; rows of no sequence are NaN)."""
    dots = [(d[x].double() * g["d" + x]).sum(-1).abs() for x in "qk"]
    return 64 * 2.0 ** -24 * max(x[~torch.isnan(x)].max().item() if (~torch.isnan(x)).any() else 0.0 for x in dots)


def check(got, ref, dtype, what, slack=0.0):
    """Worst |got - ref| over max(RMS, |ref|) where ref is a number; the RMS of the row for
    rows of tokens, of all values for states and the log-decay gradient."""
    got = got.double().cpu()
    there = ~torch.isnan(ref)
    assert torch.isfinite(got[there]).all(), what
    if not there.any():
        return
    rows = what.split()[0] in ("out", "dq", "dk", "dv")
    rms = (ref.square().mean(-1, keepdim=True) if rows else ref[there].square().mean()).sqrt().expand(ref.shape)
    err = (((got - ref).abs() - slack).clamp(min=0) / torch.maximum(ref.abs(), rms.clamp(min=1e-30)))[there].max().item()
    tol = F32_TOL if dtype == "f32" else BF16_TOL
    assert err <= tol, f"{what}: {err:.3e} > {tol:.1e}"


SHAPES = [  # B, T, H, dk, dv
    (1, 1, 1, 64, 64), (2, 1, 3, 128, 128), (1, 15, 2, 64, 128), (2, 16, 2, 128, 64), (1, 63, 1, 128, 128),
    (2, 64, 3, 128, 128), (1, 65, 2, 128, 128), (3, 130, 2, 64, 64), (1, 257, 2, 128, 128), (1, 700, 1, 128, 128),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("B,T,H,dk,dv", SHAPES)
def test_forward_and_backward(dr, B, T, H, dk, dv, gate, dtype):
    d = inputs(B, T, H, dk, dv, dtype, gate=gate, seed=T)
    out, fin, g = reference(d["q"], d["k"], d["v"], d["la"], d["s0"], do=d["do"], ds=d["ds"])
    slack = dla_slack(d, g)
    c = cuda(d)
    o, f = dr.linrec_fwd(c["q"], c["k"], c["v"], c["la"], c["s0"])
    check(o, out, dtype, "out")
    check(f, fin, "f32", "final_state")
    dq, dk_, dv_, dla, d0 = dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"], c["ds"])
    for x, n in ((dq, "dq"), (dk_, "dk"), (dv_, "dv")):
        check(x, g[n], dtype, n)
    check(d0, g["d0"], "f32", "d_init_state")
    if gate:
        check(dla, g["dla"], "f32", "d_log_alpha", slack)
    else:
        assert dla is None
    assert dr.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_states(dr, dtype):
    """Zero initial state, no final state's gradient, neither returned."""
    d = inputs(2, 150, 2, 128, 128, dtype, init=False, seed=5)
    out, fin, g = reference(d["q"], d["k"], d["v"], d["la"], None, do=d["do"])
    slack = dla_slack(d, g)
    c = cuda(d)
    o, f = dr.linrec_fwd(c["q"], c["k"], c["v"], c["la"], return_final_state=False)
    assert f is None
    check(o, out, dtype, "out")
    dq, dk_, dv_, dla, d0 = dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], None, c["do"], return_d_init=False)
    assert d0 is None
    for x, n in ((dq, "dq"), (dk_, "dk"), (dv_, "dv")):
        check(x, g[n], dtype, n)
    check(dla, g["dla"], "f32", "d_log_alpha", slack)


PACKED = [  # cu_seqlens, rows
    ([0, 1], 1), ([0, 0, 0], 5), ([0, 64, 64, 65, 200], 200), ([3, 40, 41, 41, 300, 811], 900), ([0, 128, 256], 256),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d_", [64, 128])
@pytest.mark.parametrize("cu,T", PACKED)
def test_packed_sequences(dr, cu, T, d_, dtype):
    """Empty and one-token sequences, ends inside and on tiles; rows of no sequence hold NaN and
    infinity on the way in and are left alone on the way out."""
    N, H = len(cu) - 1, 2
    d = inputs(1, T, H, d_, d_, dtype, N=N, seed=T)
    out, fin, g = reference(d["q"], d["k"], d["v"], d["la"], d["s0"], cu, d["do"], d["ds"])
    slack = dla_slack(d, g)
    for n in ("q", "k", "v", "la", "do"):
        d[n][:, :cu[0]] = float("nan")
        d[n][:, cu[-1]:] = float("inf")
    c = cuda(d)
    cuc = torch.tensor(cu, dtype=torch.int64).cuda()
    o = torch.full_like(c["v"], 7.0)
    _, f = dr.linrec_fwd(c["q"], c["k"], c["v"], c["la"], c["s0"], cu_seqlens=cuc, out=o)
    check(o, out, dtype, "out")
    check(f, fin, "f32", "final_state")
    gr = [torch.full_like(c[n], 7.0) for n in ("q", "k", "v", "la")]
    dq, dk_, dv_, dla, d0 = dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"], c["ds"], cu_seqlens=cuc,
                                          grads=gr)
    for x, n in ((dq, "dq"), (dk_, "dk"), (dv_, "dv")):
        check(x, g[n], dtype, n)
    check(dla, g["dla"], "f32", "d_log_alpha", slack)
    check(d0, g["d0"], "f32", "d_init_state")
    for x in (o, dq, dk_, dv_, dla):
        x = x.float().cpu()
        assert (x[:, :cu[0]] == 7).all() and (x[:, cu[-1]:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_neighbouring_sequences_do_not_leak(dr, dtype):
    """A sequence's results do not change with what its neighbours hold, NaN included."""
    cu = [0, 70, 130, 201]
    d = cuda(inputs(1, 201, 2, 128, 128, dtype, N=3, seed=9))
    cuc = torch.tensor(cu, dtype=torch.int64).cuda()
    run = lambda x: (dr.linrec_fwd(x["q"], x["k"], x["v"], x["la"], x["s0"], cu_seqlens=cuc),
                     dr.linrec_bwd(x["q"], x["k"], x["v"], x["la"], x["s0"], x["do"], x["ds"], cu_seqlens=cuc))
    (o1, f1), g1 = run(d)
    e = {n: x.clone() for n, x in d.items()}
    for n in ("q", "k", "v", "la", "do"):
        e[n][:, :70] = float("nan")
        e[n][:, 130:] = float("inf")
    (o2, f2), g2 = run(e)
    assert torch.equal(o1[:, 70:130], o2[:, 70:130]) and torch.equal(f1[1], f2[1])
    for a, b in zip(g1[:4], g2[:4]):
        assert torch.equal(a[:, 70:130], b[:, 70:130])
    assert torch.equal(g1[4][1], g2[4][1])


@pytest.mark.gpu
def test_offsets_outside_the_rows_are_clamped(dr):
    d = cuda(inputs(1, 100, 1, 128, 128, "bf16", N=3, seed=3))
    bad = torch.tensor([-50, 40, 30, 1 << 40], dtype=torch.int64).cuda()
    good = torch.tensor([0, 40, 40, 100], dtype=torch.int64).cuda()     # 40..30 is empty, 30..100 runs
    o, f = dr.linrec_fwd(d["q"], d["k"], d["v"], d["la"], d["s0"], cu_seqlens=bad)
    o2, f2 = dr.linrec_fwd(d["q"], d["k"], d["v"], d["la"], d["s0"], cu_seqlens=good)
    torch.cuda.synchronize()
    assert torch.equal(f[:2], f2[:2]) and torch.isfinite(f).all()
    assert dr.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("strength", [0.0, 1e-3, 1.0, 5.0, 60.0])
def test_weak_and_strong_decay(dr, strength, dtype):
    """Up to exp(-60 * 64) within a chunk.  The log-decay gradient of strong decays is small:
    its bound is that of its own size."""
    d = inputs(1, 400, 2, 128, 128, dtype, strength=strength, seed=11)
    out, fin, g = reference(d["q"], d["k"], d["v"], d["la"], d["s0"], do=d["do"], ds=d["ds"])
    slack = dla_slack(d, g)
    c = cuda(d)
    o, f = dr.linrec_fwd(c["q"], c["k"], c["v"], c["la"], c["s0"])
    check(o, out, dtype, "out")
    check(f, fin, "f32", "final_state")
    grads = dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"], c["ds"])
    for x, n in zip(grads, ("dq", "dk", "dv", "dla", "d0")):
        check(x, g[n], "f32" if n in ("dla", "d0") else dtype, n, slack if n == "dla" else 0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_full_resets(dr, dtype):
    """log_alpha = -inf forgets everything: the tokens behind a reset do not see those before."""
    d = inputs(1, 300, 2, 128, 128, dtype, seed=13)
    for t in (0, 5, 63, 64, 65, 66, 200, 299):
        d["la"][:, t] = -math.inf
    out, fin, g = reference(d["q"], d["k"], d["v"], d["la"], d["s0"], do=d["do"], ds=d["ds"])
    slack = dla_slack(d, g)
    c = cuda(d)
    o, f = dr.linrec_fwd(c["q"], c["k"], c["v"], c["la"], c["s0"])
    check(o, out, dtype, "out")
    check(f, fin, "f32", "final_state")
    grads = dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"], c["ds"])
    for x, n in zip(grads, ("dq", "dk", "dv", "dla", "d0")):
        check(x, g[n], "f32" if n in ("dla", "d0") else dtype, n, slack if n == "dla" else 0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("strength", [0.1, 1e-3])
@pytest.mark.parametrize("T,H,dk,dv,cu", [
    (4096, 1, 128, 128, None), (3001, 3, 64, 128, None), (5000, 2, 128, 64, None), (6020, 1, 64, 64, [0, 10, 4500, 4500, 6000]),
    (9000, 2, 128, 128, [5, 2000, 2001, 8999])])
def test_long_sequences_in_few_chains(dr, T, H, dk, dv, cu, strength):
    """Long enough for the sequences to be cut into segments that run side by side."""
    N = len(cu) - 1 if cu else 1
    d = inputs(1, T, H, dk, dv, "bf16", N=N if cu else 0, strength=strength, seed=T)
    cuc = None if cu is None else torch.tensor(cu, dtype=torch.int64).cuda()
    desc = dr.LinrecDesc(1, T, H, dk, dv, N if cu else 0, 1, 1, 1, 0)
    import ctypes
    n = ctypes.c_size_t(0)
    assert dr.lib().dr_linrec_fwd_workspace_bytes(ctypes.byref(desc), ctypes.byref(n)) == 0 and n.value > 0
    out, fin, g = reference(d["q"], d["k"], d["v"], d["la"], d["s0"], cu, d["do"], d["ds"])
    slack = dla_slack(d, g)
    c = cuda(d)
    o, f = dr.linrec_fwd(c["q"], c["k"], c["v"], c["la"], c["s0"], cu_seqlens=cuc)
    check(o, out, "bf16", "out")
    check(f, fin, "f32", "final_state")
    grads = dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"], c["ds"], cu_seqlens=cuc)
    for x, n in zip(grads, ("dq", "dk", "dv", "dla", "d0")):
        check(x, g[n], "f32" if n in ("dla", "d0") else "bf16", n, slack if n == "dla" else 0.0)
    assert dr.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,t", [((70, 130, 64), 0), ((70, 130, 64), 77), ((20, 3000, 40), 1500), ((10, 5, 1), 3)])
def test_nan_gate_shows_in_its_sequence(dr, lens, t, dtype):
    """A NaN log decay reaches everything that depends on it, on every path, and no neighbour."""
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T, a, b = cu[-1], cu[1], cu[2]
    c = cuda(inputs(1, T, 2, 64, 128, dtype, N=3, seed=T))
    cuc = torch.tensor(cu, dtype=torch.int64).cuda()
    run = lambda: (*dr.linrec_fwd(c["q"], c["k"], c["v"], c["la"], c["s0"], cu_seqlens=cuc),
                   *dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"], c["ds"], cu_seqlens=cuc))
    want = run()
    c["la"][0, a + t, 1] = float("nan")
    got = run()
    o, f, dq, dk_, dv_, dla, d0 = got
    for x in (o, dq):                                   # rows that read a state behind the gate
        assert torch.isnan(x[0, a + t:b, 1]).all()
    for x in (dk_, dv_):                                # rows whose write passes through it
        assert torch.isnan(x[0, a:a + t, 1]).all()
    assert torch.isnan(f[1, 1]).all() and torch.isnan(d0[1, 1]).all() and torch.isnan(dla[0, a + t, 1])
    for x, y in zip(got, want):
        if x is f or x is d0:
            assert torch.equal(x[[0, 2]], y[[0, 2]]) and torch.equal(x[:, 0], y[:, 0])
        else:
            assert torch.equal(x[:, :a], y[:, :a]) and torch.equal(x[:, b:], y[:, b:]) and torch.equal(x[:, :, 0], y[:, :, 0])
    assert dr.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,cu", [(300, None), (16, None), (3000, None), (300, [0, 5, 66, 300])])
def test_gradient_of_a_reset_is_zero(dr, T, cu, dtype):
    """d_log_alpha = alpha <S, dS> is 0 where alpha is, not the rounding of the sums it comes from."""
    N = len(cu) - 1 if cu else 0
    c = cuda(inputs(1, T, 2, 128, 64, dtype, N=N, seed=T))
    at = [t for t in (0, 5, 15, 63, 64, 65, 200, 255, 256, 299, 2999) if t < T]
    for i, t in enumerate(at):
        c["la"][:, t, 0] = -math.inf if i % 2 else -200.0
    cuc = None if cu is None else torch.tensor(cu, dtype=torch.int64).cuda()
    dla = dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"], c["ds"], cu_seqlens=cuc)[3]
    assert (dla[:, at, 0] == 0).all() and (dla[:, at, 1] != 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("gate", [True, False])
def test_one_long_sequence_among_many_short(dr, gate):
    """More sequences than segments: only the cut ones' states lie in the workspace."""
    lens = [3, 0, 70] * 20 + [2100] + [1, 64, 5] * 15 + [600, 513, 512] + [17] * 9
    cu = torch.tensor([0] + lens).cumsum(0)
    T, N = int(cu[-1]) + 11, len(lens)
    d = inputs(1, T, 2, 64, 128, "bf16", gate=gate, N=N, strength=0.01, seed=T)
    out, fin, g = reference(d["q"], d["k"], d["v"], d["la"], d["s0"], cu.tolist(), d["do"], d["ds"])
    slack = dla_slack(d, g) if gate else 0.0
    c, cuc = cuda(d), cu.cuda()
    o, f = dr.linrec_fwd(c["q"], c["k"], c["v"], c["la"], c["s0"], cu_seqlens=cuc)
    check(o, out, "bf16", "out")
    check(f, fin, "f32", "final_state")
    grads = dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"], c["ds"], cu_seqlens=cuc)
    for x, n in zip(grads, ("dq", "dk", "dv", "dla", "d0")):
        if n != "dla" or gate:
            check(x, g[n], "f32" if n in ("dla", "d0") else "bf16", n, slack if n == "dla" else 0.0)
    assert dr.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_new_buffers_hold_zeros_in_rows_of_no_sequence(dr, dtype):
    """Results that the call allocates can be summed over all rows."""
    cu = [3, 40, 40, 170]
    c = cuda(inputs(1, 200, 2, 64, 128, dtype, N=3, seed=2))
    cuc = torch.tensor(cu, dtype=torch.int64).cuda()
    for _ in range(3):
        junk = [torch.full_like(c[n], float("nan")) for n in ("v", "q", "k", "v", "la", "v")]
        del junk                                        # freed blocks that hold NaN
        o, _ = dr.linrec_fwd(c["q"], c["k"], c["v"], c["la"], c["s0"], cu_seqlens=cuc)
        g = dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"], c["ds"], cu_seqlens=cuc)[:4]
        for x in (o, *g):
            assert (x[:, :cu[0]] == 0).all() and (x[:, cu[-1]:] == 0).all() and torch.isfinite(x).all()
    other = torch.float32 if dtype == "bf16" else torch.bfloat16
    with pytest.raises(dr.DrError):                     # refused before anything is written
        dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"].to(other), c["ds"], cu_seqlens=cuc)
    o, _ = dr.linrec_fwd(c["q"], c["k"], c["v"], c["la"], c["s0"], cu_seqlens=cuc, out_dtype=other)
    assert o.dtype == other and (o[:, :cu[0]] == 0).all() and (o[:, cu[-1]:] == 0).all() and torch.isfinite(o).all()


@pytest.mark.gpu
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("B,T,H,dk,dv", [(3, 4100, 1, 128, 128), (5, 1900, 2, 64, 128), (2, 2049, 3, 128, 64), (7, 1500, 1, 64, 64)])
def test_batches_whose_sequences_are_cut(dr, B, T, H, dk, dv, gate):
    """Sequences that start off any segment's boundary, so that some slots stay empty."""
    n = ctypes.c_size_t(0)
    desc = _desc(dr, B=B, T=T, H=H, dk=dk, dv=dv, gate=int(gate))
    assert dr.lib().dr_linrec_fwd_workspace_bytes(ctypes.byref(desc), ctypes.byref(n)) == 0 and n.value > 0
    d = inputs(B, T, H, dk, dv, "bf16", gate=gate, strength=0.01, seed=T)
    out, fin, g = reference(d["q"], d["k"], d["v"], d["la"], d["s0"], None, d["do"], d["ds"])
    slack = dla_slack(d, g) if gate else 0.0
    c = cuda(d)
    o, f = dr.linrec_fwd(c["q"], c["k"], c["v"], c["la"], c["s0"])
    check(o, out, "bf16", "out")
    check(f, fin, "f32", "final_state")
    grads = dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"], c["ds"])
    for x, m in zip(grads, ("dq", "dk", "dv", "dla", "d0")):
        if m != "dla" or gate:
            check(x, g[m], "f32" if m in ("dla", "d0") else "bf16", m, slack if m == "dla" else 0.0)
    assert dr.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [None, [0, 100, 2600, 2600, 4000]])
def test_cut_sequences_on_streams_and_in_graphs(dr, cu):
    """Two streams at once, and two captured graphs with a workspace each, replayed on new inputs
    side by side, at a length whose segments' states pass through the workspace."""
    N, T = len(cu) - 1 if cu else 1, 4100
    desc, n = _desc(dr, B=1, T=T, H=2, N=N if cu else 0), ctypes.c_size_t(0)
    assert dr.lib().dr_linrec_fwd_workspace_bytes(ctypes.byref(desc), ctypes.byref(n)) == 0 and n.value > 0
    make = lambda seed: cuda(inputs(1, T, 2, 128, 128, "bf16", N=N if cu else 0, strength=0.01, seed=seed))
    cuc = None if cu is None else torch.tensor(cu, dtype=torch.int64).cuda()
    run = lambda c, **o: (*dr.linrec_fwd(c["q"], c["k"], c["v"], c["la"], c["s0"], cu_seqlens=cuc, **o),
                          *dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"], c["ds"], cu_seqlens=cuc, **o))
    first, second = make(1), make(2)
    want = run(first), run(second)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [run(c, stream=s) for c, s in zip((first, second), streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
    held, graphs, res = [make(3), make(4)], [], []
    for c in held:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            res.append(run(c))
    for c, new in zip(held, (first, second)):
        for m in c:
            c[m].copy_(new[m])
    torch.cuda.synchronize()
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for g, w in zip(res, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))
    assert dr.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("strength", [0.1, 5.0, None])
@pytest.mark.parametrize("T,dk,dv,cu", [(700, 128, 128, None), (2100, 64, 128, None), (900, 128, 64, [0, 130, 131, 890])])
def test_bf16_results_are_rounded_once(dr, T, dk, dv, cu, strength):
    """Off by their own rounding, 2^-8 of the value, and what an fp32 result is off by: scores and
    states that enter as two bf16 terms lose 2^-17 each, 6 sqrt(2) 2^-17 / sqrt(3) = 3.8e-5 of the row's RMS
    at the worst element's six standard deviations, beside the 2.5e-4 of fp32 sums."""
    N = len(cu) - 1 if cu else 0
    d = inputs(1, T, 2, dk, dv, "bf16", gate=strength is not None, N=N, strength=strength or 0.0, seed=T)
    out, fin, g = reference(d["q"], d["k"], d["v"], d["la"], d["s0"], cu, d["do"], d["ds"])
    c, cuc = cuda(d), None if cu is None else torch.tensor(cu, dtype=torch.int64).cuda()
    o, _ = dr.linrec_fwd(c["q"], c["k"], c["v"], c["la"], c["s0"], cu_seqlens=cuc)
    grads = dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"], c["ds"], cu_seqlens=cuc)
    for x, ref, n in ((o, out, "out"), *((y, g[m], m) for y, m in zip(grads, ("dq", "dk", "dv")))):
        there = ~torch.isnan(ref)
        rms = ref.square().mean(-1, keepdim=True).sqrt().expand(ref.shape)
        bound = 2.0 ** -8 * ref.abs() + (F32_TOL + 3.8e-5) * torch.maximum(rms, ref.abs())
        assert (((x.double().cpu() - ref).abs() / bound)[there] <= 1).all(), n
    assert dr.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,dk,dv", [(2, 1024, 128, 128), (3, 700, 64, 128), (2, 900, 128, 64), (4, 515, 64, 64)])
def test_log_decay_gradient_of_bf16_rows_is_an_fp32_result(dr, B, T, dk, dv):
    """In the 2-norm.  A token's two terms are sums in dk / 16 (dv / 16) <= 8 tensor-core steps on the large
    operand term, each of which cuts off less than 2^-23 of the sum so far: below 2^-20 = 9.6e-7, of one
    sign, and the states in them carry 3e-7; sums of such terms keep the relative size.  The random
    part, 2 u of each of up to 512 terms, stands against a gradient of the size of the decay's memory,
    some 20 terms: sqrt(512 / 20) 2 u = 6e-7.  1.9e-6 in all."""
    d = inputs(B, T, 2, dk, dv, "bf16", seed=T)
    _, _, g = reference(d["q"], d["k"], d["v"], d["la"], d["s0"], None, d["do"], d["ds"])
    c = cuda(d)
    dla = dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"], c["ds"])[3].double().cpu()
    assert (dla - g["dla"]).norm() <= 1.9e-6 * g["dla"].norm()


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,H", [(4, 255, 2), (2, 1000, 2), (8, 255, 3)])
def test_log_decay_gradient_of_fp32_rows(dr, B, T, H):
    """In the 2-norm.  A token's terms are off by 3.2 u (16 products in a row, sqrt(16 / 6) u, the tree over
    them and over the columns, u, and the state's own rounding over its memory of 20 tokens, sqrt(20 / 3) u); up
    to 2 * 128 of them are added, against a gradient of the size of 20: sqrt(256 / 20) 3.2 u = 6.8e-7.  The
    state's part is the same for neighbouring tokens and adds up faster, by 1.32 at most: 9e-7."""
    d = inputs(B, T, H, 128, 128, "f32", seed=T)
    _, _, g = reference(d["q"], d["k"], d["v"], d["la"], d["s0"], None, d["do"], d["ds"])
    c = cuda(d)
    dla = dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"], c["ds"])[3].double().cpu()
    assert (dla - g["dla"]).norm() <= 9e-7 * g["dla"].norm()


@pytest.mark.gpu
def test_gradients_against_differences(dr):
    """Directional derivatives of <do, out> + <ds, final> by central differences in fp32: the
    function is quadratic in q, k, v and the state, so the quotient is exact up to its
    rounding, about 2 sqrt(n) u L / step with n = 10^5 terms of L and step 2^-5: 2e-3."""
    d = cuda(inputs(1, 90, 2, 64, 64, "f32", seed=21))
    loss = lambda x: sum((a.double() * b.double()).sum() for a, b in
                         zip(dr.linrec_fwd(x["q"], x["k"], x["v"], x["la"], x["s0"]), (d["do"], d["ds"])))
    grads = dr.linrec_bwd(d["q"], d["k"], d["v"], d["la"], d["s0"], d["do"], d["ds"])
    gen = torch.Generator(device="cuda").manual_seed(4)
    for n, gr in zip(("q", "k", "v", "la", "s0"), grads):
        dirn = torch.randn(d[n].shape, generator=gen, device="cuda")
        step = 2.0 ** -5 if n != "la" else 2.0 ** -9
        lo, hi = (dict(d, **{n: d[n] + x * dirn}) for x in (-step, step))
        num = ((loss(hi) - loss(lo)) / (2 * step)).item()
        ana = (gr.double() * dirn.double()).sum().item()
        assert abs(num - ana) <= 2e-3 * max(abs(ana), (gr.double().norm() * dirn.double().norm()).item() / math.sqrt(gr.numel())), n


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("B,H,dk,dv", [(1, 1, 64, 64), (3, 5, 128, 64), (2, 7, 64, 128), (200, 3, 128, 128)])
def test_step_continues_the_forward(dr, B, H, dk, dv, gate, dtype, out_dtype):
    d = inputs(B, 4, H, dk, dv, dtype, gate=gate, seed=B)
    out, fin, _ = reference(d["q"], d["k"], d["v"], d["la"], d["s0"])
    c = cuda(d)
    at = lambda x, t: None if x is None else x[:, t].contiguous()
    s = c["s0"].clone()
    for t in range(4):
        o = dr.linrec_step(at(c["q"], t), at(c["k"], t), at(c["v"], t), at(c["la"], t), s, out_dtype=DT[out_dtype])
        check(o, out[:, t], "f32" if out_dtype == "f32" else "bf16", f"out {t}")
    check(s, fin, "f32", "state")


@pytest.mark.gpu
def test_state_carried_in_place_and_mixed_output(dr):
    """Two halves with the state carried in one tensor equal the whole; fp32 outputs of bf16
    inputs."""
    d = inputs(2, 192, 2, 128, 128, "bf16", seed=17)
    out, fin, _ = reference(d["q"], d["k"], d["v"], d["la"], d["s0"])
    c = cuda(d)
    s = c["s0"].clone()
    for a, b in ((0, 100), (100, 192)):
        x = [c[n][:, a:b].contiguous() for n in ("q", "k", "v", "la")]
        o, _ = dr.linrec_fwd(*x, s, final_state=s, out_dtype=torch.float32)
        assert o.dtype == torch.float32
        check(o, out[:, a:b], "bf16", "out")
    check(s, fin, "f32", "state")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,T,H,cu", [("bf16", 9000, 2, None), ("bf16", 9000, 2, [0, 100, 6000, 9000]), ("f32", 300, 2, None)])
def test_states_updated_in_place(dr, dtype, T, H, cu):
    """final_state over init_state, d_init_state over d_final_state (long sequences run in segments
    whose first and last blocks touch the same state)."""
    import ctypes
    N = len(cu) - 1 if cu else 1
    c = cuda(inputs(1, T, H, 128, 128, dtype, N=N if cu else 0, strength=1e-3, seed=7))
    cuc = None if cu is None else torch.tensor(cu, dtype=torch.int64).cuda()
    args = [c[n] for n in ("q", "k", "v", "la")]
    want_o, want_f = dr.linrec_fwd(*args, c["s0"], cu_seqlens=cuc)
    want_g = dr.linrec_bwd(*args, c["s0"], c["do"], c["ds"], cu_seqlens=cuc)
    for _ in range(3):
        s = c["s0"].clone()
        o, f = dr.linrec_fwd(*args, s, cu_seqlens=cuc, final_state=s)
        assert torch.equal(o, want_o) and torch.equal(s, want_f)
        d = c["ds"].clone()
        dt = dr._DT[c["q"].dtype]
        desc = dr.LinrecDesc(1, T, H, 128, 128, N if cu else 0, dt, dt, 1, 0)
        n = ctypes.c_size_t(0)
        assert dr.lib().dr_linrec_bwd_workspace_bytes(ctypes.byref(desc), ctypes.byref(n)) == 0
        ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
        g = [torch.empty_like(x) for x in args]
        p = lambda t: None if t is None else t.data_ptr()
        rc = dr.lib().dr_linrec_bwd(ctypes.byref(desc), *map(p, args), p(cuc), p(c["s0"]), p(c["do"]), p(d), *map(p, g),
                                    p(d), p(ws), n.value, torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        assert all(torch.equal(a, b) for a, b in zip((*g, d), want_g))


@pytest.mark.gpu
def test_no_tokens(dr):
    """T = 0: the state and its gradient pass through."""
    s = torch.randn(2, 3, 64, 64).cuda()
    e = torch.empty(2, 0, 3, 64).cuda()
    la = torch.empty(2, 0, 3).cuda()
    o, f = dr.linrec_fwd(e, e, e, la, s)
    assert o.shape == (2, 0, 3, 64) and torch.equal(f, s)
    g = dr.linrec_bwd(e, e, e, la, s, e, s)
    assert torch.equal(g[4], s)
    e, la, cu = e[:1], la[:1], torch.zeros(3, dtype=torch.int64).cuda()     # two empty packed sequences
    for dtype in (torch.float32, torch.bfloat16):
        o, f = dr.linrec_fwd(e.to(dtype), e.to(dtype), e.to(dtype), la, s, cu_seqlens=cu)
        assert torch.equal(f, s)


@pytest.mark.gpu
def test_equal_calls_give_equal_bits(dr):
    c = cuda(inputs(2, 500, 3, 128, 128, "bf16", seed=23))
    runs = [(*dr.linrec_fwd(c["q"], c["k"], c["v"], c["la"], c["s0"]),
             *dr.linrec_bwd(c["q"], c["k"], c["v"], c["la"], c["s0"], c["do"], c["ds"])) for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))


@pytest.mark.gpu
def test_other_stream_and_graph(dr):
    """On a side stream, two streams at once, and captured and replayed on new inputs."""
    c = cuda(inputs(2, 200, 2, 128, 128, "bf16", seed=29))
    args = [c[n] for n in ("q", "k", "v", "la", "s0")]
    want = (*dr.linrec_fwd(*args), *dr.linrec_bwd(*args, c["do"], c["ds"]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [(*dr.linrec_fwd(*args, stream=s), *dr.linrec_bwd(*args, c["do"], c["ds"], stream=s)) for s in streams]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = (*dr.linrec_fwd(*args), *dr.linrec_bwd(*args, c["do"], c["ds"]))
    e = cuda(inputs(2, 200, 2, 128, 128, "bf16", seed=31))
    for n in c:
        c[n].copy_(e[n])
    graph.replay()
    torch.cuda.synchronize()
    want = (*dr.linrec_fwd(*args), *dr.linrec_bwd(*args, c["do"], c["ds"]))
    assert all(torch.equal(a, b) for a, b in zip(want, res))


# ---------------------------------------------------------------- refusals, without a GPU
def _desc(dr, **kw):
    d = dict(B=2, T=100, H=3, dk=128, dv=128, N=0, in_dtype=dr.DR_BF16, out_dtype=dr.DR_BF16,
             gate=dr.DR_GATE_SCALAR, reserved=0)
    d.update(kw)
    return dr.LinrecDesc(**d)


@pytest.mark.parametrize("bad,status", [
    (dict(dk=96), -2), (dict(dv=32), -2), (dict(B=0), -1), (dict(H=0), -1), (dict(T=-1), -1), (dict(N=-1), -1),
    (dict(gate=3), -1), (dict(gate=2), -2), (dict(in_dtype=5), -1), (dict(out_dtype=-1), -1), (dict(reserved=1), -1),
    (dict(N=4), -1), (dict(B=1, N=1 << 21), -2), (dict(T=1 << 31), -2), (dict(H=1 << 17), -2)])
def test_bad_descriptors(dr, bad, status):
    import ctypes
    n = ctypes.c_size_t(0)
    for f in (dr.lib().dr_linrec_fwd_workspace_bytes, dr.lib().dr_linrec_bwd_workspace_bytes):
        assert f(ctypes.byref(_desc(dr, **bad)), ctypes.byref(n)) == status


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_workspace_does_not_grow_with_whole_sequences(dr, which):
    """Packed sequences that are not cut keep no state: at most two a segment's length of rows (512
    tokens at least) and one more, however many sequences there are."""
    f = getattr(dr.lib(), f"dr_linrec_{which}_workspace_bytes")

    def size(N):
        n = ctypes.c_size_t(0)
        assert f(ctypes.byref(_desc(dr, B=1, T=102400, H=16, N=N, gate=dr.DR_GATE_NONE)), ctypes.byref(n)) == 0
        return n.value

    per = 16 * (128 * 128 + 4) * 4
    assert 0 < size(1024) <= (2 * 102400 // 512 + 1) * per + 256
    assert size(1024) == size(1 << 20) and size(3) <= size(1024)


no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only without a GPU")


@no_gpu_only
def test_host_side_errors(dr):
    """Addresses that are never read: every call is refused first."""
    import ctypes
    vp = ctypes.c_void_p
    far = {n: (i + 1) << 36 for i, n in enumerate(
        ("q", "k", "v", "la", "cu", "s0", "out", "fin", "do", "ds", "dq", "dk", "dv", "dla", "d0", "ws"))}

    def call(f, names, desc, wb=1 << 40, **o):
        p = [vp(o.get(n, far[n])) if o.get(n, 1) is not None else None for n in names]
        return f(ctypes.byref(desc), *p, wb, None)

    fwd = lambda desc, **o: call(dr.lib().dr_linrec_fwd, ("q", "k", "v", "la", "cu", "s0", "out", "fin", "ws"), desc, **o)
    bwd = lambda desc, **o: call(dr.lib().dr_linrec_bwd, ("q", "k", "v", "la", "cu", "s0", "do", "ds", "dq", "dk", "dv",
                                                        "dla", "d0", "ws"), desc, **o)
    d = _desc(dr)
    pk = _desc(dr, B=1, N=3)
    for n in ("q", "k", "v", "la", "out"):
        assert fwd(d, **{n: None}) == -1
        assert fwd(d, **{n: far[n] + (2 if n == "la" else 8)}) == -1
    assert fwd(pk, cu=None) == -1 and fwd(pk, cu=far["cu"] + 4) == -1
    assert fwd(d, out=far["q"]) == -1 and fwd(d, out=far["v"] + 16) == -1
    assert fwd(d, fin=far["s0"] + 1024) == -1
    for n in ("q", "k", "v", "la", "do", "dq", "dk", "dv", "dla"):
        assert bwd(d, **{n: None}) == -1
    assert bwd(_desc(dr, gate=dr.DR_GATE_NONE)) == -1            # a gradient of no gate
    assert bwd(d, dq=far["q"]) == -1 and bwd(d, dk=far["dv"]) == -1 and bwd(d, d0=far["s0"]) == -1
    assert bwd(_desc(dr, out_dtype=dr.DR_F32)) == -2
    assert bwd(d, ws=None) == dr.DR_ERR_WORKSPACE and bwd(d, wb=16) == dr.DR_ERR_WORKSPACE
    st = dr.StepDesc(4, 2, 128, 128, dr.DR_BF16, dr.DR_BF16, dr.DR_GATE_SCALAR, 0)

    def step(desc, **o):
        p = [vp(o.get(n, far[n])) if o.get(n, 1) is not None else None for n in ("q", "k", "v", "la", "s0", "out")]
        return dr.lib().dr_linrec_step(ctypes.byref(desc), *p, None)

    for n in ("q", "k", "v", "la", "s0", "out"):
        assert step(st, **{n: None}) == -1
        assert step(st, **{n: far[n] + (2 if n == "la" else 8)}) == -1
    assert step(st, out=far["s0"]) == -1
    assert step(dr.StepDesc(4, 2, 128, 128, 1, 1, dr.DR_GATE_CHANNEL, 0)) == -2
    assert step(dr.StepDesc(4, 2, 128, 96, 1, 1, 1, 0)) == -2


def test_host_tensors_are_refused(dr):
    if not torch.cuda.is_available():
        pytest.skip("torch.cuda.current_device needs a GPU")
    x = torch.zeros(1, 4, 1, 64)
    with pytest.raises(ValueError):
        dr.linrec_fwd(x, x, x)
    c = x.cuda()
    with pytest.raises(ValueError):
        dr.linrec_fwd(c, c, c, torch.zeros(1, 4, 2).cuda())
    with pytest.raises(ValueError):
        dr.linrec_fwd(c.expand(2, 4, 1, 64), c, c)
    with pytest.raises(ValueError):
        dr.linrec_fwd(c.half(), c.half(), c.half())
    with pytest.raises(ValueError):
        dr.linrec_fwd(c, c, c, cu_seqlens=torch.tensor([0, 4], dtype=torch.int32).cuda())
    with pytest.raises(dr.DrError):
        dr.linrec_fwd(torch.zeros(1, 4, 1, 96).cuda(), torch.zeros(1, 4, 1, 96).cuda(), torch.zeros(1, 4, 1, 96).cuda())


@no_gpu_only
def test_written_buffers_over_inputs_are_refused(dr):
    import ctypes
    vp = ctypes.c_void_p
    d, big = _desc(dr), 1 << 40

    def fwd(**o):
        names = ("q", "k", "v", "la", "cu", "s0", "out", "fin", "ws")
        return dr.lib().dr_linrec_fwd(ctypes.byref(d), *[vp(o.get(n, (i + 1) << 36)) for i, n in enumerate(names)], big, None)

    st = dr.StepDesc(4, 2, 128, 128, dr.DR_BF16, dr.DR_BF16, dr.DR_GATE_SCALAR, 0)

    def step(**o):
        names = ("q", "k", "v", "la", "s0", "out")
        return dr.lib().dr_linrec_step(ctypes.byref(st), *[vp(o.get(n, (i + 1) << 36)) for i, n in enumerate(names)], None)

    for i in range(4):   # q, k, v, log_alpha
        x = (i + 1) << 36
        assert fwd(out=x) == -1 and fwd(fin=x) == -1 and fwd(fin=x + 16) == -1
        assert step(out=x) == -1 and step(s0=x) == -1 and step(s0=x + 16) == -1


@no_gpu_only
def test_offsets_and_workspace_under_written_buffers_are_refused(dr):
    """The blocks of a call read the offsets while others write."""
    vp = ctypes.c_void_p
    d = _desc(dr, B=1, T=4096, N=300)
    names = {"fwd": ("q", "k", "v", "la", "cu", "s0", "out", "fin", "ws"),
             "bwd": ("q", "k", "v", "la", "cu", "s0", "do", "ds", "dq", "dk", "dv", "dla", "d0", "ws")}
    written = {"fwd": ("out", "fin"), "bwd": ("dq", "dk", "dv", "dla", "d0")}
    for f, ns in names.items():
        far = {n: (i + 1) << 36 for i, n in enumerate(ns)}

        def call(**o):
            return getattr(dr.lib(), f"dr_linrec_{f}")(ctypes.byref(d), *[vp(o.get(n, far[n])) for n in ns], 1 << 40, None)

        for w in written[f]:
            assert call(cu=far[w]) == -1 and call(cu=far[w] + 8) == -1 and call(cu=far[w] - 8 * 300) == -1
        n = ctypes.c_size_t(0)
        assert getattr(dr.lib(), f"dr_linrec_{f}_workspace_bytes")(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 0
        for x in ns[:-1]:
            assert call(ws=far[x]) == -1 and call(ws=far[x] - n.value // 16 * 16 + 16) == -1, x


@no_gpu_only
def test_zeroing_of_the_rest_refuses_bad_calls(dr):
    vp = ctypes.c_void_p
    names = ("cu", "dq", "dk", "out", "dla")
    far = {n: (i + 1) << 36 for i, n in enumerate(names)}

    def call(desc, **o):
        p = [vp(o.get(n, far[n])) if o.get(n, 1) is not None else None for n in names]
        return dr.lib().dr_linrec_zero_rest(ctypes.byref(desc), *p, None)

    d = _desc(dr, B=1, N=3)
    assert call(_desc(dr)) == -1 and call(_desc(dr, B=1, N=3, dk=96)) == -2          # not packed; not built
    assert call(d, cu=None) == -1 and call(d, cu=far["cu"] + 4) == -1
    for n in names[1:]:
        assert call(d, **{n: far[n] + (2 if n == "dla" else 8)}) == -1 and call(d, cu=far[n]) == -1
    assert call(_desc(dr, B=1, N=3, T=0)) == 0


@no_gpu_only
def test_unused_workspaces_and_empty_inputs_overlap_nothing(dr):
    """What a call neither reads nor writes may lie anywhere: a workspace of which it needs no byte, rows
    of no token.  (Without a GPU a call that passes its checks ends in DR_ERR_CUDA.)"""
    vp = ctypes.c_void_p
    names = ("q", "k", "v", "la", "cu", "s0", "out", "fin", "ws")
    far = {n: (i + 1) << 36 for i, n in enumerate(names)}

    def fwd(desc, **o):
        return dr.lib().dr_linrec_fwd(ctypes.byref(desc), *[vp(o.get(n, far[n])) for n in names], 1 << 40, None)

    d = _desc(dr, in_dtype=dr.DR_F32, out_dtype=dr.DR_F32)
    for n in names[:-1]:
        assert fwd(d, ws=far[n] + 256) == dr.DR_ERR_CUDA, n
    assert fwd(_desc(dr, T=0), q=far["fin"] + 256, v=far["s0"] + 256) == dr.DR_ERR_CUDA
