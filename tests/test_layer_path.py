"""The operators of a linear-attention layer one behind the other, as a layer uses them: a fused
projection's rows -> norm and rotation of queries and keys -> additive recurrence (packed
prompts, then single tokens), and the same path backwards, against 64-bit autograd; and the
preparation in front of the gated delta rule.

Tolerances: each operator's own (test_linrec.py, test_qk_norm_rope.py), added along the path.
A bf16 stage hands its rounding (2^-8 of a value, random signs) to sums over 128 channels and
the sequence, which keep the relative size: in bf16 three stages' worth, 3 * 2.4e-2 of the
row's RMS; in fp32 3 * 2.5e-4.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": 3 * 2.5e-4, "bf16": 3 * 2.4e-2}
H, D, BASE = 3, 128, 10000.0


@pytest.fixture(scope="module")
def dr():
    import gated_delta_rule_15_gb300.dr as m
    return m


def rotate(x, w, pos):
    """RMS norm with weights and rotation (half layout), 64 bits, differentiable."""
    y = w * x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    ang = pos.double()[:, None] * BASE ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = y.chunk(2, -1)
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def recur(q, k, v, la, s):
    """One sequence [T, H, D]: outputs, final state."""
    out = []
    for t in range(q.shape[0]):
        s = la[t].exp()[:, None, None] * s + k[t][:, :, None] * v[t][:, None, :]
        out.append(torch.einsum("hij,hi->hj", s, q[t]))
    return torch.stack(out), s


def close(got, ref, dtype, what):
    got, ref = got.detach().double().cpu().reshape(ref.shape), ref.detach()
    rms = ref.square().mean(-1, keepdim=True).sqrt().expand(ref.shape).clamp(min=ref.square().mean().sqrt().item())
    err = ((got - ref).abs() / torch.maximum(rms, ref.abs())).max().item()
    assert err <= TOL[dtype], f"{what}: {err:.3e}"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompts_tokens_and_gradients(dr, dtype):
    lens = [5, 0, 130, 64]
    T, N = sum(lens), len(lens)
    gen = torch.Generator().manual_seed(3)
    qkv = torch.randn((T, 3 * H, D), generator=gen).to(DT[dtype])
    la = -0.1 * torch.rand((1, T, H), generator=gen)
    wq, wk = 0.1 * (1 + 0.2 * torch.randn(D, generator=gen)), 0.1 * (1 + 0.2 * torch.randn(D, generator=gen))
    s0 = 0.3 * torch.randn((N, H, D, D), generator=gen)
    do = torch.randn((1, T, H, D), generator=gen).to(DT[dtype])
    ds = torch.randn((N, H, D, D), generator=gen)
    starts = torch.tensor([0] + lens).cumsum(0)
    pos = torch.cat([torch.arange(n) for n in lens])
    # the path
    table = dr.rope_table(D, base=BASE)
    c = qkv.cuda()
    parts = [c[:, :H], c[:, H:2 * H], c[:, 2 * H:].contiguous()[None]]
    kw = dict(positions=pos.cuda(), wq=wq.cuda(), wk=wk.cuda())
    q, k = dr.qk_norm_rope(parts[0], parts[1], table, **kw)
    cu = starts.cuda()
    out, fin = dr.linrec_fwd(q[None], k[None], parts[2], la.cuda(), s0.cuda(), cu_seqlens=cu)
    dq, dk, dv, dla, d0 = dr.linrec_bwd(q[None], k[None], parts[2], la.cuda(), s0.cuda(), do.cuda(), ds.cuda(), cu_seqlens=cu)
    dqkv = torch.empty_like(c)
    dqkv[:, 2 * H:] = dv[0]
    _, _, dwq, dwk = dr.qk_norm_rope_bwd(parts[0], parts[1], table, dq[0], dk[0], dq=dqkv[:, :H], dk=dqkv[:, H:2 * H], **kw)
    # 64 bits
    leaves = [x.double().clone().requires_grad_() for x in (qkv, la, wq, wk, s0)]
    x, a, uq, uk, z0 = leaves
    rq, rk = rotate(x[:, :H], uq, pos), rotate(x[:, H:2 * H], uk, pos)
    outs, fins = [], []
    for n in range(N):
        i, j = int(starts[n]), int(starts[n + 1])
        o, f = recur(rq[i:j], rk[i:j], x[i:j, 2 * H:], a[0, i:j], z0[n]) if j > i else (rq[i:j], z0[n])
        outs.append(o)
        fins.append(f)
    o, f = torch.cat(outs), torch.stack(fins)
    ((o * do[0].double()).sum() + (f * ds.double()).sum()).backward()
    close(out[0], o, dtype, "out")
    close(fin, f, dtype, "state")
    close(dqkv, x.grad, dtype, "dqkv")
    close(dwq, uq.grad, dtype, "dwq")
    close(dwk, uk.grad, dtype, "dwk")
    close(dla, a.grad, dtype, "d_log_alpha")
    close(d0, z0.grad, dtype, "d_init_state")
    # one more token of every sequence
    x1 = torch.randn((N, 3 * H, D), generator=gen).to(DT[dtype])
    la1 = -0.1 * torch.rand((N, H), generator=gen)
    c1, p1 = x1.cuda(), torch.tensor(lens)
    q1, k1 = dr.qk_norm_rope(c1[:, :H], c1[:, H:2 * H], table, positions=p1.cuda(), wq=wq.cuda(), wk=wk.cuda())
    o1 = dr.linrec_step(q1, k1, c1[:, 2 * H:].contiguous(), la1.cuda(), fin)
    r1, r2 = rotate(x1[:, :H].double(), wq.double(), p1), rotate(x1[:, H:2 * H].double(), wk.double(), p1)
    s1 = la1.double().exp()[..., None, None] * f.detach() + r2[..., :, None] * x1[:, 2 * H:].double()[..., None, :]
    close(o1, torch.einsum("nhij,nhi->nhj", s1, r1), dtype, "token")
    close(fin, s1, dtype, "state after the token")
    assert dr.device_status() == 0


def test_preparation_in_front_of_the_delta_rule(dr):
    """The L2 norm alone equals the delta rule's own fused one up to the rounding of the stored q, k."""
    from gated_delta_rule_15_gb300 import inputs
    d = inputs.chunk_inputs(2, 130, 3, 128, 128, gate="scalar", dtype="f32", init_state=True, seed=5, raw=True)
    g = {k: None if v is None else v.cuda() for k, v in d.items()}
    want, fin = dr.chunk_fwd(g["q"], g["k"], g["v"], g["log_alpha"], g["beta"], g["init_state"], qk_l2norm=True, beta_sigmoid=True)
    q, k = dr.qk_norm_rope(g["q"], g["k"], None, norm="l2", eps=dr.L2NORM_EPS)
    out, fin2 = dr.chunk_fwd(q, k, g["v"], g["log_alpha"], g["beta"], g["init_state"], beta_sigmoid=True)
    # fp32 rows differ by their rounding, 2^-24 of 128 values in unit-size sums: the chunk form's own
    # fp32 bound, 1e-4, on both sides
    assert (out - want).abs().max() <= 2e-4 and (fin2 - fin).abs().max() <= 2e-4
