"""The additive gated linear recurrence and the query/key preparation in front of it: what
is measured of them.

Operators (by the case's "op"):
  fwd        S_t = a_t S_{t-1} + k_t v_t^T, o_t = S_t^T q_t over a sequence (a_t = exp(log_alpha_t),
             a scalar per head and token, or 1), optionally over packed sequences
  bwd        every gradient of fwd
  step       one token, the state updated in place
  rope       q and k of each head normalised (RMS with weights, L2, or not at all) and rotated
             by their positions
  rope_bwd   its gradients

`run` computes them in elementary torch operations where `own` is false, and through
gated_delta_rule_15_gb300.dr where it is true.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # training forward of a whole batch (this repository's benchmark shape)
        dict(name="fwd_B8_T4096_H16_d128", op="fwd", B=8, T=4096, H=16, dk=128, dv=128, dtype="bf16",
             gate=True, packed=0, init=False),
        # long context, few chains, a state carried in
        dict(name="fwd_B1_T65536_H16_d128_init", op="fwd", B=1, T=65536, H=16, dk=128, dv=128, dtype="bf16",
             gate=True, packed=0, init=True),
        # prefill of ragged prompts packed behind one another, some of them empty or one token long
        dict(name="fwd_packed23_T20011_H8_d64", op="fwd", B=1, T=20011, H=8, dk=64, dv=64, dtype="bf16",
             gate=True, packed=23, init=True),
        # the small single-precision problem of a numerics check, latency
        dict(name="fwd_B1_T256_H1_d64_fp32", op="fwd", B=1, T=256, H=1, dk=64, dv=64, dtype="fp32",
             gate=True, packed=0, init=False),
        # training backward of a batch
        dict(name="bwd_B8_T2048_H16_d128", op="bwd", B=8, T=2048, H=16, dk=128, dv=128, dtype="bf16",
             gate=True, packed=0, init=False),
        # training backward of ragged packed documents, without decay
        dict(name="bwd_packed11_T5003_H8_d128", op="bwd", B=1, T=5003, H=8, dk=128, dv=128, dtype="bf16",
             gate=True, packed=11, init=True),
        # a full serving batch's token
        dict(name="step_B256_H32_d128", op="step", B=256, T=1, H=32, dk=128, dv=128, dtype="bf16",
             gate=True, packed=0, init=True),
        # one user's token: latency
        dict(name="step_B1_H16_d128", op="step", B=1, T=1, H=16, dk=128, dv=128, dtype="bf16",
             gate=True, packed=0, init=True),
        # prompt tokens in front of the recurrence, q and k inside a fused projection's rows
        dict(name="rope_T32768_H16_d128", op="rope", T=32768, Hq=16, Hk=16, d=128, rot=128, dtype="bf16",
             norm="rms", layout="half", scaling="none", fused=True, far=False),
        # a decode batch's tokens at far positions, shared key heads, half of the head rotated
        dict(name="rope_T64_H32_8_d128_far", op="rope", T=64, Hq=32, Hk=8, d=128, rot=64, dtype="bf16",
             norm="rms", layout="interleaved", scaling="by_parts", fused=False, far=True),
        # training backward of the preparation
        dict(name="rope_bwd_T16384_H16_d128", op="rope_bwd", T=16384, Hq=16, Hk=16, d=128, rot=128,
             dtype="bf16", norm="rms", layout="half", scaling="none", fused=True, far=False),
        # an odd number of single-precision rows, L2 norms, part of the head
        dict(name="rope_bwd_T1037_H6_3_d64_fp32", op="rope_bwd", T=1037, Hq=6, Hk=3, d=64, rot=32,
             dtype="fp32", norm="l2", layout="interleaved", scaling="linear", fused=False, far=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "rope", "rope_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "step":
        return dict(op=op, B=_log_int(rng, 1, 256), T=1, H=rng.randint(1, 32), dk=rng.choice([64, 128]),
                    dv=rng.choice([64, 128]), dtype=dtype, gate=rng.random() < 0.8, packed=0, init=True)
    if op in ("rope", "rope_bwd"):
        d = rng.choice([64, 128, 256])
        Hq = rng.randint(1, 24)
        return dict(op=op, T=_log_int(rng, 1, 16384), Hq=Hq, Hk=rng.randint(1, Hq), d=d,
                    rot=rng.choice([d, d, d // 2, d // 4]), dtype=dtype, norm=rng.choice(["rms", "rms", "l2", "none"]),
                    layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "by_parts"]),
                    fused=rng.random() < 0.5, far=rng.random() < 0.5)
    # chunk lengths and sequence ends fall anywhere: odd lengths, one token, few and many chains
    d = rng.choice([64, 128, 128])
    dv = d if rng.random() < 0.8 else 192 - d
    packed = rng.choice([0, 0, rng.randint(1, 32)])
    top = (1 << 18) if op == "fwd" else (1 << 17)      # head-tokens
    if dtype == "fp32" or dv != d:
        top >>= 2
    H = rng.randint(1, 16)
    T = _log_int(rng, 1 if packed == 0 else 64, min(16384, top // H))
    B = 1 if packed else max(1, min(8, _log_int(rng, 1, max(1, top // (H * T)))))
    return dict(op=op, B=B, T=T, H=H, dk=d, dv=dv, dtype=dtype, gate=rng.random() < 0.85, packed=packed,
                init=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _lengths(n, total, seed):
    """`n` sequence lengths whose sum is at most `total` (some rows may lie behind the last
    one): ragged over a factor of a hundred, one of them empty and one a single token."""
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(4.6 * torch.rand(n, generator=g, dtype=torch.float64))
    keep = total - (total // 50 if n > 2 else 0)
    ls = torch.floor(w / w.sum() * keep).to(torch.int64)
    if n > 4:
        ls[n // 3], ls[n // 2] = 0, 1
    return [int(x) for x in ls]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    st = dict(case=case)
    if case["op"] in ("rope", "rope_bwd"):
        T, Hq, Hk, d = case["T"], case["Hq"], case["Hk"], case["d"]
        scale = 0.25 + 3.75 * torch.rand((T, 1, 1), generator=g, device=dev)
        if case["fused"]:      # q | k | v of one projection's output row
            qkv = (randn(T, Hq + 2 * Hk, d) * scale).to(dt)
            st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        else:
            st["q"], st["k"] = (randn(T, Hq, d) * scale).to(dt), (randn(T, Hk, d) * scale).to(dt)
        st["wq"] = st["wk"] = None
        if case["norm"] == "rms":
            st["wq"] = 1.0 + 0.2 * randn(d)
            st["wk"] = 1.0 + 0.2 * randn(d)
        if case["far"]:
            st["pos"] = torch.randint(0, 1 << 20, (T,), generator=g, device=dev)
        else:
            st["pos"] = torch.arange(T, device=dev) + int(torch.randint(0, 4096, (1,), generator=g, device=dev))
        st["scaling"] = {"none": None,
                         "linear": dict(kind="linear", factor=8.0),
                         "by_parts": dict(kind="by_parts", factor=16.0, original=8192.0, low=1.0, high=32.0)}[case["scaling"]]
        st["base"] = 500000.0 if case["far"] else 10000.0
        if case["op"] == "rope_bwd":
            st["dqo"], st["dko"] = randn(T, Hq, d).to(dt), randn(T, Hk, d).to(dt)
        if own:
            from gated_delta_rule_15_gb300 import dr
            st["table"] = dr.rope_table(case["rot"], base=st["base"], scaling=st["scaling"], device=dev)
        return st
    B, T, H, dk, dv = case["B"], case["T"], case["H"], case["dk"], case["dv"]
    lead = (B, H) if case["op"] == "step" else (B, T, H)
    q, k, v = randn(*lead, dk), randn(*lead, dk), randn(*lead, dv)
    st["q"] = (q / q.norm(dim=-1, keepdim=True)).to(dt)
    st["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dt)
    st["v"] = v.to(dt)
    st["la"] = -(0.001 + 0.099 * torch.rand(lead, generator=g, device=dev)) if case["gate"] else None
    st["cu"], N = None, B
    if case["packed"]:
        N = case["packed"]
        ls = _lengths(N, T, seed)
        st["longest"] = max(ls)
        st["cu"] = torch.tensor([0] + ls, dtype=torch.int64).cumsum(0).to(dev)
    st["s0"] = 0.02 * randn(N, H, dk, dv) if case["init"] else None
    if case["op"] == "bwd":
        st["do"] = randn(B, T, H, dv).to(dt)
        st["ds"] = randn(N, H, dk, dv) if case["init"] else None
    st["into"] = None
    if case["packed"]:      # the program's buffers: rows behind the last sequence are left as they are
        st["into"] = torch.zeros_like(st["v"])
        if case["op"] == "bwd":
            st["into"] = [None if st[n] is None else torch.zeros_like(st[n]) for n in ("q", "k", "v", "la")]
    return st


# ------------------------------------------------------------------ plain forms
def _rows(x, cu, longest):
    """[1, T, ...] packed rows as [N, longest, ...], and which of them are there."""
    n = cu.numel() - 1
    at = cu[:n, None] + torch.arange(longest, device=cu.device)[None]
    there = at < cu[1:, None]
    got = x[0][at.clamp(max=x.shape[1] - 1)]
    return torch.where(there.view(n, longest, *([1] * (x.dim() - 2))), got, torch.zeros_like(got))


def _packed(y, cu, total):
    """[N, longest, ...] back as [1, total, ...]; rows of no sequence are zero."""
    n, longest = y.shape[:2]
    at = cu[:n, None] + torch.arange(longest, device=cu.device)[None]
    at = torch.where(at < cu[1:, None], at, total)
    out = y.new_zeros((total + 1,) + y.shape[2:])
    out[at.reshape(-1)] = y.reshape(-1, *y.shape[2:])
    return out[None, :total]


def _blocks(x, C):
    """[N, T, H, e] as [N, H, chunks, C, e] in 32 bits, zero rows at the end."""
    N, T, H = x.shape[:3]
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -T % C))
    return x.reshape(N, -1, C, H, x.shape[3]).permute(0, 3, 1, 2, 4)


def _recurrence(q, k, v, la, s0, C):
    """Chunk form of the recurrence for [N, T, H, e] inputs: outputs [N, T, H, dv] in 32 bits, the
    states before each chunk and after the last [N, H, chunks + 1, dk, dv]."""
    N, T, H, dk = q.shape
    dv = v.shape[-1]
    q, k, v = (_blocks(x.float(), C) for x in (q, k, v))
    nc = q.shape[2]
    g = _blocks(la.double()[..., None], C)[..., 0].cumsum(-1)            # log decay inside a chunk
    ends = g[..., -1].cumsum(-1)                                         # and over whole chunks
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    d = torch.where(low, g[..., :, None] - g[..., None, :], -math.inf).exp().float()
    out = ((q @ k.transpose(-1, -2)) * d) @ v
    e = (k * (g[..., -1:] - g).exp().float()[..., None]).transpose(-1, -2) @ v
    upto = torch.nn.functional.pad(ends, (1, 0))                          # chunks + 1 boundaries
    later = torch.arange(nc + 1, device=q.device)[:, None] > torch.arange(nc, device=q.device)[None]
    w = torch.where(later, upto[..., :, None] - ends[..., None, :], -math.inf).exp().float()
    s = (w @ e.reshape(N, H, nc, dk * dv)).reshape(N, H, nc + 1, dk, dv)
    if s0 is not None:
        s = s + upto.exp().float()[..., None, None] * s0[:, :, None].float()
    out = out + (q * g.exp().float()[..., None]) @ s[:, :, :-1]
    return out.permute(0, 2, 3, 1, 4).reshape(N, nc * C, H, dv)[:, :T], s


def _chunk(T):
    return 64 if T <= 8192 else 256


def _plain_inputs(st):
    xs = [st["q"], st["k"], st["v"]]
    la = st["la"] if st["la"] is not None else torch.zeros(st["q"].shape[:-1], device=st["q"].device)
    xs.append(la)
    if "do" in st:
        xs.append(st["do"])
    if st["cu"] is not None:
        xs = [_rows(x, st["cu"], st["longest"]) for x in xs]
    return xs


def _plain_fwd(st):
    q, k, v, la = _plain_inputs(st)
    out, s = _recurrence(q, k, v, la, st["s0"], _chunk(q.shape[1]))
    if st["cu"] is not None:
        out = _packed(out, st["cu"], st["q"].shape[1])
    return dict(out=out.to(st["q"].dtype), state=s[:, :, -1].clone())


def _plain_bwd(st):
    q, k, v, la, do = _plain_inputs(st)
    C = _chunk(q.shape[1])
    T0 = q.shape[1]
    q, k, v, do = (torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -T0 % C)) for x in (q, k, v, do))
    la = torch.nn.functional.pad(la, (0, 0, 0, -T0 % C))

    def t(s):
        return None if s is None else s.transpose(-1, -2)

    # dq is the forward with (do, v, k) as queries, keys and values; dk and dv are forwards in
    # reversed time, where the decay in front of token t is that of token t + 1
    dq, s = _recurrence(do, v, k, la, t(st["s0"]), C)
    nla = torch.nn.functional.pad(la[:, 1:], (0, 0, 0, 1))
    dk, r = _recurrence(v.flip(1), do.flip(1), q.flip(1), nla.flip(1), t(st["ds"]), C)
    dv, rv = _recurrence(k.flip(1), q.flip(1), do.flip(1), nla.flip(1), st["ds"], C)
    dk, dv = dk.flip(1), dv.flip(1)
    # log-decay gradient: <S_t, dS_t> at each chunk's end, and inside a chunk the later
    # tokens' q.dq - k.dk
    N, T, H = la.shape
    ab = (q.double() * dq).sum(-1) - (k.double() * dk).sum(-1)
    ab = ab.reshape(N, T // C, C, H).flip(2).cumsum(2).flip(2)
    end = (s[:, :, 1:].double() * r[:, :, :-1].flip(2)).sum((-1, -2))      # [N, H, chunks]
    end = end * _blocks(nla.double()[..., None], C)[..., -1, 0].exp()
    dla = (ab + end.transpose(1, 2)[:, :, None]).reshape(N, T, H)[:, :T0].float()
    d0 = la[:, 0].double().exp().float()[..., None, None] * rv[:, :, -1]
    if st["cu"] is not None:        # an empty sequence hands its state's gradient through
        dq, dk, dv, dla = (_packed(x[:, :T0], st["cu"], st["q"].shape[1]) for x in (dq, dk, dv, dla))
    dt = st["q"].dtype
    return dict(dq=dq[:, :st["q"].shape[1]].to(dt), dk=dk[:, :st["q"].shape[1]].to(dt),
                dv=dv[:, :st["q"].shape[1]].to(dt), dla=dla if st["la"] is not None else None,
                d0=d0 if st["s0"] is not None else None)


def _plain_step(st):
    q, k, v = (st[x].float() for x in "qkv")
    s = st["s0"]        # updated in place
    if st["la"] is not None:
        s.mul_(st["la"].exp()[..., None, None])
    s.addcmul_(k[..., :, None], v[..., None, :])
    return dict(out=(q[..., :, None] * s).sum(-2).to(st["q"].dtype), state=s)


def _inv_freq(rot, base, scaling, device):
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=device)
    f = base ** (-i / rot)
    if scaling is not None and scaling["kind"] == "linear":
        f = f / scaling["factor"]
    if scaling is not None and scaling["kind"] == "by_parts":
        turns = scaling["original"] * f / (2 * math.pi)
        w = ((turns - scaling["low"]) / (scaling["high"] - scaling["low"])).clamp(0, 1)
        f = f * (w + (1 - w) / scaling["factor"])
    return f


EPS = 1e-6


def _angles(st, case):
    a = st["pos"].double()[:, None] * _inv_freq(case["rot"], st["base"], st["scaling"], st["pos"].device)
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _halves(x, layout):
    return x.chunk(2, -1) if layout == "half" else (x[..., 0::2], x[..., 1::2])


def _joined(a, b, layout):
    return torch.cat((a, b), -1) if layout == "half" else torch.stack((a, b), -1).flatten(-2)


def _rotate(x, cos, sin, case):
    rot = case["rot"]
    a, b = _halves(x[..., :rot], case["layout"])
    return torch.cat((_joined(a * cos - b * sin, b * cos + a * sin, case["layout"]), x[..., rot:]), -1)


def _inverse_norm(x, norm):
    if norm == "none":
        return torch.ones_like(x[..., :1])
    s = x.square().mean(-1, keepdim=True) if norm == "rms" else x.square().sum(-1, keepdim=True)
    return (s + EPS).rsqrt()


def _plain_rope(st):
    case = st["case"]
    cos, sin = _angles(st, case)
    got = {}
    for n in "qk":
        x = st[n].float()
        y = x * _inverse_norm(x, case["norm"])
        if st["w" + n] is not None:
            y = y * st["w" + n]
        got[n] = _rotate(y, cos, sin, case).to(st[n].dtype)
    return got


def _plain_rope_bwd(st):
    case = st["case"]
    cos, sin = _angles(st, case)
    got = {}
    for n in "qk":
        x = st[n].float()
        r = _inverse_norm(x, case["norm"])
        u = _rotate(st["d" + n + "o"].float(), cos, -sin, case)
        gw = u if st["w" + n] is None else u * st["w" + n]
        dx = gw * r
        if case["norm"] != "none":
            m = (gw * x).sum(-1, keepdim=True)
            if case["norm"] == "rms":
                m = m / x.shape[-1]
            dx = dx - x * (r * r * r * m)
        got["d" + n] = dx.to(st[n].dtype)
        if st["w" + n] is not None:
            got["dw" + n] = (u * x * r).double().sum((0, 1)).float()
    return got


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "rope": _plain_rope,
                "rope_bwd": _plain_rope_bwd}[op](state)
    from gated_delta_rule_15_gb300 import dr
    st = state
    if op == "fwd":
        out, s = dr.linrec_fwd(st["q"], st["k"], st["v"], st["la"], st["s0"], cu_seqlens=st["cu"], out=st["into"])
        return dict(out=out, state=s)
    if op == "bwd":
        dq, dk, dv, dla, d0 = dr.linrec_bwd(st["q"], st["k"], st["v"], st["la"], st["s0"], st["do"], st["ds"],
                                            cu_seqlens=st["cu"], grads=st["into"],
                                            return_d_init=st["s0"] is not None)
        return dict(dq=dq, dk=dk, dv=dv, dla=dla, d0=d0)
    if op == "step":
        return dict(out=dr.linrec_step(st["q"], st["k"], st["v"], st["la"], st["s0"]), state=st["s0"])
    kw = dict(positions=st["pos"], norm=case["norm"], wq=st["wq"], wk=st["wk"], eps=EPS, layout=case["layout"])
    if op == "rope":
        q, k = dr.qk_norm_rope(st["q"], st["k"], st["table"], **kw)
        return dict(q=q, k=k)
    dq, dk, dwq, dwk = dr.qk_norm_rope_bwd(st["q"], st["k"], st["table"], st["dqo"], st["dko"], **kw)
    return {n: x for n, x in (("dq", dq), ("dk", dk), ("dwq", dwq), ("dwk", dwk)) if x is not None}


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("rope", "rope_bwd"):
        rows, d = case["T"] * (case["Hq"] + case["Hk"]), case["d"]
        w = (8 * d if case["norm"] == "rms" else 0) + 8 * case["T"] + 4 * case["rot"]
        if case["op"] == "rope":
            return {"bytes": 2 * rows * d * e + w, "flops": 8 * rows * d}
        return {"bytes": 3 * rows * d * e + 2 * w, "flops": 16 * rows * d}
    B, T, H, dk, dv = case["B"], case["T"], case["H"], case["dk"], case["dv"]
    N = case["packed"] or B
    tok, gate = B * T * H, 4 if case["gate"] else 0
    state = 4 * N * H * dk * dv
    if case["op"] == "bwd":
        return {"bytes": tok * (e * (4 * dk + 3 * dv) + 2 * gate) + (3 if case["init"] else 0) * state,
                "flops": 10 * tok * dk * dv}
    return {"bytes": tok * (e * 2 * (dk + dv) + gate) + (2 if case["init"] else 1) * state,
            "flops": 4 * tok * dk * dv}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_tokens(st):
    """The sequences one beside the other in 64 bits, [N, H, T, e], zero behind their ends."""
    names = [n for n in ("q", "k", "v", "la", "do") if st.get(n) is not None]
    if st["cu"] is None:
        return {n: st[n].double().transpose(1, 2) for n in names}, [st["q"].shape[1]] * st["q"].shape[0]
    cu = st["cu"].tolist()
    ls = [b - a for a, b in zip(cu, cu[1:])]
    top = max(max(ls), 1)
    got = {}
    for n in names:
        x = st[n][0].double()
        y = x.new_zeros((len(ls), top) + x.shape[1:])
        for i, (a, b) in enumerate(zip(cu, cu[1:])):
            y[i, :b - a] = x[a:b]
        got[n] = y.transpose(1, 2)
    return got, ls


def _exact_back(y, st, ls):
    """[N, H, T, ...] in the inputs' layout."""
    y = y.transpose(1, 2)
    if st["cu"] is None:
        return y
    out = y.new_zeros((1, st["q"].shape[1]) + y.shape[2:])
    at = 0
    for i, n in enumerate(ls):
        out[0, at:at + n] = y[i, :n]
        at += n
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("rope", "rope_bwd"):
        return _exact_rope(st, case)
    if case["op"] == "step":
        s = st["s0"].double()
        if st["la"] is not None:
            s = st["la"].double().exp()[..., None, None] * s
        s = s + torch.einsum("bhi,bhj->bhij", st["k"].double(), st["v"].double())
        return dict(out=torch.einsum("bhij,bhi->bhj", s, st["q"].double()), state=s)
    x, ls = _exact_tokens(st)
    N, H, T, dk = x["q"].shape
    dv = x["v"].shape[-1]
    live = torch.arange(T, device="cuda")[None] < torch.tensor(ls, device="cuda")[:, None]      # [N, T]
    a = (x["la"].exp() if "la" in x else torch.ones_like(x["q"][..., 0])) * live[:, None] + ~live[:, None]
    s0 = st["s0"].double() if st["s0"] is not None else torch.zeros(N, H, dk, dv, dtype=torch.float64, device="cuda")
    s = s0.clone()
    if case["op"] == "fwd":
        out = torch.zeros_like(x["v"])
        for t in range(T):      # padded rows have a = 1 and k = 0: the state stays
            s.mul_(a[:, :, t, None, None])
            s.addcmul_(x["k"][:, :, t, :, None], x["v"][:, :, t, None, :])
            out[:, :, t] = (x["q"][:, :, t, None, :] @ s)[:, :, 0]
        return dict(out=_exact_back(out, st, ls), state=s)
    if T * N * H * dk * dv * 8 > 60e9:
        return None
    before = torch.empty(T, N, H, dk, dv, dtype=torch.float64, device="cuda")
    dq, dk_, dv_ = (torch.zeros_like(x[n]) for n in ("q", "k", "v"))
    dla = torch.zeros_like(a)
    for t in range(T):
        before[t] = s
        s.mul_(a[:, :, t, None, None])
        s.addcmul_(x["k"][:, :, t, :, None], x["v"][:, :, t, None, :])
        dq[:, :, t] = (s @ x["do"][:, :, t, :, None])[..., 0]
    ds = st["ds"].double() if st["ds"] is not None else torch.zeros_like(s)
    for t in range(T - 1, -1, -1):
        ds = ds + x["q"][:, :, t, :, None] * x["do"][:, :, t, None, :]
        dk_[:, :, t] = (ds @ x["v"][:, :, t, :, None])[..., 0]
        dv_[:, :, t] = (x["k"][:, :, t, None, :] @ ds)[:, :, 0]
        ds = ds * a[:, :, t, None, None]
        dla[:, :, t] = (before[t] * ds).sum((-1, -2))
    back = [_exact_back(y, st, ls) for y in (dq, dk_, dv_, dla)]
    return dict(dq=back[0], dk=back[1], dv=back[2], dla=back[3] if st["la"] is not None else None,
                d0=ds if st["s0"] is not None else None)


def _exact_rope(st, case):
    rot, d = case["rot"], case["d"]
    sc, freq = st["scaling"], []
    for i in range(rot // 2):
        f = math.pow(st["base"], -2.0 * i / rot)
        if sc is not None and sc["kind"] == "linear":
            f /= sc["factor"]
        elif sc is not None:
            full = (sc["original"] / (2 * math.pi / f) - sc["low"]) / (sc["high"] - sc["low"])
            full = min(1.0, max(0.0, full))
            f = full * f + (1 - full) * f / sc["factor"]
        freq.append(f)
    ang = torch.outer(st["pos"].double(), torch.tensor(freq, dtype=torch.float64, device="cuda"))
    i = torch.arange(rot // 2, device="cuda")
    one, two = (i, i + rot // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
    # the rotation of every token as a matrix [T, d, d] would be large: by its two columns instead
    z = torch.complex(ang.cos(), ang.sin())[:, None]

    def turn(x, by):
        y = x.clone()
        c = torch.complex(x[..., one], x[..., two]) * by
        y[..., one], y[..., two] = c.real, c.imag
        return y

    got = {}
    for n in "qk":
        x = st[n].double()
        w = torch.ones(d, dtype=torch.float64, device="cuda") if st["w" + n] is None else st["w" + n].double()
        size = {"rms": (x * x).sum(-1, keepdim=True) / d + EPS, "l2": (x * x).sum(-1, keepdim=True) + EPS,
                "none": torch.ones_like(x[..., :1])}[case["norm"]].sqrt()
        if case["op"] == "rope":
            got[n] = turn(x / size * w, z)
            continue
        u = turn(st["d" + n + "o"].double(), z.conj())
        dx = u * w / size
        if case["norm"] != "none":
            dx = dx - x * (u * w * x).sum(-1, keepdim=True) / (size ** 3 * (d if case["norm"] == "rms" else 1))
        got["d" + n] = dx
        if st["w" + n] is not None:
            got["dw" + n] = (u * x / size).sum((0, 1))
    return got
