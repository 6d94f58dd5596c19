"""Window attention (forward, gradients, one token over a paged cache) and the cache's filling
against their definitions in 64 bits.

Tolerances, u = 2^-24; a bf16 rounding is off by at most 2^-8 of the value.  Every bound is a sum of
absolute values that the reference forms beside the result, element by element.
  Weights.  A score is an fp32 sum of up to 128 products (off by some 16 u of the sum of their
sizes, which is about 8 for rows of unit scale), one rounding of the exponent's argument and an
exponential good to a few u: the weight p is off by at most 2^-17 = 128 u of itself, times the scores'
size where that is larger than 16 (`size`).  The same holds for lse in absolute terms.
  fp32: out is off by at most 2^-17 size sum p |v|; the gradients by 2^-17 size times the sums of absolute
values of all their factors (dq: scale sum p (sum |do v| + sum |do o|) |k|, dk the same with |q|; dv: sum p |do|).
  bf16: besides that a weight, and a score gradient ds, is rounded once, 2^-8 of it, and so is the result.
The backward's delta = do.out takes out as it is given, which the forward has rounded: off by
sum |do| e(out), which enters dq as scale sum p |k| times that.
  One token: weights are two bf16 terms (2^-16 of a weight is lost), so only the result's rounding counts.
"""
import ctypes
import math
import random

import pytest
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = 2.0 ** -8     # half a step of bf16
U17 = 2.0 ** -17


@pytest.fixture(scope="module")
def dr():
    import gated_delta_rule_15_gb300.dr as m
    return m


def visible(T, window, sinks):
    i, j = torch.arange(T)[:, None], torch.arange(T)[None]
    return (j <= i) & (((i - j < window) if window else torch.ones(T, T, dtype=torch.bool)) | (j < sinks))


def spans_of(x, cu):
    B, T = x.shape[:2]
    return [(b, 0, T) for b in range(B)] if cu is None else [(0, int(a), int(e)) for a, e in zip(cu[:-1], cu[1:])]


def reference(q, k, v, window, sinks, scale, bf16, cu=None, do=None):
    """Results and, by the docstring, how far they may be off; rows of no sequence are NaN."""
    q, k, v = (x.double().cpu() for x in (q, k, v))
    g = q.shape[2] // k.shape[2]
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.float64)
    names = ["out", "lse"] + ([] if do is None else ["dq", "dk", "dv"])
    shape = dict(out=q.shape, lse=q.shape[:3], dq=q.shape, dk=k.shape, dv=v.shape)
    R, E = {n: nan(*shape[n]) for n in names}, {n: nan(*shape[n]) for n in names}
    rnd = HALF if bf16 else 0.0
    for b, lo, hi in spans_of(q, cu):
        if hi == lo:
            continue
        see = visible(hi - lo, window, sinks)
        for h in range(q.shape[2]):
            Q, K, V = q[b, lo:hi, h], k[b, lo:hi, h // g], v[b, lo:hi, h // g]
            s = scale * Q @ K.T
            sizes = scale * Q.abs() @ K.abs().T
            size = max(1.0, float(sizes[see].max()) / 16)
            u = U17 * size
            s = s.masked_fill(~see, -math.inf)
            lse = torch.logsumexp(s, 1)
            p = (s - lse[:, None]).exp()
            o = p @ V
            R["out"][b, lo:hi, h], R["lse"][b, lo:hi, h] = o, lse
            e_o = (u + rnd) * (p @ V.abs()) + rnd * o.abs()
            E["out"][b, lo:hi, h], E["lse"][b, lo:hi, h] = e_o, u * (1 + lse.abs())
            if do is None:
                continue
            D = do[b, lo:hi, h].double().cpu()
            dp, delta = D @ V.T, (D * o).sum(1, keepdim=True)
            ds = p * (dp - delta)
            off = p * (u * (D.abs() @ V.abs().T + (D.abs() * o.abs()).sum(1, keepdim=True)) + (D.abs() * e_o).sum(1, keepdim=True))
            off = off + rnd * ds.abs()
            R["dq"][b, lo:hi, h] = scale * ds @ K
            E["dq"][b, lo:hi, h] = scale * off @ K.abs() + rnd * R["dq"][b, lo:hi, h].abs()
            for n, x, e in (("dk", scale * ds.T @ Q, scale * off.T @ Q.abs()), ("dv", p.T @ D, (u + rnd) * p.T @ D.abs())):
                for dst, y in ((R, x), (E, e)):
                    t = dst[n][b, lo:hi, h // g]
                    t.copy_(y if h % g == 0 else t + y)
        if do is not None:      # the last rounding
            for n in ("dk", "dv"):
                E[n][b, lo:hi] += rnd * R[n][b, lo:hi].abs()
    return R, E


def compare(got, R, E, names=None):
    for n in names or R:
        x, r, e = got[n].double().cpu(), R[n], E[n]
        rows = ~torch.isnan(r)
        assert torch.isfinite(x[rows]).all(), n
        worst = ((x - r).abs() / (e + 1e-30))[rows].max().item() if rows.any() else 0.0
        assert worst <= 1, f"{n}: {worst:.3f} of the bound"


def make(B, T, Hq, Hk, d, dtype, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed)
    q, do = (torch.randn((B, T, Hq, d), generator=g) for _ in range(2))
    k, v = (torch.randn((B, T, Hk, d), generator=g) for _ in range(2))
    return [x.to(DT[dtype]) for x in (q * size, k, v, do)]


def run(dr, q, k, v, do, window, sinks, scale=None, cu=None, backward=True):
    c = [x.cuda() for x in (q, k, v, do)]
    cu_d = None if cu is None else torch.tensor(cu, dtype=torch.int64).cuda()
    kw = dict(window=window, sinks=sinks, scale=scale, cu_seqlens=cu_d)
    out, lse = dr.window_attn_fwd(*c[:3], **kw)
    got = dict(out=out, lse=lse)
    if backward:
        got["dq"], got["dk"], got["dv"] = dr.window_attn_bwd(*c[:3], out, lse, c[3], **kw)
    torch.cuda.synchronize()
    assert dr.lib().dr_get_device_status(None) == 0
    return got


def both(dr, B, T, Hq, Hk, d, window, sinks, dtype, seed=0, scale=None, cu=None, size=1.0):
    q, k, v, do = make(B, T, Hq, Hk, d, dtype, seed, size)
    got = run(dr, q, k, v, do, window, sinks, scale, cu)
    R, E = reference(q, k, v, window, sinks, scale or d ** -0.5, dtype == "bf16", cu, do)
    compare(got, R, E)
    return got, R


SHAPES = [  # B, T, Hq, Hk, d, window, sinks
    (1, 1, 1, 1, 64, 0, 0), (1, 1, 3, 1, 128, 1, 0), (2, 2, 2, 1, 64, 1, 0), (3, 5, 2, 2, 128, 2, 1),
    (1, 16, 4, 2, 64, 0, 0), (1, 63, 3, 1, 128, 0, 0), (2, 64, 2, 2, 64, 17, 2), (1, 65, 2, 1, 128, 64, 1),
    (1, 127, 2, 2, 64, 0, 0), (2, 128, 2, 1, 128, 128, 0), (2, 129, 4, 2, 128, 64, 4), (1, 255, 1, 1, 64, 30, 40),
    (1, 257, 6, 2, 64, 100, 3), (1, 300, 8, 1, 128, 130, 200), (1, 400, 2, 2, 128, 1, 1), (1, 513, 2, 1, 64, 512, 0),
    (1, 640, 3, 3, 128, 128, 128), (3, 200, 2, 1, 64, 1000, 5), (1, 384, 2, 1, 128, 0, 7), (1, 520, 2, 1, 64, 7, 130),
    (1, 641, 1, 1, 128, 129, 1), (1, 256, 16, 1, 64, 200, 16),
    (1, 2500, 2, 1, 64, 40, 5), (2, 1400, 2, 1, 128, 200, 200), (1, 2300, 1, 1, 64, 50, 1100), (1, 1500, 3, 1, 64, 0, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hk,d,window,sinks", SHAPES)
def test_forward_and_gradients(dr, B, T, Hq, Hk, d, window, sinks, dtype):
    both(dr, B, T, Hq, Hk, d, window, sinks, dtype, seed=T)


PACKED = [([0, 100, 100, 101, 257, 700, 700], 720), ([0, 1], 1), ([0, 0, 64, 128, 129], 129), ([5, 130, 131, 400], 411),
          ([0, 3, 5, 9, 10, 11, 12, 40, 41, 47], 50), ([0, 0, 0], 30), ([0, 640], 640), ([0, 1300, 1310, 3500], 3600)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3), (128, 0), (2, 140)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cu,T", PACKED)
def test_packed_sequences(dr, cu, T, d, window, sinks, dtype):
    got, R = both(dr, 1, T, 4, 2, d, window, sinks, dtype, seed=T + d, cu=cu)
    rest = torch.isnan(R["lse"][0, :, 0])
    for n, x in got.items():      # new buffers hold zeros in the rows of no sequence
        assert (x[0].cpu()[rest] == 0).all(), n


@pytest.mark.gpu
def test_many_short_sequences(dr):
    cu = [0]
    for i in range(300):
        cu.append(cu[-1] + (i * 7) % 5)
    both(dr, 1, cu[-1] + 3, 2, 1, 64, 3, 1, "bf16", seed=3, cu=cu)


def lengths_between_short_ones(long, short, n):
    """n sequences: the long ones with 0 to `short` tokens' ones between them."""
    ls = [(5 * i) % (short + 1) for i in range(n)]
    for i, x in enumerate(long):
        ls[(i * n) // len(long)] = x
    return [int(x) for x in torch.tensor([0] + ls).cumsum(0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hk", [(4, 2), (2, 1)])
@pytest.mark.parametrize("long,short,n,window,sinks", [
    ([600, 17, 16], 2, 50, 1, 20), ([600, 260, 280], 3, 50, 2, 130), ([2500, 131, 130, 1300], 6, 160, 3, 20), ([2500, 400, 1400, 300], 8, 160, 100, 150),
    ([1250, 200, 329, 328], 5, 220, 200, 1), ([2600, 1200], 4, 200, 1, 1000)])
def test_sinks_of_some_of_many_sequences(dr, long, short, n, window, sinks, Hq, Hk, dtype):
    """More sequences than can be longer than the window: sums of sinks' rows lie by rows, not by sequence.  The workspace is
    full of NaN beforehand."""
    cu = lengths_between_short_ones(long, short, n)
    T = cu[-1] + 2
    q, k, v, do = make(1, T, Hq, Hk, 64, dtype, seed=n + window)
    c, cu_d = [x.cuda() for x in (q, k, v, do)], torch.tensor(cu).cuda()
    kw = dict(window=window, sinks=sinks, cu_seqlens=cu_d)
    out, lse = dr.window_attn_fwd(*c[:3], **kw)
    size = bwd_bytes(dr, B=1, T=T, Hq=Hq, Hk=Hk, d=64, N=n, window=window, sinks=sinks, dtype=dr.DR_BF16 if dtype == "bf16" else dr.DR_F32)
    ws = torch.full((size // 4,), float("nan"), device="cuda")
    dq, dk, dv = dr.window_attn_bwd(*c[:3], out, lse, c[3], workspace=ws, **kw)
    torch.cuda.synchronize()
    assert dr.lib().dr_get_device_status(None) == 0
    R, E = reference(q, k, v, window, sinks, 0.125, dtype == "bf16", cu, do)
    compare(dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv), R, E)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 5)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hk", [(8, 16, 16), (4, 32, 16), (4, 32, 8), (9, 12, 4), (1, 32, 16), (1, 20, 20)])
def test_blocks_of_many_items(dr, B, Hq, Hk, d, window, sinks):
    """Each of 152 blocks gets four items and more, of up to a dozen key tiles (B 1: ragged sequences in one row): the bits of calls for a
    key head of a batch row, where a block has one, and those against the reference."""
    T, g, cu = 1451, Hq // Hk, None
    if B == 1:
        cu = [int(x) for x in torch.tensor([3, 700, 0, 129, 1, 1451, 128, 64, 900, 257, 0, 77, 1023, 300, 65, 1100]).cumsum(0)]
        T = cu[-1] + 9
    tokens = 256 // (4 if g % 4 == 0 else 2 if g % 2 == 0 else 1)
    per = g if g % 2 else g // (4 if g % 4 == 0 else 2)
    lens = [T] * B if cu is None else [b - a for a, b in zip(cu, cu[1:])]
    assert sum(-(-n // tokens) for n in lens) * Hk * per >= 4 * 152
    q, k, v, do = make(B, T, Hq, Hk, d, "bf16", seed=Hq + B)
    got = run(dr, q, k, v, do, window, sinks, cu=cu)
    c = [x.cuda() for x in (q, k, v, do)]
    kw = dict(window=window, sinks=sinks, cu_seqlens=None if cu is None else torch.tensor(cu).cuda())
    for b in range(B):
        for h in range(Hk):
            one = [x[b:b + 1, :, h * n:(h + 1) * n] for x, n in zip(c, (g, 1, 1, g))]
            out, lse = dr.window_attn_fwd(*one[:3], **kw)
            grads = dr.window_attn_bwd(*one[:3], out, lse, one[3], **kw)
            for name, x, n in zip(("out", "lse", "dq", "dk", "dv"), (out, lse) + grads, (g, g, g, 1, 1)):
                assert torch.equal(x[0], got[name][b, :, h * n:(h + 1) * n]), (name, b, h)
    b, h = B - 1, Hk // 2
    one = [x[b:b + 1, :, h * n:(h + 1) * n] for x, n in zip((q, k, v, do), (g, 1, 1, g))]
    R, E = reference(*one[:3], window, sinks, d ** -0.5, True, cu, one[3])
    compare({name: got[name][b:b + 1, :, h * n:(h + 1) * n] for name, n in zip(("out", "lse", "dq", "dk", "dv"), (g, g, g, 1, 1))}, R, E)


def log_int(rng, lo, hi):
    return round(math.exp(rng.uniform(math.log(lo), math.log(hi))))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seed", range(40))
def test_drawn_problems(dr, seed, dtype):
    """Any heads, lengths, windows, sinks, sequences and strides together."""
    rng = random.Random(seed)
    d, Hk = rng.choice([64, 128]), rng.randint(1, 8)
    Hq = Hk * rng.choice([1, 2, 3, 4, 8])
    window = rng.choice([0, 1, 2, 2]) and log_int(rng, 1, 700)
    sinks = rng.choice([0, rng.randint(1, 8), log_int(rng, 1, 400)])
    n, cu = rng.choice([0, 0, rng.randint(1, 32)]), None
    T = log_int(rng, 1 if n == 0 else 64, 700)
    B = 1 if n else rng.randint(1, 3)
    if n:
        ends = sorted(rng.randint(0, T) for _ in range(n))
        cu = [rng.choice([0, ends[0]])] + ends
    q, k, v, do = make(B, T, Hq, Hk, d, dtype, seed)
    fused = rng.random() < 0.5
    row = torch.cat((q, k, v), 2).cuda()
    c = row.split((Hq, Hk, Hk), 2) if fused else [x.cuda() for x in (q, k, v)]
    kw = dict(window=window, sinks=sinks, cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int64).cuda())
    out, lse = dr.window_attn_fwd(*c, **kw)
    grads = dr.window_attn_bwd(*c, out, lse, do.cuda(), grads=torch.zeros_like(row).split((Hq, Hk, Hk), 2) if fused else None, **kw)
    torch.cuda.synchronize()
    assert dr.lib().dr_get_device_status(None) == 0
    R, E = reference(q, k, v, window, sinks, d ** -0.5, dtype == "bf16", cu, do)
    compare(dict(zip(R, (out, lse) + grads)), R, E)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seed", range(20))
def test_drawn_steps(dr, seed, dtype):
    rng = random.Random(seed)
    Hk = rng.randint(1, 8)
    window, sinks = rng.choice([0, 1, 2]) and log_int(rng, 1, 700), rng.choice([0, rng.randint(1, 8), log_int(rng, 1, 200)])
    lens = [rng.choice([-1, 0, log_int(rng, 1, 900), log_int(rng, 1, 900)]) for _ in range(log_int(rng, 1, 30))]
    step_case(dr, lens, Hk * rng.choice([1, 2, 3, 4, 8]), Hk, rng.choice([64, 128]), window, sinks, 16 << rng.randint(0, 4), dtype, seed=seed)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_others_do_not_matter(dr, d, dtype):
    cu, T = [20, 150, 150, 290], 300
    q, k, v, do = make(1, T, 2, 1, d, dtype, seed=5)
    rest = torch.ones(T, dtype=torch.bool)
    rest[20:290] = False
    clean = run(dr, q, k, v, do, 40, 3, cu=cu)
    for x in (q, k, v, do):
        x[:, rest] = float("nan")
    x = [t.clone() for t in (q, k, v, do)]
    dirty = run(dr, *x, 40, 3, cu=cu)
    for n in clean:
        assert torch.equal(clean[n], dirty[n]), n
    for t in x[:3]:      # the second sequence is full of infinities: the first does not see them
        t[:, 150:290] = float("inf")
    dirty = run(dr, *x, 40, 3, cu=cu)
    for n in clean:
        assert torch.equal(clean[n][:, :150], dirty[n][:, :150]), n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_given_buffers_keep_rows_of_no_sequence(dr, dtype):
    cu, T = torch.tensor([7, 100, 200], dtype=torch.int64).cuda(), 230
    q, k, v, do = (x.cuda() for x in make(1, T, 4, 2, 64, dtype, seed=9))
    kw = dict(window=33, sinks=2, cu_seqlens=cu)
    out, lse = dr.window_attn_fwd(q, k, v, **kw)
    grads = dr.window_attn_bwd(q, k, v, out, lse, do, **kw)
    into = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    g_into = tuple(torch.full_like(x, 7.0) for x in (q, k, v))
    a, b = dr.window_attn_fwd(q, k, v, out=into[0], lse=into[1], **kw)
    assert a.data_ptr() == into[0].data_ptr() and b.data_ptr() == into[1].data_ptr()
    g = dr.window_attn_bwd(q, k, v, out, lse, do, grads=g_into, **kw)
    for x, y in zip((out, lse) + grads, (a, b) + g):
        assert torch.equal(x[:, 7:200], y[:, 7:200])
        assert (y[:, :7] == 7).all() and (y[:, 200:] == 7).all()
        assert (x[:, :7] == 0).all() and (x[:, 200:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,cu", [(2, 150, None), (1, 300, [0, 100, 290])])
def test_rows_of_a_fused_projection(dr, B, T, cu, dtype):
    Hq, Hk, d = 6, 2, 64
    q, k, v, do = (x.cuda() for x in make(B, T, Hq, Hk, d, dtype, seed=2))
    cu = None if cu is None else torch.tensor(cu, dtype=torch.int64).cuda()
    kw = dict(window=70, sinks=2, cu_seqlens=cu)
    out, lse = dr.window_attn_fwd(q, k, v, **kw)
    grads = dr.window_attn_bwd(q, k, v, out, lse, do, **kw)
    row = torch.cat((q, k, v), 2)
    parts = row.split((Hq, Hk, Hk), 2)
    o2, l2 = dr.window_attn_fwd(*parts, **kw)
    d_row = torch.zeros_like(row)
    g2 = dr.window_attn_bwd(*parts, o2, l2, do, grads=d_row.split((Hq, Hk, Hk), 2), **kw)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    for x, y in zip(grads, g2):
        assert torch.equal(x, y)
    assert torch.equal(d_row, torch.cat(grads, 2))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,cu", [(2, 130, None), (3, 1, None), (1, 300, [0, 100, 290])])
def test_backward_takes_views(dr, B, T, cu, dtype):
    """Results that are the front of padded ones, gradients that are transposed or expanded: the bits of
    the contiguous call, on this stream, on another one and in a graph."""
    q, k, v, do = (x.cuda() for x in make(B, T, 4, 2, 64, dtype, seed=12))
    kw = dict(window=40, sinks=2, cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int64).cuda())
    out, lse = dr.window_attn_fwd(q, k, v, **kw)
    pad = lambda x: torch.cat((x, torch.full_like(x[:, :1], float("nan")).expand(-1, 5, *x.shape[2:])), 1)[:, :T]
    views = [(pad(out), pad(lse), do.transpose(1, 2).contiguous().transpose(1, 2), do),
             (out, lse.transpose(1, 2).contiguous().transpose(1, 2), do[:1, :1, :, :1].expand(B, T, 4, 64),
              do[:1, :1, :, :1].expand(B, T, 4, 64).contiguous())]
    side = torch.cuda.Stream()
    for o, l, d, d_whole in views:
        want = dr.window_attn_bwd(q, k, v, out, lse, d_whole, **kw)
        torch.cuda.synchronize()
        got = [dr.window_attn_bwd(q, k, v, o, l, d, **kw), dr.window_attn_bwd(q, k, v, o, l, d, stream=side, **kw)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(dr.window_attn_bwd(q, k, v, o, l, d, **kw))
        graph.replay()
        torch.cuda.synchronize()
        for g in got:
            for x, y in zip(want, g):
                assert torch.equal(x, y)
    with pytest.raises(ValueError):
        dr.window_attn_bwd(q, k, v, out, lse.transpose(1, 2), do, **kw)
    with pytest.raises(ValueError):
        dr.window_attn_bwd(q, k, v, out, lse, do.cpu(), **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size,scale", [(20.0, None), (1.0, 2.0), (1e-3, None), (0.0, None), (1.0, 1e-4)])
def test_sharp_and_flat_weights(dr, size, scale, dtype):
    both(dr, 1, 300, 2, 1, 128, 90, 2, dtype, seed=11, size=size, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rising_scores(dr, dtype):
    """Every key beats all before it, so the running maximum rises at each."""
    T, d = 330, 64
    q, k, v, do = make(1, T, 1, 1, d, dtype, seed=1)
    q = torch.ones_like(q)
    k = (torch.arange(T).float()[None, :, None, None] / 8).expand(1, T, 1, d).to(DT[dtype]).contiguous()
    got = run(dr, q, k, v, do, 0, 0)
    R, E = reference(q, k, v, 0, 0, d ** -0.5, dtype == "bf16", None, do)
    compare(got, R, E)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_windows_and_sinks_beyond_the_sequence(dr, dtype):
    q, k, v, do = make(1, 200, 2, 1, 64, dtype, seed=4)
    a = run(dr, q, k, v, do, 0, 0)
    for window, sinks in ((200, 0), (1 << 40, 0), (0, 1 << 40), (3, 200), (1, 1 << 40), (1 << 62, 1 << 62)):
        b = run(dr, q, k, v, do, window, sinks)
        R, E = reference(q, k, v, 0, 0, 64 ** -0.5, dtype == "bf16", None, do)
        compare(b, R, E)
        if sinks == 0:
            for n in a:
                assert torch.equal(a[n], b[n])


@pytest.mark.gpu
def test_gradients_against_differences(dr):
    q, k, v, do = (x.cuda() for x in make(1, 90, 2, 1, 64, "f32", seed=8))
    kw = dict(window=20, sinks=2)
    out, lse = dr.window_attn_fwd(q, k, v, **kw)
    grads = dr.window_attn_bwd(q, k, v, out, lse, do, **kw)
    loss = lambda *x: (dr.window_attn_fwd(*x, **kw)[0].double() * do.double()).sum().item()
    g = torch.Generator().manual_seed(1)
    for n in range(3):
        x = [q, k, v]
        step = torch.randn(x[n].shape, generator=g).cuda()
        step /= step.norm()
        h = 2.0 ** -5
        diffs = []
        for f in (h, h / 2):
            up, dn = list(x), list(x)
            up[n], dn[n] = x[n] + f * step, x[n] - f * step
            diffs.append((loss(*up) - loss(*dn)) / (2 * f))
        diff = (4 * diffs[1] - diffs[0]) / 3        # off by h^4
        want = (grads[n].double() * step.double()).sum().item()
        # the loss is a sum of 11520 terms of unit size, each off by 2^-17 at random: 108 * 2^-17 / h
        assert abs(diff - want) <= 2 * 108 * U17 / h + 1e-3 * abs(want), n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_calls_give_equal_bits(dr, dtype):
    q, k, v, do = make(2, 500, 4, 2, 128, dtype, seed=6)
    a, b = (run(dr, q, k, v, do, 150, 5) for _ in range(2))
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_streams_and_graphs(dr, dtype):
    """On a side stream, and captured twice with one workspace and replayed on other inputs."""
    xs = [make(1, 300, 4, 2, 64, dtype, seed=s) for s in range(2)]
    cu = torch.tensor([0, 120, 290], dtype=torch.int64).cuda()
    kw = dict(window=64, sinks=3, cu_seqlens=cu)
    want = [run(dr, *x, 64, 3, cu=[0, 120, 290]) for x in xs]
    side = torch.cuda.Stream()
    c = [x.cuda() for x in xs[0]]
    torch.cuda.synchronize()
    out, lse = dr.window_attn_fwd(*c[:3], stream=side, **kw)
    g = dr.window_attn_bwd(*c[:3], out, lse, c[3], stream=side, **kw)
    side.synchronize()
    for n, x in zip(want[0], (out, lse) + g):
        assert torch.equal(x, want[0][n]), n
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    graphs = []
    for _ in range(2):
        ins = [x.cuda() for x in xs[0]]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, lse = dr.window_attn_fwd(*ins[:3], **kw)
            g = dr.window_attn_bwd(*ins[:3], out, lse, ins[3], workspace=ws, **kw)
        graphs.append((graph, ins, (out, lse) + g))
    for i, j in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for dst, src in zip(graphs[i][1], xs[j]):
            dst.copy_(src)
        graphs[i][0].replay()
        torch.cuda.synchronize()
        for n, x in zip(want[j], graphs[i][2]):
            assert torch.equal(x, want[j][n]), (i, j, n)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_first_tokens_with_most_of_the_weight(dr, d):
    """A row whose weight is nearly all one key's has score gradients that are differences of nearly equal numbers; that they
    add up to zero over the row has to hold for those that the kernel forms, whatever the roundings of out and lse (here 8 u at
    random, as of a forward with other sums), or dq is off by the key's size.  fp32, u = 2^-24, roundings at random: a product do.v is off by 4 u
    sqrt(d) (sums of 16 channels of size 4, 8 of them), a weight by 8 u of it; moving score gradient j by e with the sum
    kept zero moves dq by scale e (k_j - sum p k).  The sum over the keys and the result: 4 u of the terms' norm and of dq.  The
    bound is the 2-norm of these over all elements, times 2 for what 73 rows may deviate from the mean."""
    u, scale, cu, sinks = 2.0 ** -24, d ** -0.5, [0, 1, 9, 20, 31, 60, 73], 8
    q, k, v, do = make(1, 73, 6, 3, d, "f32", seed=13)
    lean = torch.randn((3, d), generator=torch.Generator().manual_seed(14))
    lean = lean / lean.norm(dim=1, keepdim=True) * d ** 0.25
    q = q + lean.repeat_interleave(2, 0)
    for lo in cu[:-1]:
        for t in range(lo, min(lo + 4, 73)):
            k[:, t] += 3.0 * lean
    R, _ = reference(q, k, v, 0, sinks, scale, False, cu, do)
    g = torch.Generator().manual_seed(15)
    out, lse = (R[n] * (1 + 8 * u * torch.randn(R[n].shape, generator=g, dtype=torch.float64)) for n in ("out", "lse"))
    c = [x.cuda() for x in (q, k, v, out.float(), lse.float(), do)]
    dq, _, _ = dr.window_attn_bwd(*c, sinks=sinks, cu_seqlens=torch.tensor(cu).cuda())
    bound = 0.0
    for lo, hi in zip(cu[:-1], cu[1:]):
        for h in range(6):
            Q, K, V, D = (x[0, lo:hi, i].double() for x, i in ((q, h), (k, h // 2), (v, h // 2), (do, h)))
            s = (scale * Q @ K.T).masked_fill(~visible(hi - lo, 0, sinks), -math.inf)
            p = torch.softmax(s, 1)
            dp = D @ V.T
            ds = p * (dp - (p * dp).sum(1, keepdim=True))
            e = 8 * u * ds.abs() + 4 * u * d ** 0.5 * p
            apart = K[None] - (p @ K)[:, None]                      # [i, j, channel]
            terms = (e[:, :, None] * apart) ** 2 + (4 * u * ds[:, :, None] * K[None]) ** 2
            bound += scale ** 2 * terms.sum().item()
    bound = 2 * (bound + (4 * u * R["dq"].norm().item()) ** 2) ** 0.5
    off = (dq.double().cpu() - R["dq"]).norm().item()
    assert off <= bound, f"{off / bound:.2f} of the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sequences_without_tokens(dr, dtype):
    q, k, v, do = make(1, 40, 2, 1, 64, dtype, seed=3)
    for cu in ([0, 0, 0], [40, 40], [17] * 300):
        got = run(dr, q, k, v, do, 9, 2, cu=cu)
        assert all((x == 0).all() for x in got.values())
    both(dr, 1, 40, 2, 1, 64, 9, 2, dtype, seed=3)      # and the next call is as ever


@pytest.mark.gpu
def test_no_tokens(dr):
    x = torch.empty((2, 0, 2, 64), device="cuda")
    out, lse = dr.window_attn_fwd(x, x, x)
    assert out.shape == x.shape and lse.shape == (2, 0, 2)
    assert all(g.shape == x.shape for g in dr.window_attn_bwd(x, x, x, out, lse, x))


# ------------------------------------------------------------------ one token over the cache
def paged(k, v, lens, page, seed, garbage, drop=None):
    """Sequences [B, T, Hk, d] in pages in any order, `garbage` in every slot that holds no token; pages for
    which drop(b, first, end) are not there."""
    B, T, Hk, d = k.shape
    most = max(1, -(-max(lens) // page))
    g = torch.Generator().manual_seed(seed)
    slots = [(b, p) for b in range(B) for p in range(-(-lens[b] // page))
             if not (drop and drop(b, p * page, min(lens[b], (p + 1) * page)))]
    n = len(slots) + 3
    order = torch.randperm(n, generator=g)
    pages = torch.full((B, most), -1, dtype=torch.int32)
    if drop:
        pages[:, ::2] = n + 5          # any number outside is no page
    kc, vc = (torch.full((n, Hk, page, d), garbage, dtype=k.dtype) for _ in range(2))
    for i, (b, p) in enumerate(slots):
        at = int(order[i])
        pages[b, p] = at
        e = min(lens[b], (p + 1) * page) - p * page
        kc[at, :, :e] = k[b, p * page:p * page + e].transpose(0, 1)
        vc[at, :, :e] = v[b, p * page:p * page + e].transpose(0, 1)
    return kc, vc, pages


def step_reference(q, k, v, lens, window, sinks, scale, bf16, drop=None, page=16):
    B, Hq, d = q.shape
    g = Hq // k.shape[2]
    R = dict(out=torch.zeros(B, Hq, d, dtype=torch.float64), lse=torch.full((B, Hq), -math.inf, dtype=torch.float64))
    E = dict(out=torch.zeros(B, Hq, d, dtype=torch.float64), lse=torch.zeros(B, Hq, dtype=torch.float64))
    for b, n in enumerate(lens):
        j = torch.arange(max(n, 0))
        see = ((n - 1 - j < window) if window else torch.ones_like(j, dtype=torch.bool)) | (j < sinks)
        if drop:
            see &= torch.tensor([not drop(b, x // page * page, min(n, (x // page + 1) * page)) for x in range(n)], dtype=torch.bool)
        j = j[see]
        if len(j) == 0:
            continue
        for h in range(Hq):
            Q, K, V = q[b, h].double(), k[b, j, h // g].double(), v[b, j, h // g].double()
            s = scale * K @ Q
            u = U17 * max(1.0, float((scale * K.abs() @ Q.abs()).max()) / 16)
            lse = torch.logsumexp(s, 0)
            p = (s - lse).exp()
            o = p @ V
            R["out"][b, h], R["lse"][b, h] = o, lse
            E["out"][b, h] = (u + (2.0 ** -16 if bf16 else 0)) * (p @ V.abs()) + (HALF * o.abs() if bf16 else 0)
            E["lse"][b, h] = u * (1 + abs(float(lse)))
    return R, E


def step_case(dr, lens, Hq, Hk, d, window, sinks, page, dtype, seed=0, garbage=float("nan"), drop=None, scale=None, ws=None):
    B, T = len(lens), max(max(lens), 1)
    q, k, v, _ = make(B, T, Hk, Hk, d, dtype, seed)
    q = make(B, 1, Hq, Hk, d, dtype, seed + 1)[0][:, 0].contiguous()
    kc, vc, pages = paged(k, v, [max(n, 0) for n in lens], page, seed, garbage, drop)
    got = dr.window_attn_step(q.cuda(), kc.cuda(), vc.cuda(), pages.cuda(), torch.tensor(lens).cuda(), window=window,
                              sinks=sinks, scale=scale, return_lse=True, workspace=ws)
    torch.cuda.synchronize()
    assert dr.lib().dr_get_device_status(None) == 0
    R, E = step_reference(q, k, v, lens, window, sinks, scale or d ** -0.5, dtype == "bf16", drop, page)
    out, lse = (x.double().cpu() for x in got)
    none = R["lse"] == -math.inf
    assert (out[none] == 0).all() and (lse[none] == -math.inf).all()
    for n, x in (("out", out), ("lse", lse)):
        x, r, e = x[~none], R[n][~none], E[n][~none]
        assert torch.isfinite(x).all(), n
        if x.numel():
            worst = ((x - r).abs() / (e + 1e-30)).max().item()
            assert worst <= 1, f"{n}: {worst:.3f} of the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (50, 4), (64, 100), (16, 16), (1000, 17)])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (6, 2), (16, 1), (20, 1), (35, 1)])
def test_step(dr, Hq, Hk, window, sinks, d, dtype):
    step_case(dr, [1, 0, 15, 16, 17, 300, 129, -3, 64, 0], Hq, Hk, d, window, sinks, 16, dtype, seed=Hq + window)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [16, 48, 64, 256, 1024])
def test_step_page_sizes(dr, page, dtype):
    step_case(dr, [1000, 5, 700, 257], 4, 2, 64, 333, 5, page, dtype, seed=page)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,Hq,Hk,window", [([5000], 4, 1, 0), ([9000, 1, 4001], 2, 2, 0), ([30000], 8, 1, 20000), ([2500] * 3, 17, 1, 0)])
def test_step_long_contexts_are_cut(dr, lens, Hq, Hk, window, dtype):
    step_case(dr, lens, Hq, Hk, 128 if dtype == "bf16" else 64, window, 4, 64, dtype, seed=len(lens))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_many_sequences(dr, dtype):
    lens = [(i * 37) % 90 for i in range(700)]
    step_case(dr, lens, 2, 1, 64, 40, 2, 16, dtype, seed=1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_pages_that_are_not_there(dr, dtype):
    # given back behind the window (nothing visible is lost), and missing inside it
    step_case(dr, [700, 90, 10], 4, 2, 64, 100, 20, 16, dtype, garbage=float("inf"),
              drop=lambda b, a, e: e <= [700, 90, 10][b] - 100 and a >= 20)
    step_case(dr, [700, 90, 10], 4, 2, 64, 0, 0, 16, dtype, seed=1, drop=lambda b, a, e: (a // 16) % 3 == 1 or b == 2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_lengths_behind_the_table(dr, dtype):
    """Tokens behind the table's pages are not there; the window still ends at the length."""
    q, k, v, _ = make(2, 64, 2, 2, 64, dtype, seed=3)
    q = q[:, 0].contiguous()
    kc, vc, pages = paged(k, v, [64, 64], 16, 0, 0.0)
    big = torch.tensor([70, 1 << 40])
    got = dr.window_attn_step(q.cuda(), kc.cuda(), vc.cuda(), pages.cuda(), big.cuda(), window=20, sinks=3, return_lse=True)
    k2, v2 = (torch.cat((x, torch.zeros_like(x[:, :6])), 1) for x in (k, v))
    R, E = step_reference(q, k2, v2, [70, 3], 20, 3, 0.125, dtype == "bf16", lambda b, a, e: a >= 64)
    for n, x in zip(("out", "lse"), got):
        assert ((x.double().cpu() - R[n]).abs() <= E[n] + 1e-30).all(), n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,Hk", [("f32", 16), ("bf16", 32)])
def test_step_units_that_pass_31_bits(dr, Hk, dtype):
    """A context of 2^30 tokens, nearly all of its pages not there: its groups of tokens times its heads are more than 2^31.  A
    short one behind it."""
    page, d, most = 1024, 64, 1 << 20
    there = [0, 5, most // 2 + 1, most - 1]
    n = len(there) * page
    q, k, v, _ = make(2, n, Hk, Hk, d, dtype, seed=31)
    q = q[:, 0].contiguous()
    kc, vc = (torch.cat((x[0].view(4, page, Hk, d), x[1, :page][None])).transpose(1, 2).contiguous() for x in (k, v))
    pages = torch.full((2, most), -1, dtype=torch.int32)
    pages[0, there] = torch.arange(4, dtype=torch.int32)
    pages[1, 0] = 4
    assert Hk * (2 ** 30 // (16 if dtype == "bf16" else 8) + 1) >= 2 ** 31
    got = dr.window_attn_step(q.cuda(), kc.cuda(), vc.cuda(), pages.cuda(), torch.tensor([1 << 30, 40]).cuda(), return_lse=True)
    torch.cuda.synchronize()
    assert dr.lib().dr_get_device_status(None) == 0
    # (tokens that are not there take no part, so those that are may stand side by side)
    R, E = step_reference(q, k, v, [n, 40], 0, 0, d ** -0.5, dtype == "bf16")
    for name, x in zip(("out", "lse"), got):
        worst = ((x.double().cpu() - R[name]).abs() / (E[name] + 1e-30)).max().item()
        assert worst <= 1, f"{name}: {worst:.3f} of the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_in_graphs_with_one_workspace(dr, dtype):
    """Two captured steps that share a workspace, their lengths updated on the device between replays."""
    lens = [4000, 17, 900]
    q, k, v, _ = make(3, 4100, 2, 1, 64, dtype, seed=2)
    q = q[:, 0].contiguous().cuda()
    kc, vc, pages = (x.cuda() for x in paged(k, v, [4100] * 3, 32, 1, float("nan")))
    ws = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    want = {n: dr.window_attn_step(q, kc, vc, pages, torch.tensor(lens).cuda() + n, window=3000, sinks=2, return_lse=True)
            for n in range(4)}
    graphs = []
    for _ in range(2):
        ln = torch.tensor(lens).cuda()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = dr.window_attn_step(q, kc, vc, pages, ln, window=3000, sinks=2, return_lse=True, workspace=ws)
            ln += 1
        graphs.append((graph, res, ln))
    for n in range(4):
        for graph, res, _ in graphs:
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(res[0], want[n][0]) and torch.equal(res[1], want[n][1])


# ------------------------------------------------------------------ filling the cache
def define_rope(x, w, pos, rot, base, norm, layout, eps, scale):
    d = x.shape[-1]
    x = x.double()
    if norm != "none":
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / (d if norm == "rms" else 1) + eps)
    if w is not None:
        x = x * w.double()
    f = torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    ang = pos.double()[:, None] * f
    c, s = scale * ang.cos()[:, None], scale * ang.sin()[:, None]
    i = torch.arange(rot // 2)
    a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def near_rope(got, want, bf16, what, pos):
    """The bound of the query/key preparation's tests: 2^-16 of max(RMS, |value|), and bf16's rounding;
    and what far positions add: a frequency is good to 2^-52.6 turns a position (the header's bound), the
    reference's 64-bit angle to 2^-53 of itself, together at most p (2 pi 2^-52.6 + 2^-53) < p 2^-49 radians of the
    pair's size, itself at most sqrt(2) times the largest value."""
    rms = want.square().mean().sqrt().clamp(min=1e-30)
    bound = 2.0 ** -16 * torch.maximum(want.abs(), rms) + (HALF * want.abs() if bf16 else 0)
    if want.numel():
        bound = bound + (pos.double() * 2.0 ** -49 * math.sqrt(2) * want.abs().max())[:, None, None]
    worst = ((got.double() - want).abs() / bound).max().item() if want.numel() else 0.0
    assert worst <= 1, f"{what}: {worst:.3f} of the bound"


def append_case(dr, rows, start, Hq, Hk, d, rot, page, dtype, norm="rms", layout="half", cu=None, n_tok=None, drop=(), fused=False,
                seed=0, in_place=False, max_pages=None, given=True):
    """rows[n] tokens of each sequence; cu None: one each."""
    g = torch.Generator().manual_seed(seed)
    N = len(rows)
    n_tok = n_tok or (N if cu is None else cu[-1])
    dt = DT[dtype]
    qkv = torch.randn((n_tok, Hq + 2 * Hk, d), generator=g).to(dt)
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g) for _ in range(2)) if norm == "rms" else (None, None)
    most = max_pages or max(1, max(-(-(max(s, 0) + r) // page) for s, r in zip(start, rows)))
    n_pages = N * most + 2
    pages = torch.randperm(n_pages, generator=g)[:N * most].to(torch.int32).view(N, most)
    for n, p, x in drop:
        pages[n, p] = x
    kc, vc = (torch.randn((n_pages, Hk, page, d), generator=g).to(dt) for _ in range(2))
    # by the definition
    seq, pos = [-1] * n_tok, [0] * n_tok
    for n in range(N):
        lo, hi = (n, n + 1) if cu is None else (cu[n], cu[n + 1])
        for t in range(lo, hi):
            if start[n] >= 0:
                seq[t], pos[t] = n, start[n] + t - lo
    live = [t for t in range(n_tok) if seq[t] >= 0]
    P = torch.tensor([pos[t] for t in live])
    base = 10000.0
    parts = qkv.split((Hq, Hk, Hk), 1)
    want_q = define_rope(parts[0][live], wq, P, rot, base, norm, layout, 1e-6, 1.0) if Hq else None
    want_k = define_rope(parts[1][live], wk, P, rot, base, norm, layout, 1e-6, 1.0)
    cu_t = None if cu is None else torch.tensor(cu, dtype=torch.int64).cuda()
    c = qkv.cuda()
    q, k, v = c.split((Hq, Hk, Hk), 1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    kd, vd = kc.cuda(), vc.cuda()
    cuda = lambda x: None if x is None else x.cuda()
    into = None
    if given and Hq:
        into = q if in_place else torch.full((n_tok, Hq, d), 7.0, dtype=dt, device="cuda")
    table = dr.rope_table(rot, base=base) if rot else None
    got = dr.kv_append(q if Hq else None, k, v, table, kd, vd, pages.cuda(), torch.tensor(start).cuda(), cu_seqlens=cu_t,
                       norm=norm, wq=cuda(wq) if Hq else None, wk=cuda(wk), layout=layout, q_out=into)
    bf = dtype == "bf16"
    if Hq:
        got = got.cpu()
        near_rope(got[live], want_q, bf, "q", P)
        rest = [t for t in range(n_tok) if seq[t] < 0]
        keep = parts[0][rest] if in_place else torch.full((len(rest), Hq, d), 7.0 if given else 0.0, dtype=dt)
        assert torch.equal(got[rest], keep)
    else:
        assert got is None
    touched = torch.zeros((n_pages, page), dtype=torch.bool)
    hits_k, hits_v, src = [], [], []
    for i, t in enumerate(live):
        p = pos[t] // page
        pg = int(pages[seq[t], p]) if p < most else -1
        if 0 <= pg < n_pages:
            touched[pg, pos[t] % page] = True
            hits_k.append(kd[pg, :, pos[t] % page].cpu())
            hits_v.append(vd[pg, :, pos[t] % page].cpu())
            src.append(i)
    if src:
        near_rope(torch.stack(hits_k), want_k[src], bf, "k", P[src])
        assert torch.equal(torch.stack(hits_v), parts[2][live][src])
    for before, after in ((kc, kd), (vc, vd)):     # every other slot is as it was
        m = touched[:, None, :, None].expand_as(before)
        assert torch.equal(torch.where(m, before, after.cpu()), before)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 0)])
@pytest.mark.parametrize("norm,layout", [("rms", "half"), ("l2", "interleaved"), ("none", "half")])
def test_append_tokens(dr, norm, layout, d, rot, dtype):
    append_case(dr, [1] * 9, [0, 15, 16, -1, 100, 31, 47, -5, 48], 3, 2, d, rot, 16, dtype, norm, layout, seed=d + rot)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [16, 80, 256])
@pytest.mark.parametrize("fused,given,in_place", [(False, True, False), (True, False, False), (True, True, True)])
def test_append_prompts(dr, fused, given, in_place, page, dtype):
    cu = [3, 40, 40, 41, 150, 160, 200]
    append_case(dr, [37, 0, 1, 109, 10, 40], [0, 5, 16, 70, -1, 3], 4, 2, 64, 64, page, dtype, cu=cu, n_tok=210,
                drop=[(0, 0, -1), (3, 0, 1000)], fused=fused, given=given, in_place=in_place, seed=page)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_without_queries_and_behind_the_table(dr, dtype):
    append_case(dr, [1] * 4, [0, 1, 2, 3], 0, 3, 128, 128, 16, dtype, seed=1)
    append_case(dr, [1] * 3, [15, 40, 1 << 40], 2, 1, 64, 64, 16, dtype, max_pages=2, seed=2, norm="none")
    append_case(dr, [70], [0], 2, 1, 64, 64, 16, dtype, cu=[0, 70], max_pages=3, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_rows_of_no_sequence_may_hold_anything(dr, dtype):
    dt = DT[dtype]
    q, k, v = (torch.full((4, 2, 64), float("nan"), dtype=dt, device="cuda") for _ in range(3))
    kc, vc = (torch.ones((3, 2, 16, 64), dtype=dt, device="cuda") for _ in range(2))
    pages = torch.tensor([[0], [1], [2], [1]], dtype=torch.int32).cuda()
    out = dr.kv_append(q, k, v, dr.rope_table(64), kc, vc, pages, torch.tensor([-1, -2, -1, -9]).cuda(), eps=0.0)
    assert (out == 0).all() and (kc == 1).all() and (vc == 1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_where_positions_end(dr, dtype):
    dt = DT[dtype]
    q, k, v = (torch.randn((7, h, 64), device="cuda").to(dt) for h in (2, 1, 1))
    kc, vc = (torch.ones((2, 1, 16, 64), dtype=dt, device="cuda") for _ in range(2))
    pages = torch.tensor([[0], [1]], dtype=torch.int32).cuda()
    out = torch.full_like(q, 7.0)
    dr.kv_append(q, k, v, dr.rope_table(64), kc, vc, pages, torch.tensor([2 ** 63 - 2, -2 ** 63]).cuda(),
                 cu_seqlens=torch.tensor([0, 4, 7]).cuda(), q_out=out)
    assert (kc == 1).all() and (vc == 1).all()
    assert torch.isfinite(out[:2]).all() and not (out[:2] == 7).any() and (out[2:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_many_heads_of_many_sequences(dr, dtype):
    append_case(dr, [1] * 300, [5 * n - 3 for n in range(300)], 70, 10, 64, 32, 16, dtype, seed=6, fused=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seed", range(20))
def test_drawn_appends(dr, seed, dtype):
    rng = random.Random(seed)
    d, Hk, N = rng.choice([64, 128]), rng.randint(1, 8), log_int(rng, 1, 40)
    packed = rng.random() < 0.6
    rows = [rng.choice([0, 1, log_int(rng, 1, 60)]) if packed else 1 for _ in range(N)]
    cu = [0] + [int(x) for x in torch.tensor(rows).cumsum(0)] if packed else None
    if packed and cu[-1] == 0:
        rows, cu = [3] * N, [3 * n for n in range(N + 1)]
    start = [rng.choice([-1, 0, rng.randint(0, 300), rng.randint(0, 300)]) for _ in range(N)]
    fused, given = rng.random() < 0.5, rng.random() < 0.7
    append_case(dr, rows, start, Hk * rng.choice([0, 1, 2, 3, 4, 8]), Hk, d, rng.choice([0, d, d // 2, d // 4]), 16 << rng.randint(0, 4), dtype,
                rng.choice(["rms", "l2", "none"]), rng.choice(["half", "interleaved"]), cu, fused=fused, given=given,
                in_place=fused and given and rng.random() < 0.5, seed=seed)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_in_a_graph(dr, dtype):
    q, k, v, _ = make(1, 3, 2, 2, 64, dtype, seed=4)
    q, k, v = (x[0].cuda() for x in (q, k, v))
    table = dr.rope_table(64)
    pages = torch.arange(6, dtype=torch.int32).view(3, 2).cuda()
    caches = [torch.zeros((6, 2, 16, 64), dtype=DT[dtype], device="cuda") for _ in range(4)]
    start = torch.tensor([0, 14, 30]).cuda()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dr.kv_append(q, k, v, table, caches[0], caches[1], pages, start)
        start += 1
    for n in range(3):
        graph.replay()
        want = dr.kv_append(q, k, v, table, caches[2], caches[3], pages, torch.tensor([0, 14, 30]).cuda() + n)
        assert torch.equal(got, want)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pages_behind_four_gigabytes(dr, dtype):
    """The same pages' contents at either end of a cache of more than 2^31 values: the same bits."""
    dt, Hk, d, page, n_pages = DT[dtype], 8, 128, 16, 132000
    q, k, v, _ = make(1, 40, 16, Hk, d, dtype, seed=21)
    q, k, v = (x[0].cuda() for x in (q, k, v))
    kc, vc = (torch.empty((n_pages, Hk, page, d), dtype=dt, device="cuda") for _ in range(2))
    table, start, cu = dr.rope_table(d), torch.tensor([0]).cuda(), torch.tensor([0, 40]).cuda()
    got = []
    for first in (0, n_pages - 3):
        kc[first:first + 3] = 0
        vc[first:first + 3] = 0
        pages = torch.arange(first, first + 3, dtype=torch.int32).view(1, 3).cuda()
        q1 = dr.kv_append(q, k, v, table, kc, vc, pages, start, cu_seqlens=cu)
        out, lse = dr.window_attn_step(q1[39:], kc, vc, pages, start + 40, window=30, sinks=2, return_lse=True)
        got.append((q1, out, lse, kc[first:first + 3].clone(), vc[first:first + 3].clone()))
    for x, y in zip(*got):
        assert torch.isfinite(x).all() and torch.equal(x, y)


@pytest.mark.gpu
def test_millions_of_tokens_in_sight(dr):
    """Items of 36,000 key tiles (the last one's second stage without rows): waits that last an item do not run out.  Of a sample of rows, by
    the docstring's bounds and what long sums add at worst: a tensor-core accumulator is off by one step, 2^-23, with each of
    its T / 16 additions, a softmax's sum by half a step, 2^-24, with each of its four chains' T / 4.  The gradients' reference
    takes out and lse as they are given."""
    T, d = 256 * 18359 + 96, 64
    g = torch.Generator(device="cuda").manual_seed(41)
    q, k, v, do = (torch.randn((1, T, 1, d), generator=g, device="cuda") for _ in range(4))
    q, k, v, do = (x.to(torch.bfloat16) for x in (q, k, v.mul_(0.5).add_(1.0), do))
    out, lse = dr.window_attn_fwd(q, k, v)
    grads = dr.window_attn_bwd(q, k, v, out, lse, do)
    torch.cuda.synchronize()
    assert dr.lib().dr_get_device_status(None) == 0
    for x in (out, lse) + grads:
        assert torch.isfinite(x).all()
    scale, steps, chain = d ** -0.5, T / 16 * 2.0 ** -23, T / 4 * 2.0 ** -24
    last = 64
    K, V = k[0, :, 0].double(), v[0, :, 0].double()
    dk, dv, e_dk, e_dv = (torch.zeros((last, d), dtype=torch.float64, device="cuda") for _ in range(4))

    def near(what, got, want, bound):
        worst = ((got.double() - want).abs() / bound).max().item()
        assert worst <= 1, f"{what}: {worst:.3f} of the bound"

    rows = torch.cat((torch.tensor([0, 1, 127, 128, 255, 256, 5000, T // 3, T // 2 + 77, T - 300, T - 97, T - 96, T - 70, T - 66, T - 65]),
                      torch.arange(T - last, T))).cuda()
    for at in rows.split(8):
        Q, D, o, l = q[0, at, 0].double(), do[0, at, 0].double(), out[0, at, 0].double(), lse[0, at, 0].double()
        n = int(at.max()) + 1
        s = (scale * Q @ K[:n].T).masked_fill(torch.arange(n, device="cuda")[None] > at[:, None], -math.inf)
        u = U17 * max(1.0, scale * float((Q.abs() @ K[:n].abs().T).max()) / 16)
        want_l = torch.logsumexp(s, 1)
        p = (s - want_l[:, None]).exp()
        want_o, size = p @ V[:n], p @ V[:n].abs()
        near("lse", l, want_l, u * (1 + want_l.abs()) + chain)
        near("out", o, want_o, (u + HALF + steps + chain) * size + HALF * want_o.abs())
        p = (s - l[:, None]).exp()
        ds = p * (D @ V[:n].T - (D * o).sum(1, keepdim=True))
        off = u * p * (D.abs() @ V[:n].abs().T + (D * o).abs().sum(1, keepdim=True)) + HALF * ds.abs()
        want = scale * ds @ K[:n]
        near("dq", grads[0][0, at, 0], want, scale * (off + steps * ds.abs()) @ K[:n].abs() + HALF * want.abs())
        if n > T - last:       # (rows in front of these keys do not see them: p is 0)
            dk += torch.nn.functional.pad(scale * ds[:, T - last:].T @ Q, (0, 0, 0, T - n))
            dv += torch.nn.functional.pad(p[:, T - last:].T @ D, (0, 0, 0, T - n))
            e_dk += torch.nn.functional.pad(scale * off[:, T - last:].T @ Q.abs(), (0, 0, 0, T - n))
            e_dv += torch.nn.functional.pad((u + HALF) * p[:, T - last:].T @ D.abs(), (0, 0, 0, T - n))
    near("dk", grads[1][0, T - last:, 0], dk, e_dk + HALF * dk.abs())
    near("dv", grads[2][0, T - last:, 0], dv, e_dv + HALF * dv.abs())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_far_apart(dr, dtype):
    """Rows whose last one is more than 2^32 values behind the first: the same bits as next to one another."""
    T, apart = 1100, 1 << 22
    q, k, v, do = (x.cuda() for x in make(1, T, 2, 1, 64, dtype, seed=22))
    kw = dict(window=100, sinks=3)
    out, lse = dr.window_attn_fwd(q, k, v, **kw)
    grads = dr.window_attn_bwd(q, k, v, out, lse, do, **kw)
    room = torch.empty(T * apart, dtype=DT[dtype], device="cuda")
    at = lambda h, first: room.as_strided((1, T, h, 64), (T * apart, apart, 64, 1), first)
    far = [at(h, 1024 * i) for i, h in enumerate((2, 1, 1, 2, 1, 1))]
    for x, y in zip(far, (q, k, v)):
        x.copy_(y)
    out2, lse2 = dr.window_attn_fwd(*far[:3], **kw)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for x, y in zip(grads, dr.window_attn_bwd(*far[:3], out, lse, do, grads=far[3:], **kw)):
        assert torch.equal(x, y)


# ------------------------------------------------------------------ together
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 3)])
def test_prompt_then_tokens(dr, window, sinks, dtype):
    """Prompts through the preparation and the attention, their keys and values into the cache, then token
    by token over the cache: the same results as the attention of the whole sequences."""
    lens, extra, Hq, Hk, d, page = [50, 1, 33], 20, 4, 2, 64, 16
    B, T = len(lens), max(lens) + extra
    g = torch.Generator().manual_seed(3)
    raw = torch.randn((B, T, Hq + 2 * Hk, d), generator=g).to(DT[dtype]).cuda()
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).cuda() for _ in range(2))
    table = dr.rope_table(d)
    kw = dict(window=window, sinks=sinks)
    q, k, v = raw.split((Hq, Hk, Hk), 2)
    qr, kr = dr.qk_norm_rope(q, k, table, wq=wq, wk=wk)
    full, _ = dr.window_attn_fwd(qr, kr, v, **kw)
    # prompts, packed
    rows = torch.cat([raw[b, :n] for b, n in enumerate(lens)])
    cu = torch.tensor([0, 50, 51, 84]).cuda()
    most = -(-T // page)
    pages = torch.randperm(B * most, generator=g).to(torch.int32).view(B, most).cuda()
    kc, vc = (torch.full((B * most, Hk, page, d), float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2))
    pq, pk, pv = rows.split((Hq, Hk, Hk), 1)
    start = torch.zeros(B, dtype=torch.int64).cuda()
    q1 = dr.kv_append(pq, pk, pv, table, kc, vc, pages, start, cu_seqlens=cu, wq=wq, wk=wk)
    for b, (a, e) in enumerate(zip([0, 50, 51], [50, 51, 84])):
        assert torch.equal(q1[a:e], qr[b, :e - a])          # the same preparation, bit by bit
    ends = torch.tensor(lens).cuda()
    for t in range(extra):
        at = ends + t
        tok = torch.stack([raw[b, n + t] for b, n in enumerate(lens)])
        tq, tk, tv = tok.split((Hq, Hk, Hk), 1)
        q1 = dr.kv_append(tq, tk, tv, table, kc, vc, pages, at, wq=wq, wk=wk)
        out, _ = dr.window_attn_step(q1, kc, vc, pages, at + 1, **kw)
        want = torch.stack([full[b, n + t] for b, n in enumerate(lens)])
        bound = 2 ** -14 if dtype == "f32" else 0.03
        # fp32: two results within 2^-17 sum p |v| each; bf16: weights and results rounded, at most
        # 2^-8 (sum p |v| + |o|) and 2^-8 |o|, with |v| up to 4
        assert (out.double() - want.double()).abs().max().item() <= bound


# ------------------------------------------------------------------ refusals (no GPU)
def attn_desc(dr, **kw):
    d = dict(B=2, T=100, Hq=4, Hk=2, d=64, N=0, window=16, sinks=2, q_stride=0, k_stride=0, v_stride=0, dq_stride=0,
             dk_stride=0, dv_stride=0, dtype=dr.DR_BF16, zero_rest=0, reserved=0, scale=0.125)
    d.update(kw)
    return dr.AttnDesc(**d)


def step_desc(dr, **kw):
    d = dict(B=2, Hq=4, Hk=2, d=64, n_pages=8, page=16, max_pages=4, window=16, sinks=2, dtype=dr.DR_BF16, reserved=0, scale=0.125)
    d.update(kw)
    return dr.AttnStepDesc(**d)


def append_desc(dr, **kw):
    d = dict(n_tok=4, N=4, Hq=4, Hk=2, d=64, rot=64, q_stride=0, k_stride=0, v_stride=0, q_out_stride=0, n_pages=8, page=16,
             max_pages=4, dtype=dr.DR_BF16, norm=dr.DR_NORM_RMS, layout=dr.DR_ROPE_HALF, zero_rest=0, reserved=0, eps=1e-6, rot_scale=1.0)
    d.update(kw)
    return dr.KvAppendDesc(**d)


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), -1), (dict(T=-1), -1), (dict(Hq=0), -1), (dict(Hk=0), -1), (dict(Hq=3), -1), (dict(N=-1), -1), (dict(N=2), -1),
    (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(dtype=5), -1), (dict(reserved=1), -1), (dict(zero_rest=2), -1),
    (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(d=96), -2), (dict(d=256), -2), (dict(T=(1 << 30) + 1), -2), (dict(B=1 << 21), -2), (dict(q_stride=200), -1),
    (dict(k_stride=132), -1), (dict(v_stride=64), -1), (dict(dq_stride=8), -1), (dict(dk_stride=129), -1), (dict(dv_stride=1 << 32), -2)])
def test_bad_attention_descriptors(dr, bad, status):
    n = ctypes.c_size_t(0)
    assert dr.lib().dr_window_attn_bwd_workspace_bytes(ctypes.byref(attn_desc(dr, **bad)), ctypes.byref(n)) == status


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), -1), (dict(Hq=3), -1), (dict(Hk=0), -1), (dict(n_pages=0), -1), (dict(page=0), -1), (dict(max_pages=0), -1),
    (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(dtype=2), -1), (dict(reserved=1), -1), (dict(scale=0.0), -1), (dict(d=32), -2),
    (dict(page=24), -2), (dict(page=2048), -2), (dict(n_pages=1 << 31), -2), (dict(max_pages=1 << 28), -2)])
def test_bad_step_descriptors(dr, bad, status):
    n = ctypes.c_size_t(0)
    assert dr.lib().dr_window_attn_step_workspace_bytes(ctypes.byref(step_desc(dr, **bad)), ctypes.byref(n)) == status


def bwd_bytes(dr, **kw):
    n = ctypes.c_size_t(0)
    assert dr.lib().dr_window_attn_bwd_workspace_bytes(ctypes.byref(attn_desc(dr, **kw)), ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("dtype", ["DR_F32", "DR_BF16"])
@pytest.mark.parametrize("window,sinks", [(1024, 4), (1024, 128), (1024, 1024), (64, 200), (1, 1024), (1, 1), (65000, 500)])
def test_workspace_of_many_sequences(dr, window, sinks, dtype):
    """Only sequences longer than the window can have sums of sinks' rows, at most T / window of them: the
    workspace does not grow with the sequences behind that, and never past four times the gradients in fp32."""
    T, H, d = 65536, 8, 128
    kw = dict(B=1, T=T, Hq=H, Hk=H, d=d, window=window, sinks=sinks, dtype=getattr(dr, dtype))
    stats = 8 * T * H + 256
    few, many, most = (bwd_bytes(dr, N=n, **kw) for n in (1, 4096, 65536))
    assert all(stats - 256 <= x <= stats + 4 * 4 * T * 3 * H * d + 512 for x in (few, many, most))
    assert many == most
    # sums of one sequence's own blocks and of two chunks of queries for every `window` rows
    assert most <= stats + 512 + 4 * H * (-(-sinks // 128) * 128) * 2 * d * (3 * T // window + 1)


no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only without a GPU")
far = lambda i: ctypes.c_void_p((i + 1) << 32)      # disjoint addresses, never used


@no_gpu_only
@pytest.mark.parametrize("bad,status", [
    (dict(n_tok=-1), -1), (dict(N=0), -1), (dict(N=3), -1), (dict(Hk=0), -1), (dict(Hq=-1), -1), (dict(rot=80), -1), (dict(n_pages=0), -1),
    (dict(page=0), -1), (dict(max_pages=0), -1), (dict(dtype=3), -1), (dict(norm=4), -1), (dict(layout=2), -1), (dict(eps=-1.0), -1),
    (dict(rot_scale=float("nan")), -1), (dict(reserved=1), -1), (dict(zero_rest=3), -1), (dict(d=256), -2), (dict(rot=24), -2), (dict(page=40), -2),
    (dict(q_stride=8), -1), (dict(k_stride=132), -1), (dict(norm=0), -1), (dict(n_pages=1 << 28), -2)])
def test_bad_append_calls(dr, bad, status):
    assert dr.lib().dr_kv_append(ctypes.byref(append_desc(dr, **bad)), *[far(i) for i in range(8)], None, *[far(i) for i in range(9, 12)],
                                 None) == status


@no_gpu_only
def test_append_pointers_and_overlaps(dr):
    names = ("q", "k", "v", "wq", "wk", "table", "pages", "start", "cu", "q_out", "kc", "vc")
    desc = append_desc(dr)
    call = lambda **o: dr.lib().dr_kv_append(ctypes.byref(desc), *[o.get(n, None if n == "cu" else far(i)) for i, n in enumerate(names)], None)
    at = lambda n, off=0: ctypes.c_void_p(((names.index(n) + 1) << 32) + off)
    for n in ("q", "k", "v", "table", "pages", "start", "q_out", "kc", "vc"):
        assert call(**{n: None}) == dr.DR_ERR_INVALID, n
    for n in ("q", "k", "v", "q_out", "kc", "vc"):
        assert call(**{n: at(n, 8)}) == dr.DR_ERR_INVALID, n
    for n in ("start", "table"):
        assert call(**{n: at(n, 4)}) == dr.DR_ERR_INVALID, n
    for n in ("q", "k", "v", "wq", "wk", "table", "pages", "start", "q_out", "vc"):
        assert call(kc=at(n)) == dr.DR_ERR_INVALID, n
    for n in ("k", "v", "wq", "pages", "start", "kc", "vc"):
        assert call(q_out=at(n)) == dr.DR_ERR_INVALID, n
    assert call(q_out=at("q", 512)) == dr.DR_ERR_INVALID      # q_out is q or apart from it
    assert dr.lib().dr_kv_append(None, *[far(i) for i in range(12)], None) == dr.DR_ERR_INVALID


@no_gpu_only
def test_attention_pointers_and_overlaps(dr):
    lib = dr.lib()
    names = ("q", "k", "v", "cu", "out", "lse")
    desc = attn_desc(dr)
    at = lambda n, off=0: ctypes.c_void_p(((names.index(n) + 1) << 32) + off)
    call = lambda d=desc, **o: lib.dr_window_attn_fwd(ctypes.byref(d), *[o.get(n, far(i)) for i, n in enumerate(names)], None)
    assert lib.dr_window_attn_fwd(None, *[far(i) for i in range(6)], None) == dr.DR_ERR_INVALID
    for n in ("q", "k", "v", "out", "lse"):
        assert call(**{n: None}) == dr.DR_ERR_INVALID, n
        assert call(**{n: at(n, 2)}) == dr.DR_ERR_INVALID, n
    for n in ("q", "k", "v"):
        assert call(out=at(n)) == dr.DR_ERR_INVALID and call(lse=at(n, 64)) == dr.DR_ERR_INVALID, n
    assert call(lse=at("out")) == dr.DR_ERR_INVALID
    packed = attn_desc(dr, B=1, N=3)
    assert call(packed, cu=None) == dr.DR_ERR_INVALID and call(packed, cu=at("cu", 4)) == dr.DR_ERR_INVALID
    assert call(packed, lse=at("cu")) == dr.DR_ERR_INVALID
    names = ("q", "k", "v", "cu", "out", "lse", "do", "dq", "dk", "dv", "ws")
    back = lambda d=desc, wb=1 << 30, **o: lib.dr_window_attn_bwd(ctypes.byref(d), *[o.get(n, far(i)) for i, n in enumerate(names)], wb, None)
    for n in ("q", "k", "v", "out", "lse", "do", "dq", "dk", "dv"):
        assert back(**{n: None}) == dr.DR_ERR_INVALID, n
        assert back(**{n: at(n, 2)}) == dr.DR_ERR_INVALID, n
        assert back(ws=at(n)) == dr.DR_ERR_INVALID, n
    for n in ("q", "k", "v", "out", "lse", "do", "dq"):
        assert back(dk=at(n)) == dr.DR_ERR_INVALID, n
    assert back(ws=None) == dr.DR_ERR_WORKSPACE and back(wb=100) == dr.DR_ERR_WORKSPACE
    assert back(packed, dv=at("cu")) == dr.DR_ERR_INVALID


@no_gpu_only
def test_step_pointers_and_overlaps(dr):
    lib = dr.lib()
    names = ("q", "kc", "vc", "pages", "lens", "out", "lse", "ws")
    desc = step_desc(dr)
    at = lambda n, off=0: ctypes.c_void_p(((names.index(n) + 1) << 32) + off)
    call = lambda wb=1 << 30, **o: lib.dr_window_attn_step(ctypes.byref(desc), *[o.get(n, far(i)) for i, n in enumerate(names)], wb, None)
    assert lib.dr_window_attn_step(None, *[far(i) for i in range(8)], 1 << 30, None) == dr.DR_ERR_INVALID
    for n in ("q", "kc", "vc", "pages", "lens", "out"):
        assert call(**{n: None}) == dr.DR_ERR_INVALID and call(**{n: at(n, 2)}) == dr.DR_ERR_INVALID, n
    for n in ("q", "kc", "vc", "pages", "lens"):
        for w in ("out", "lse", "ws"):
            assert call(**{w: at(n)}) == dr.DR_ERR_INVALID, (n, w)
    assert call(ws=None) == dr.DR_ERR_WORKSPACE and call(wb=64) == dr.DR_ERR_WORKSPACE


def test_host_tensors_and_shapes_are_refused(dr):
    x = torch.zeros(1, 4, 2, 64)
    with pytest.raises((ValueError, RuntimeError)):
        dr.window_attn_fwd(x, x, x)
    if not torch.cuda.is_available():
        return
    c = x.cuda()
    l = torch.zeros(1, 4, 2, device="cuda")
    for bad in (lambda: dr.window_attn_fwd(c, c[:, :3], c), lambda: dr.window_attn_fwd(c, c.half(), c), lambda: dr.window_attn_fwd(c, x, c),
                lambda: dr.window_attn_fwd(c, c, c, window=-1), lambda: dr.window_attn_fwd(c, c.expand(1, 4, 2, 64)[:, :1].expand(1, 4, 2, 64), c),
                lambda: dr.window_attn_fwd(c, c, c, out=c.bfloat16()), lambda: dr.window_attn_fwd(c, c, c, lse=l.double()),
                lambda: dr.window_attn_bwd(c, c, c, c, l[:, :3], c), lambda: dr.window_attn_bwd(c, c, c, c.clone(), l, c, grads=(c, c)),
                lambda: dr.window_attn_fwd(c, c, c, cu_seqlens=torch.zeros(2, dtype=torch.int32, device="cuda")),
                lambda: dr.window_attn_fwd(c.transpose(1, 2), c.transpose(1, 2), c.transpose(1, 2))):
        with pytest.raises(ValueError):
            bad()
    q, cache = torch.zeros(3, 2, 64, device="cuda"), torch.zeros(4, 2, 16, 64, device="cuda")
    pages, lens = torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int64, device="cuda")
    t = dr.rope_table(64)
    for bad in (lambda: dr.window_attn_step(q, cache, cache[:3], pages, lens), lambda: dr.window_attn_step(q, cache, cache, pages.long(), lens),
                lambda: dr.window_attn_step(q, cache, cache, pages, lens.int()), lambda: dr.window_attn_step(q, cache.bfloat16(), cache, pages, lens),
                lambda: dr.window_attn_step(q, cache, cache, pages[:2], lens), lambda: dr.window_attn_step(q, cache, cache, pages.cpu(), lens),
                lambda: dr.kv_append(q, q, q, t, cache[:, :1].contiguous(), cache[:, :1].contiguous(), pages, lens),
                lambda: dr.kv_append(q, q, q[:2], t, cache, cache.clone(), pages, lens),
                lambda: dr.kv_append(None, q, q, t, cache, cache.clone(), pages, lens, q_out=q),
                lambda: dr.kv_append(q, q, q, t, cache, cache.clone(), pages, lens, norm="no"),
                lambda: dr.kv_append(q, q, q, t, cache, cache.clone(), pages, lens[:2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(dr.DrError):
        dr.window_attn_fwd(torch.zeros(1, 4, 3, 64, device="cuda"), c, c)
