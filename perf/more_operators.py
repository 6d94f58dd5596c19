"""Attention over a sliding window with first tokens that stay visible, its paged cache and its
single-token form: what is measured of them.

Operators (by the case's "op"):
  fwd      o_i = sum_j softmax_j(scale q_i.k_j) v_j over the visible keys of a token i of its
           sequence: j <= i, and i - j < window (window 0: no limit) or j < sinks; and the log
           of the softmax's sum
  bwd      the gradients of fwd's outputs, from its outputs
  step     one token for each sequence over a paged cache of keys and values
  append   keys (normalised and rotated by their positions) and values written into such a
           cache, the queries of the same tokens normalised and rotated on the way

`run` computes them in elementary torch operations where `own` is false, and through
gated_delta_rule_15_gb300.dr where it is true.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def _attn(op, B, T, Hq, Hk, d, window, sinks, dtype="bf16", packed=0, fused=False):
    return dict(op=op, B=B, T=T, Hq=Hq, Hk=Hk, d=d, window=window, sinks=sinks, dtype=dtype, packed=packed, fused=fused)


def _step(B, Hq, Hk, d, window, sinks, longest, page, dtype="bf16"):
    return dict(op="step", B=B, Hq=Hq, Hk=Hk, d=d, window=window, sinks=sinks, longest=longest, page=page, dtype=dtype)


def _append(B, T, Hq, Hk, d, rot, page, dtype="bf16", norm="rms", layout="half", fused=False):
    return dict(op="append", B=B, T=T, Hq=Hq, Hk=Hk, d=d, rot=rot, page=page, dtype=dtype, norm=norm, layout=layout,
                fused=fused)


def listed():
    return [
        # training forward of a whole batch (this repository's benchmark shape), rows of a fused projection
        dict(_attn("fwd", 8, 4096, 16, 4, 128, 1024, 4, fused=True), name="fwd_B8_T4096_H16_4_d128_w1024_s4"),
        # prefill of one long context
        dict(_attn("fwd", 1, 65536, 16, 4, 128, 4096, 4), name="fwd_B1_T65536_H16_4_d128_w4096_s4"),
        # prefill of ragged prompts packed behind one another, some of them empty or one token long
        dict(_attn("fwd", 1, 20011, 8, 2, 64, 512, 0, packed=23), name="fwd_packed23_T20011_H8_2_d64_w512"),
        # a layer that sees everything before it, a key head for each query head
        dict(_attn("fwd", 2, 8192, 16, 16, 128, 0, 0), name="fwd_B2_T8192_H16_d128_all"),
        # the small single-precision problem of a numerics check, latency
        dict(_attn("fwd", 1, 256, 2, 1, 64, 64, 4, dtype="fp32"), name="fwd_B1_T256_H2_1_d64_w64_s4_fp32"),
        # training backward of a batch
        dict(_attn("bwd", 8, 2048, 16, 4, 128, 1024, 4), name="bwd_B8_T2048_H16_4_d128_w1024_s4"),
        # training backward of ragged packed documents
        dict(_attn("bwd", 1, 5003, 8, 8, 128, 256, 4, packed=11, fused=True), name="bwd_packed11_T5003_H8_d128_w256_s4"),
        # backward of odd single-precision rows
        dict(_attn("bwd", 1, 1037, 6, 3, 64, 200, 2, dtype="fp32"), name="bwd_B1_T1037_H6_3_d64_w200_s2_fp32"),
        # a full serving batch's token, contexts of all lengths
        dict(_step(256, 32, 8, 128, 4096, 4, 16384, 16), name="step_B256_H32_8_d128_w4096_s4"),
        # one user's token over a long context that stays visible: latency
        dict(_step(1, 16, 4, 128, 0, 0, 131072, 64), name="step_B1_H16_4_d128_all_131072"),
        # prompts into the cache, rows of a fused projection
        dict(_append(7, 32768, 16, 4, 128, 128, 16, fused=True), name="append_T32768_H16_4_d128"),
        # a decode batch's tokens into the cache: latency
        dict(_append(64, 64, 32, 8, 128, 64, 16, layout="interleaved"), name="append_B64_H32_8_d128"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "step", "append"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([64, 128, 128])
    Hk = rng.randint(1, 8)
    Hq = Hk * rng.choice([1, 2, 3, 4, 8])
    window = rng.choice([0, 1, 2, 2]) and _log_int(rng, 1, 4096)
    sinks = rng.choice([0, rng.randint(1, 8), _log_int(rng, 1, 200)])
    if op == "append":
        B = rng.randint(1, 64)
        T = rng.choice([B, _log_int(rng, B, 16384)])
        return _append(B, T, Hq, Hk, d, rng.choice([d, d, d // 2, d // 4]), 16 << rng.randint(0, 4), dtype,
                       rng.choice(["rms", "rms", "l2", "none"]), rng.choice(["half", "interleaved"]), rng.random() < 0.5)
    if op == "step":
        B = _log_int(rng, 1, 256)
        room = (1 << 28) // (Hk * d * B)           # tokens a sequence
        return _step(B, Hq, Hk, d, window, sinks, _log_int(rng, 1, min(131072, max(1, room))), 16 << rng.randint(0, 4), dtype)
    # lengths, windows and sequence ends fall anywhere: odd lengths, one token
    packed = rng.choice([0, 0, rng.randint(1, 32)])
    pairs = 1 << (30 if op == "fwd" else 29)       # (query, visible key) pairs of all heads
    if dtype == "fp32":
        pairs >>= 3
    least = 1
    if op == "bwd":      # (a softmax over one key has no gradient: nothing but rounding would be compared)
        window, least = window and max(2, window), 2
    T = _log_int(rng, least if packed == 0 else 64, 8192 if op == "fwd" else 4096)
    seen = min(T, window + sinks) if window else T
    while T > 3 and T * seen * Hq > pairs:
        T //= 2
        seen = min(T, seen)
    B = 1 if packed else max(1, min(8, _log_int(rng, 1, max(1, pairs // (T * seen * Hq)))))
    return _attn(op, B, T, Hq, Hk, d, window, sinks, dtype, packed, rng.random() < 0.4)


# ------------------------------------------------------------------ inputs
def _lengths(n, total):
    """`n` sequence lengths whose sum is at most `total` (some rows may lie behind the last
    one): ragged over a factor of a hundred, one of them empty and one a single token."""
    g = torch.Generator().manual_seed(n)
    w = torch.exp(4.6 * torch.rand(n, generator=g, dtype=torch.float64))
    keep = total - (total // 50 if n > 2 else 0)
    ls = torch.floor(w / w.sum() * keep).to(torch.int64)
    if n > 4:
        ls[n // 3], ls[n // 2] = 0, 1
    return [int(x) for x in ls]


def _contexts(case):
    """Tokens of each sequence, the new one among them: the longest, and down to a thousandth
    of it; a slot of a larger batch without a sequence."""
    n, top = case["B"], case["longest"]
    ls = [max(1, int(top * 1000.0 ** (-i / max(1, n - 1)))) for i in range(n)]
    if n > 4:
        ls[n // 3] = 0
    return ls


def _page_table(counts, keep, page, g):
    """A table of pages in any order for sequences of `counts` tokens; pages none of whose tokens
    `keep(i, first, end)` needs are -1.  Also the number of pages."""
    most = max(1, max(-(-c // page) for c in counts))
    need = [[keep(i, p * page, min(c, (p + 1) * page)) if p * page < c else False for p in range(most)]
            for i, c in enumerate(counts)]
    need = torch.tensor(need)
    n = max(1, int(need.sum()))
    table = torch.full(need.shape, -1, dtype=torch.int32)
    table[need] = torch.randperm(n, generator=g)[:int(need.sum())].to(torch.int32)
    return table, n


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    cg = torch.Generator().manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    st = dict(case=case)
    if case["op"] == "append":
        return _prepare_append(case, st, g, cg, randn, dt)
    # queries share a direction that the first tokens' keys point along, as trained layers' do
    lean = randn(Hk, 1, d)
    lean = lean / lean.norm(dim=-1, keepdim=True) * d ** 0.25
    if case["op"] == "step":
        B, page, w, sinks = case["B"], case["page"], case["window"], case["sinks"]
        ls = _contexts(case)
        table, n = _page_table(ls, lambda i, a, b: w == 0 or b > ls[i] - w or a < sinks, page, cg)
        st["pages"] = table.to(dev)
        st["lens"] = torch.tensor(ls, dtype=torch.int64, device=dev)
        st["q"] = (randn(B, Hk, Hq // Hk, d) + lean).reshape(B, Hq, d).to(dt)
        st["kc"] = torch.randn((n, Hk, page, d), generator=g, device=dev, dtype=dt)
        st["vc"] = torch.randn((n, Hk, page, d), generator=g, device=dev, dtype=dt)
        return st
    B, T = case["B"], case["T"]
    q = (randn(B, T, Hk, Hq // Hk, d) + lean).reshape(B, T, Hq, d)
    k, v = randn(B, T, Hk, d), randn(B, T, Hk, d)
    st["cu"] = None
    firsts = [0]
    if case["packed"]:
        ls = _lengths(case["packed"], T)
        st["longest"] = max(max(ls), 1)
        st["cu"] = torch.tensor([0] + ls, dtype=torch.int64).cumsum(0).to(dev)
        firsts = st["cu"][:-1]
    for s in range(min(case["sinks"], 4)):
        k[:, torch.as_tensor(firsts, device=dev).add(s).clamp(max=T - 1)] += 3.0 * lean[:, 0]
    if case["fused"]:          # q | k | v of one projection's output row
        qkv = torch.cat((q, k, v), 2).to(dt)
        q, k, v = qkv.split((Hq, Hk, Hk), 2)
    st["q"], st["k"], st["v"] = q.to(dt), k.to(dt), v.to(dt)
    if case["op"] == "bwd":    # the forward's results, which a training program keeps
        st["do"] = randn(B, T, Hq, d).to(dt)
        fw = _plain_fwd(st)
        st["out"], st["lse"] = fw["out"], fw["lse"]
    st["into"] = None
    if case["packed"]:         # the program's buffers: rows behind the last sequence are left as they are
        if case["op"] == "fwd":
            st["into"] = (torch.zeros((B, T, Hq, d), device=dev, dtype=dt), torch.zeros((B, T, Hq), device=dev))
        else:
            st["into"] = tuple(torch.zeros((B, T, h, d), device=dev, dtype=dt) for h in (Hq, Hk, Hk))
    return st


def _append_lengths(case):
    """Rows of each sequence in this call, and the tokens that its cache holds before it."""
    B, T = case["B"], case["T"]
    rows = [1] * B if T == B else _lengths(B, T)
    before = [(37 * i * i) % 300 for i in range(B)]
    if B > 4:
        before[B // 4] = -1        # a slot of the batch without a sequence
    return rows, before


def _prepare_append(case, st, g, cg, randn, dt):
    dev = "cuda"
    B, T, Hq, Hk, d, page = (case[n] for n in ("B", "T", "Hq", "Hk", "d", "page"))
    rows, before = _append_lengths(case)
    scale = 0.25 + 3.75 * torch.rand((T, 1, 1), generator=g, device=dev)
    qkv = (randn(T, Hq + 2 * Hk, d) * scale).to(dt)
    st["q"], st["k"], st["v"] = qkv.split((Hq, Hk, Hk), 1)
    if not case["fused"]:
        st["q"], st["k"], st["v"] = (st[n].contiguous() for n in "qkv")
    st["cu"] = None if T == B else torch.tensor([0] + rows, dtype=torch.int64).cumsum(0).to(dev)
    st["start"] = torch.tensor(before, dtype=torch.int64, device=dev)
    st["wq"] = st["wk"] = None
    if case["norm"] == "rms":
        st["wq"], st["wk"] = 1.0 + 0.2 * randn(d), 1.0 + 0.2 * randn(d)
    # pages whose tokens have left the window are given back: the first ones of every third sequence
    table, n = _page_table([r + max(b, 0) for r, b in zip(rows, before)],
                           lambda i, a, b: i % 3 != 0 or b > rows[i] // 2, page, cg)
    st["pages"] = table.to(dev)
    # one page more than the cache has, where the plain form writes rows that go nowhere
    st["store"] = [torch.randn((n + 1, Hk, page, d), generator=g, device=dev, dtype=dt) for _ in "kv"]
    st["kc"], st["vc"] = (x[:n] for x in st["store"])
    st["qo"] = torch.zeros((T, Hq, d), device=dev, dtype=dt)     # rows of no sequence are left as they are
    if own:
        from gated_delta_rule_15_gb300 import dr
        st["table"] = dr.rope_table(case["rot"], base=500000.0, device=dev)
    return st


# ------------------------------------------------------------------ plain forms
def _rows(x, cu, longest):
    """[1, T, ...] packed rows as [N, longest, ...]; rows of no sequence are zero."""
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


class _Blocks:
    """Blocks of C query tokens, each with the C + W key tokens that its window reaches and the
    first S ones."""

    def __init__(self, case, T, dev):
        self.T, w = T, case["window"]
        if w == 0 or w >= T:
            w, self.C, self.W, self.S = T, T, 0, 0
        else:
            self.C = 128
            self.C = min(max(128, 1 << ((w - 1) // 2).bit_length()), 1024)
            self.W = -(-(w - 1) // self.C) * self.C
            self.S = min(case["sinks"], T)
        self.n = -(-T // self.C)
        i = torch.arange(self.n * self.C, device=dev).view(self.n, self.C, 1)
        self.at = torch.arange(self.n, device=dev)[:, None] * self.C - self.W + torch.arange(self.C + self.W, device=dev)[None]
        j = self.at[:, None]
        near = (j >= 0) & (j <= i) & (i - j < w)
        first = torch.arange(self.S, device=dev)[None, None]
        self.seen = torch.cat((near, (i - first >= w)), -1)           # [blocks, C, W + C + S]
        self.at = self.at.clamp(0, T - 1)

    def queries(self, x, Hk):
        """[N, T, H, e] as [N, Hk, blocks, heads of the group * C, e] in 32 bits."""
        N, T, H, e = x.shape
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, self.n * self.C - T))
        return x.view(N, self.n, self.C, Hk, H // Hk, e).permute(0, 3, 1, 4, 2, 5).flatten(3, 4)

    def back(self, y, H):
        """The inverse of queries."""
        N, Hk, n, _, e = y.shape
        y = y.view(N, Hk, n, H // Hk, self.C, e).permute(0, 2, 4, 1, 3, 5)
        return y.reshape(N, n * self.C, H, e)[:, :self.T]

    def keys(self, x):
        """[N, T, Hk, e] as [N, Hk, blocks, W + C + S, e] in 32 bits."""
        x = x.float()
        near = x[:, self.at]                                           # [N, blocks, W + C, Hk, e]
        first = x[:, None, :self.S].expand(-1, self.n, -1, -1, -1)
        return torch.cat((near, first), 2).permute(0, 3, 1, 2, 4)

    def gather(self, y):
        """The transpose of keys."""
        y = y.permute(0, 2, 3, 1, 4)                                   # [N, blocks, W + C + S, Hk, e]
        N, Hk, e = y.shape[0], y.shape[3], y.shape[4]
        out = y.new_zeros((N, self.T, Hk, e))
        out.index_add_(1, self.at.reshape(-1), y[:, :, :self.W + self.C].reshape(N, -1, Hk, e))
        out[:, :self.S] += y[:, :, self.W + self.C:].sum(1)
        return out

    def scores(self, q, k, scale):
        s = (q @ k.transpose(-1, -2)) * scale
        N, Hk, n, m, c = s.shape
        return s.view(N, Hk, n, m // self.C, self.C, c).masked_fill_(~self.seen[:, None], -math.inf).view(s.shape)


def _plain_inputs(st, names):
    xs = [st[n] for n in names]
    return xs if st["cu"] is None else [_rows(x, st["cu"], st["longest"]) for x in xs]


def _plain_fwd(st):
    case = st["case"]
    q, k, v = _plain_inputs(st, ("q", "k", "v"))
    b = _Blocks(case, q.shape[1], q.device)
    s = b.scores(b.queries(q, case["Hk"]), b.keys(k), case["d"] ** -0.5)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = b.back((p @ b.keys(v)) / total, case["Hq"])
    lse = b.back(top + total.log(), case["Hq"])[..., 0]
    if st["cu"] is not None:
        out, lse = (_packed(x, st["cu"], st["q"].shape[1]) for x in (out, lse))
    return dict(out=out.to(st["q"].dtype), lse=lse)


def _plain_bwd(st):
    case = st["case"]
    Hq, Hk, scale = case["Hq"], case["Hk"], case["d"] ** -0.5
    q, k, v, out, do = _plain_inputs(st, ("q", "k", "v", "out", "do"))
    lse = _plain_inputs(st, ("lse",))[0][..., None]
    b = _Blocks(case, q.shape[1], q.device)
    delta = b.queries((do.float() * out.float()).sum(-1, keepdim=True), Hk)
    q, do, lse = (b.queries(x, Hk) for x in (q, do, lse))
    kb = b.keys(k)
    p = b.scores(q, kb, scale).sub_(lse).exp_()
    dv = b.gather(p.transpose(-1, -2) @ do)
    ds = p.mul_((do @ b.keys(v).transpose(-1, -2)).sub_(delta)).mul_(scale)
    dq = b.back(ds @ kb, Hq)
    dk = b.gather(ds.transpose(-1, -2) @ q)
    if st["cu"] is not None:
        dq, dk, dv = (_packed(x, st["cu"], st["q"].shape[1]) for x in (dq, dk, dv))
    dt = st["q"].dtype
    return dict(dq=dq.to(dt), dk=dk.to(dt), dv=dv.to(dt))


def _plain_step(st):
    case = st["case"]
    Hq, Hk, d, page, w = (case[n] for n in ("Hq", "Hk", "d", "page", "window"))
    q, pages, lens = st["q"], st["pages"], st["lens"][:, None]
    B, room = pages.shape[0], pages.shape[1] * page
    i = torch.arange(min(room, w + case["sinks"]) if w else room, device=q.device)[None]
    if w:                # the window's tokens, then the first ones
        j = torch.where(i < w, lens - w + i, i - w)
        seen = (j >= 0) & (j < lens) & ((i < w) | (j < lens - w))
        if room <= w + case["sinks"]:
            j, seen = i.expand(B, -1), (i < lens) & ((i >= lens - w) | (i < case["sinks"]))
    else:
        j, seen = i.expand(B, -1), i < lens
    j = j.clamp(0, room - 1)
    pg = pages.gather(1, j // page).long()
    seen = seen & (pg >= 0)
    pg = pg.clamp(min=0)
    k, v = (c[pg, :, j % page].float().transpose(1, 2) for c in (st["kc"], st["vc"]))      # [B, Hk, M, d]
    s = (q.float().view(B, Hk, Hq // Hk, d) @ k.transpose(-1, -2)) * d ** -0.5
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (s - top).exp()
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / total.clamp(min=1e-30)      # no key: zeros
    return dict(out=out.view(B, Hq, d).to(q.dtype), lse=(top + total.log()).view(B, Hq))


def _row_positions(st, T):
    """Each row's sequence and position; rows of none are at -1."""
    dev = st["start"].device
    t = torch.arange(T, device=dev)
    if st["cu"] is None:
        return t, st["start"]
    n = torch.bucketize(t, st["cu"][1:], right=True)
    there = n < st["start"].numel()
    n = n.clamp(max=st["start"].numel() - 1)
    at = st["start"][n]
    return n, torch.where(there & (at >= 0), at + t - st["cu"][n], -1)


def _plain_append(st):
    case = st["case"]
    T, d, page, rot, layout = (case[n] for n in ("T", "d", "page", "rot", "layout"))
    n, pos = _row_positions(st, T)
    f = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=pos.device) / rot)
    a = pos.double()[:, None] * f
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    got = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        x = x.float()
        if case["norm"] != "none":
            ss = x.square().sum(-1, keepdim=True)
            x = x * ((ss / d if case["norm"] == "rms" else ss) + EPS).rsqrt()
        if w is not None:
            x = x * w
        one, two = x[..., :rot].chunk(2, -1) if layout == "half" else (x[..., :rot:2], x[..., 1:rot:2])
        turned = (one * cos - two * sin, two * cos + one * sin)
        turned = torch.cat(turned, -1) if layout == "half" else torch.stack(turned, -1).flatten(-2)
        got.append(torch.cat((turned, x[..., rot:]), -1).to(st["q"].dtype))
    live = pos >= 0
    st["qo"].copy_(torch.where(live[:, None, None], got[0], st["qo"]))
    at = pos.clamp(min=0)
    pg = st["pages"][n, at // page].long()
    pg = torch.where(live & (pg >= 0), pg, st["store"][0].shape[0] - 1)
    st["store"][0][pg, :, at % page] = got[1]
    st["store"][1][pg, :, at % page] = st["v"]
    return dict(q=st["qo"], kc=st["kc"], vc=st["vc"])


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "append": _plain_append}[op](state)
    from gated_delta_rule_15_gb300 import dr
    st = state
    if op == "append":
        q = dr.kv_append(st["q"], st["k"], st["v"], st["table"], st["kc"], st["vc"], st["pages"], st["start"],
                         cu_seqlens=st["cu"], norm=case["norm"], wq=st["wq"], wk=st["wk"], eps=EPS,
                         layout=case["layout"], q_out=st["qo"])
        return dict(q=q, kc=st["kc"], vc=st["vc"])
    seen = dict(window=case["window"], sinks=case["sinks"])
    if op == "step":
        out, lse = dr.window_attn_step(st["q"], st["kc"], st["vc"], st["pages"], st["lens"], return_lse=True, **seen)
        return dict(out=out, lse=lse)
    if op == "fwd":
        into = {} if st["into"] is None else dict(out=st["into"][0], lse=st["into"][1])
        out, lse = dr.window_attn_fwd(st["q"], st["k"], st["v"], cu_seqlens=st["cu"], **seen, **into)
        return dict(out=out, lse=lse)
    dq, dk, dv = dr.window_attn_bwd(st["q"], st["k"], st["v"], st["out"], st["lse"], st["do"], cu_seqlens=st["cu"],
                                    grads=st["into"], **seen)
    return dict(dq=dq, dk=dk, dv=dv)


def _pairs(length, window, sinks):
    """(query, visible key) pairs of a sequence."""
    if window == 0 or window >= length:
        return length * (length + 1) // 2
    near = window * (window + 1) // 2 + (length - window) * window
    far = length - window                     # queries with keys in front of their window: 1, 2, .. of them
    m = min(sinks, far)
    return near + m * (m + 1) // 2 + (far - m) * m


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    if case["op"] == "append":
        rows, before = _append_lengths(case)
        T = sum(r for r, b in zip(rows, before) if b >= 0)
        return {"bytes": 2 * T * (Hq + 2 * Hk) * d * e + 8 * case["B"], "flops": 8 * T * (Hq + Hk) * d}
    if case["op"] == "step":
        w = case["window"]
        seen = sum(min(n, w + min(case["sinks"], max(0, n - w))) if w else n for n in _contexts(case))
        return {"bytes": seen * 2 * Hk * d * e + case["B"] * Hq * (2 * d * e + 4) + 4 * seen // case["page"],
                "flops": 4 * seen * Hq * d}
    B, T = case["B"], case["T"]
    ls = _lengths(case["packed"], T) if case["packed"] else [T] * B
    pairs, rows = sum(_pairs(n, case["window"], case["sinks"]) for n in ls) * Hq, sum(ls)
    if case["op"] == "fwd":
        return {"bytes": rows * (2 * (Hq + Hk) * d * e + 4 * Hq), "flops": 4 * pairs * d}
    return {"bytes": rows * (4 * (Hq + Hk) * d * e + 4 * Hq), "flops": 10 * pairs * d}


# ------------------------------------------------------------------ the definition in 64 bits
def _visible(case, i, j):
    """Whether the token at position i sees the one at j."""
    near = (i - j < case["window"]) if case["window"] else torch.ones_like(i - j, dtype=torch.bool)
    return (j <= i) & (near | (j < case["sinks"]))


def _softmax_rows(case, q, k, v, first, js):
    """Queries [m, g, d] at positions first, first + 1, .. against keys [c, d] at positions js."""
    i = first + torch.arange(q.shape[0], device=q.device)
    s = torch.einsum("mgd,cd->mgc", q, k) / math.sqrt(case["d"])
    s = s.masked_fill(~_visible(case, i[:, None], js[None])[:, None], -math.inf)
    lse = torch.logsumexp(s, -1)
    return torch.einsum("mgc,cd->mgd", (s - lse[..., None]).exp(), v), lse


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st, case)
    if case["op"] == "step":
        return _exact_step(st, case)
    q, k, v = (st[n].double() for n in "qkv")
    Hk, g = case["Hk"], case["Hq"] // case["Hk"]
    if st["cu"] is None:
        spans = [(b, 0, case["T"]) for b in range(case["B"])]
    else:
        cu = st["cu"].tolist()
        spans = [(0, a, e) for a, e in zip(cu, cu[1:])]
    if case["op"] == "bwd":
        grads = [torch.zeros_like(x) for x in (q, k, v)]
    else:
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], dtype=torch.float64, device=q.device)
    for b, lo, hi in spans:
        for h in range(Hk):
            hs = slice(h * g, (h + 1) * g)
            if case["op"] == "bwd":
                xs = [x[b, lo:hi, s].clone().requires_grad_() for x, s in ((q, hs), (k, h), (v, h))]
                if hi > lo:
                    o, _ = _softmax_rows(case, *xs, 0, torch.arange(hi - lo, device=q.device))
                    for dst, s, gr in zip(grads, (hs, h, h), torch.autograd.grad(o, xs, st["do"][b, lo:hi, hs].double())):
                        dst[b, lo:hi, s] = gr
                continue
            for a in range(0, hi - lo, 512):
                e = min(a + 512, hi - lo)
                at = torch.arange(max(0, a - case["window"] + 1) if case["window"] else 0, e, device=q.device)
                early = torch.arange(min(case["sinks"], int(at[0])), device=q.device)
                js = torch.cat((early, at))
                out[b, lo + a:lo + e, hs], lse[b, lo + a:lo + e, hs] = _softmax_rows(
                    case, q[b, lo + a:lo + e, hs], k[b, lo + js, h], v[b, lo + js, h], a, js)
    if case["op"] == "bwd":
        return dict(dq=grads[0], dk=grads[1], dv=grads[2])
    return dict(out=out, lse=lse)


def _exact_step(st, case):
    Hk, g, page = case["Hk"], case["Hq"] // case["Hk"], case["page"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lens"].tolist()):
        if n == 0:
            continue
        js = torch.arange(n, device="cuda")
        js = js[_visible(case, torch.tensor(n - 1, device="cuda"), js)]
        pg = st["pages"][b].long()[js // page]
        for h in range(Hk):
            o, x = _softmax_rows(case, st["q"][b:b + 1, h * g:(h + 1) * g].double(), st["kc"][pg, h, js % page].double(),
                                 st["vc"][pg, h, js % page].double(), n - 1, js)
            out[b, h * g:(h + 1) * g], lse[b, h * g:(h + 1) * g] = o[0], x[0]
    return dict(out=out, lse=lse)


def _exact_append(st, case):
    T, d, page, rot = (case[n] for n in ("T", "d", "page", "rot"))
    rows, before = _append_lengths(case)
    seq, pos = [], []
    for n, (r, b) in enumerate(zip(rows, before)):
        seq += [n] * r
        pos += [b + t if b >= 0 else -1 for t in range(r)]
    live = [t for t in range(len(pos)) if pos[t] >= 0]
    at = torch.tensor([pos[t] for t in live], device="cuda")
    sq = torch.tensor([seq[t] for t in live], device="cuda")
    t = torch.tensor(live, device="cuda")
    freq = torch.tensor([math.pow(500000.0, -2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device="cuda")
    ang = torch.outer(at.double(), freq)
    turn = torch.complex(ang.cos(), ang.sin())[:, None]
    i = torch.arange(rot // 2, device="cuda")
    one, two = (i, i + rot // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
    made = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        x = x[t].double()
        if case["norm"] != "none":
            x = x / ((x * x).sum(-1, keepdim=True) / (d if case["norm"] == "rms" else 1) + EPS).sqrt()
        if w is not None:
            x = x * w.double()
        c = torch.complex(x[..., one], x[..., two]) * turn
        x = x.clone()
        x[..., one], x[..., two] = c.real, c.imag
        made.append(x)
    q, kc, vc = (st[n].double() for n in ("qo", "kc", "vc"))
    q[t] = made[0]
    pg = st["pages"][sq, at // page].long()
    kept = pg >= 0
    kc[pg[kept], :, (at % page)[kept]] = made[1][kept]
    vc[pg[kept], :, (at % page)[kept]] = st["v"][t].double()[kept]
    return dict(q=q, kc=kc, vc=vc)
