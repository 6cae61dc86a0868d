"""Cases of the linear attention with a decay for each head (chunked form,
its gradients, the single-token form) and of the gated norm that follows an
attention block, with their plain forms.

A case is a dict of plain values; ``op`` says which call it makes:
  la_fwd     the forward pass over prompts
  la_train   forward and backward pass
  la_decode  one token for each of ``N`` sequences, the state updated
  norm_fwd   the gated norm
  norm_train its forward and backward pass
Packed batches (``seqs`` > 0) hold ``seqs`` sequences of ``lo`` to ``hi``
tokens (drawn from ``lens``, so that sizes are the case's own) and ``tail``
rows behind the last one.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
CHUNK = 64


# ------------------------------------------------------------------ cases
def _la(op, **kw):
    c = dict(op=op, B=1, T=0, H=1, K=128, V=128, seqs=0, lo=0, hi=0, lens=0, tail=0, init=False)
    c.update(kw)
    return c


def listed():
    return [
        # one short prompt of a small model: the call's latency
        dict(_la("la_fwd", B=1, T=256, H=4, K=64, V=64), name="prompt short"),
        # an ordinary batch of two prompts that continue earlier ones
        dict(_la("la_fwd", B=2, T=2048, H=32, init=True), name="prompts 2x2048"),
        # a serving batch of unequal prompts without padding
        dict(_la("la_fwd", H=32, seqs=16, lo=256, hi=8192, lens=2), name="prompts packed"),
        # one very long document: few heads, a long chain
        dict(_la("la_fwd", B=1, T=131072, H=16, init=True), name="prompt 131072"),
        # training on odd sizes: heads and tokens that fill no tile
        dict(_la("la_train", B=3, T=777, H=5, K=64, V=128, init=True), name="train odd"),
        # a training step's share of one attention layer
        dict(_la("la_train", B=2, T=2048, H=32, init=True), name="train 2x2048"),
        # training on packed documents, one-token ones among them, with padding behind them
        dict(_la("la_train", H=16, K=128, V=64, seqs=24, lo=1, hi=2048, lens=7, tail=37),
             name="train packed"),
        # one user's next token
        dict(op="la_decode", N=1, H=16, K=128, V=128, name="token 1 sequence"),
        # a serving batch's next tokens
        dict(op="la_decode", N=64, H=32, K=128, V=128, name="token 64 sequences"),
        # the norm behind a decode step: the call's latency
        dict(op="norm_fwd", rows=64, H=32, D=128, act="silu", res=True, name="norm tokens"),
        # the norm of a training step, sigmoid gate
        dict(op="norm_train", rows=4096, H=32, D=128, act="sigmoid", res=False,
             name="norm train"),
        # with the block's skip, at a head size and counts that fill no tile
        dict(op="norm_train", rows=3001, H=5, D=72, act="silu", res=True, name="norm train odd"),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["la_fwd", "la_train", "la_decode", "norm_fwd", "norm_train"])
    if op == "la_decode":
        return dict(op=op, N=_spread(rng, 1, 192), H=_spread(rng, 1, 48),
                    K=rng.choice([64, 128]), V=rng.choice([64, 128]))
    if op.startswith("norm"):
        H = _spread(rng, 1, 64)
        D = 8 * _spread(rng, 1, 64)
        return dict(op=op, rows=_spread(rng, 1, max(1, min(16384, 2 ** 25 // (H * D)))), H=H, D=D,
                    act=rng.choice(["sigmoid", "silu"]), res=rng.random() < 0.5)
    H = _spread(rng, 1, 32)
    most = (1 << 20 if op == "la_fwd" else 1 << 18) // H  # tokens
    c = dict(H=H, K=rng.choice([64, 128]), V=rng.choice([64, 128]), init=rng.random() < 0.5)
    if rng.random() < 0.5:
        n = _spread(rng, 1, 48)
        hi = _spread(rng, 1, max(1, min(8192, most // n)))
        c.update(seqs=n, lo=rng.randint(0, hi), hi=hi, lens=rng.randint(1, 10 ** 6),
                 tail=rng.choice([0, 0, rng.randint(1, 100)]))
        if c["lo"] == 0 and hi < 64:
            c["lo"] = 1
    else:
        T = _spread(rng, 1, min(32768, most))
        c.update(B=_spread(rng, 1, max(1, min(32, most // T))), T=T)
    return _la(op, **c)


def _lengths(c):
    """Tokens of each sequence."""
    if not c["seqs"]:
        return [c["T"]] * c["B"]
    r = random.Random(c["lens"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]


def _rows(c):
    """[B, T] of the token tensors."""
    return (1, sum(_lengths(c)) + c["tail"]) if c["seqs"] else (c["B"], c["T"])


def work(case):
    c = case
    if c["op"] == "la_decode":
        pairs = c["N"] * c["H"]
        return {"bytes": pairs * (8 * c["K"] * c["V"] + 4 * c["K"] + 4 * c["V"]),
                "flops": 4 * pairs * c["K"] * c["V"]}
    if c["op"].startswith("norm"):
        e = c["rows"] * c["H"] * c["D"]
        fwd = 3 + c["res"]
        if c["op"] == "norm_fwd":
            return {"bytes": 2 * e * fwd, "flops": 10 * e}
        return {"bytes": 2 * e * (fwd + (3 + c["res"]) + (2 + c["res"])), "flops": 30 * e}
    n = len(_lengths(c))
    th = sum(_lengths(c)) * c["H"]
    K, V = c["K"], c["V"]
    state = n * c["H"] * K * V * 4
    by = th * (4 * K + 4 * V) + state * (1 + c["init"])
    fl = 4 * th * K * V
    if c["op"] == "la_train":  # q, k, v, do read; dq, dk, dv written; both state gradients
        by += th * (8 * K + 6 * V) + state * (2 + c["init"])
        fl += 10 * th * K * V
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)

    def feature(*shape):
        # queries and keys come out of an activation that is positive for the most part
        return torch.nn.functional.silu(torch.randn(*shape, generator=g, device=DEV)).to(
            torch.bfloat16)

    s = dict(case=c)
    if c["op"].startswith("norm"):
        R, H, D = c["rows"], c["H"], c["D"]
        s["x"] = normal(R, H, D)
        s["gate"] = normal(R, H, D)
        s["weight"] = 1.0 + normal(D, dtype=torch.float32, std=0.1)
        s["residual"] = normal(R, H, D) if c["res"] else None
        s["residual_scale"] = normal(H, dtype=torch.float32) if c["res"] else None
        if c["op"] == "norm_train":
            s["dy"] = normal(R, H, D)
        return s
    H, K, V = c["H"], c["K"], c["V"]
    # from a head that forgets within a few tokens to one that remembers hundreds
    s["log_decay"] = -torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV,
                                                     dtype=torch.float32) / H)
    if c["op"] == "la_decode":
        N = c["N"]
        s["q"], s["k"], s["v"] = feature(N, H, K), feature(N, H, K), normal(N, H, V)
        s["state"] = normal(N, H, K, V, dtype=torch.float32)
        s["new_state"] = torch.empty_like(s["state"])
        return s
    B, T = _rows(c)
    lens = _lengths(c)
    s["q"], s["k"], s["v"] = feature(B, T, H, K), feature(B, T, H, K), normal(B, T, H, V)
    s["h0"] = normal(len(lens), H, K, V, dtype=torch.float32) if c["init"] else None
    s["cu"] = None
    if c["seqs"]:
        at = [0]
        for n in lens:
            at.append(at[-1] + n)
        s["cu"] = torch.tensor(at, dtype=torch.int32, device=DEV)
    if c["op"] == "la_train":
        s["do"] = normal(B, T, H, V)
        s["dfinal"] = normal(len(lens), H, K, V, dtype=torch.float32)
    return s


# ------------------------------------------------------------------ the calls
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    if op == "la_decode":
        return _plain_decode(state)
    if op.startswith("norm"):
        return _plain_norm(state, op == "norm_train")
    return _plain_la(state, op == "la_train")


def _own(op, s):
    import chunked_gated_delta_kda_amd as kda

    c = s["case"]
    if op == "la_decode":
        o, new = kda.la_decode(s["q"], s["k"], s["v"], s["log_decay"], state=s["state"],
                               state_out=s["new_state"])
        return dict(o=o, state=new)
    if op.startswith("norm"):
        kw = dict(activation=c["act"], eps=EPS, residual=s["residual"],
                  residual_scale=s["residual_scale"])
        y = kda.gated_norm_fwd(s["x"], s["gate"], s["weight"], **kw)
        if op == "norm_fwd":
            return dict(y=y)
        r = kda.gated_norm_bwd(s["x"], s["gate"], s["weight"], s["dy"], **kw)
        out = dict(y=y, dx=r["dx"], dgate=r["dgate"], dweight=r["dweight"])
        if c["res"]:
            out.update(dresidual=r["dresidual"], dresidual_scale=r["dresidual_scale"])
        return out
    o, final = kda.la_fwd(s["q"], s["k"], s["v"], s["log_decay"], initial_state=s["h0"],
                          cu_seqlens=s["cu"])
    if op == "la_fwd":
        return dict(o=o, final_state=final)
    r = kda.la_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"], initial_state=s["h0"],
                   dfinal=s["dfinal"], cu_seqlens=s["cu"], need_dh0=c["init"])
    out = dict(o=o, final_state=final, dq=r["dq"], dk=r["dk"], dv=r["dv"])
    if c["init"]:
        out["dh0"] = r["dh0"]
    return out


# ------------------------------------------------------------------ plain forms
def _rows_of(s):
    """Token row of every position of every sequence, aligned at the end of a
    [N, Tp] table (Tp a multiple of CHUNK), and which places are no token."""
    c = s["case"]
    lens = torch.tensor(_lengths(c), device=DEV)
    Tp = -(-max(1, max(_lengths(c))) // CHUNK) * CHUNK
    first = torch.cumsum(lens, 0) - lens
    pos = torch.arange(Tp, device=DEV)[None] - (Tp - lens)[:, None]
    return first[:, None] + pos, pos, lens


def _chunked(x, y, z, ld, late, x_scale, in_scale, z_scale, state, pos, lens):
    """One pass over [N, Tp, H, *] 32-bit rows aligned at their end: outputs
    sum_{j<=i} a^(i-j) (x_i y_j) z_j (times in_scale) and the state's part, and
    the state behind the last token.  late = 1: a token decays its own state too."""
    N, Tp, H, D1 = x.shape
    D2 = z.shape[-1]
    nc = Tp // CHUNK

    def split(t):
        return t.view(N, nc, CHUNK, H, -1).permute(0, 3, 1, 2, 4).contiguous()

    xc, yc, zc = split(x), split(y), split(z)
    i = torch.arange(CHUNK, device=DEV, dtype=torch.float64)
    l64 = ld.double()
    gap = i[:, None] - i[None, :]
    dec = torch.where(gap >= 0, torch.exp(l64[:, None, None] * gap.clamp(min=0)), 0.0).float()
    p = torch.matmul(xc, yc.transpose(-1, -2)) * (dec[None, :, None] * in_scale)
    out = torch.matmul(p, zc)
    # what each chunk adds to the state, and the states entering the chunks
    w = torch.exp(l64[:, None] * (CHUNK - 1 - i + late)).float()
    add = torch.matmul((yc * (w[None, :, None, :, None] * z_scale)).transpose(-1, -2), zc)
    a = torch.exp(l64 * CHUNK)[None, :, None, None]
    S = torch.zeros(N, H, D1, D2, device=DEV, dtype=torch.float64)
    enter = torch.empty(N, H, nc, D1, D2, device=DEV)
    for n in range(nc):  # a recurrence: each chunk's state needs the one before
        enter[:, :, n] = S
        S = S * a + add[:, :, n]
    up = torch.exp(l64[:, None] * (i + 1 - late)).float()
    out += torch.matmul(xc, enter) * (up[None, :, None, :, None] * x_scale)
    out = out.permute(0, 2, 3, 1, 4).reshape(N, Tp, H, D2)
    if state is not None:
        far = torch.exp(l64 * (pos.clamp(min=0) + 1 - late)[..., None]).float() * x_scale
        out = out + torch.matmul(x.permute(0, 2, 1, 3), state).permute(0, 2, 1, 3) * far[..., None]
        S = S + state * torch.exp(l64 * lens[:, None])[..., None, None]
    return out, S.float()


def _plain_la(s, train):
    c = s["case"]
    row, pos, lens = _rows_of(s)
    there = pos >= 0
    B, T = _rows(c)
    ld, h0, scale = s["log_decay"], s["h0"], c["K"] ** -0.5

    def rows(t, at):  # 32-bit rows in sequence order, zeros where no token is
        flat = t.reshape(B * T, c["H"], -1)
        got = flat[at.clamp(0, max(0, B * T - 1))].float() if B * T else flat.new_zeros(
            *at.shape, *flat.shape[1:]).float()
        return torch.where(there[..., None, None], got, 0.0)

    def back(t, at, like):  # to the tokens' own rows, rounded once
        out = torch.zeros_like(like).reshape(B * T, c["H"], -1)
        out[at[there]] = t[there].to(out.dtype)
        return out.view(like.shape)

    q, k, v = (rows(s[n], row) for n in "qkv")
    o, final = _chunked(q, k, v, ld, 0, scale, scale, 1.0, h0, pos, lens)
    out = dict(o=back(o, row, s["v"]), final_state=final)
    if not train:
        return out
    do = rows(s["do"], row)
    h0t = None if h0 is None else h0.transpose(-1, -2).contiguous()
    dq, _ = _chunked(do, v, k, ld, 0, scale, scale, 1.0, h0t, pos, lens)
    out["dq"] = back(dq, row, s["q"])
    del q, k, v, do, o, dq
    turned = row + lens[:, None] - 1 - 2 * pos  # the same sequences, last token first
    q, k, v, do = (rows(s[n], turned) for n in ("q", "k", "v", "do"))
    df = s["dfinal"]
    dv, dh0 = _chunked(k, q, do, ld, 1, 1.0, scale, scale, df, pos, lens)
    dk, _ = _chunked(v, do, q, ld, 1, 1.0, scale, scale, df.transpose(-1, -2).contiguous(), pos,
                     lens)
    out.update(dk=back(dk, turned, s["k"]), dv=back(dv, turned, s["v"]))
    if c["init"]:
        out["dh0"] = dh0
    return out


def _plain_decode(s):
    a = torch.exp(s["log_decay"].double()).float()[None, :, None, None]
    q, k, v = (s[n].float() for n in "qkv")
    new = s["state"] * a + k[..., :, None] * v[..., None, :]
    o = torch.matmul(q[..., None, :], new)[..., 0, :] * q.shape[-1] ** -0.5
    return dict(o=o.to(s["v"].dtype), state=new)


def _plain_norm(s, train):
    c = s["case"]
    x, z, w = s["x"].float(), s["gate"].float(), s["weight"]
    sg = 1.0 / (1.0 + torch.exp(-z))
    act = sg if c["act"] == "sigmoid" else z * sg
    if c["res"]:
        r, rs = s["residual"].float(), s["residual_scale"][None, :, None]
        x = x + rs * r
    rho = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * rho
    out = dict(y=(n * w * act).to(s["x"].dtype))
    if not train:
        return out
    dy = s["dy"].float()
    slope = sg * (1 - sg) if c["act"] == "sigmoid" else sg * (1 + z * (1 - sg))
    p = dy * w * act
    dx = rho * (p - n * (p * n).mean(-1, keepdim=True))
    bf = s["x"].dtype
    out.update(dx=dx.to(bf), dgate=(dy * n * w * slope).to(bf),
               dweight=(dy * n * act).sum((0, 1), dtype=torch.float64).float())
    if c["res"]:
        out.update(dresidual=(dx * rs).to(bf),
                   dresidual_scale=(dx * r).sum((0, 2), dtype=torch.float64).float())
    return out


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    c = dict(case)
    if not c["op"].startswith("norm") and c["op"] != "la_decode" and max(_lengths(c)) > 140000:
        return None
    s = prepare(case, seed)
    if c["op"].startswith("norm"):
        return _exact_norm(s, c)
    a = torch.exp(s["log_decay"].double())[None, :, None, None]
    if c["op"] == "la_decode":
        q, k, v = (s[n].double() for n in "qkv")
        new = a * s["state"].double() + k.unsqueeze(-1) * v.unsqueeze(-2)
        return dict(o=(q.unsqueeze(-1) * new).sum(-2) / math.sqrt(c["K"]), state=new)
    return _exact_la(s, c, a)


def _exact_la(s, c, a):
    """The recurrence, token by token."""
    lens = _lengths(c)
    N, H, K, V = len(lens), c["H"], c["K"], c["V"]
    B, T = _rows(c)
    f = {n: s[n].reshape(B * T, H, -1).double() for n in ("q", "k", "v", "do") if n in s}
    start = [sum(lens[:i]) for i in range(N)]
    scale = 1.0 / math.sqrt(K)
    new = lambda d: torch.zeros(B * T, H, d, device=DEV, dtype=torch.float64)  # noqa: E731
    o, dq, dk, dv = new(V), new(K), new(K), new(V)
    S = torch.zeros(N, H, K, V, device=DEV, dtype=torch.float64)
    if s["h0"] is not None:
        S += s["h0"]
    train = c["op"] == "la_train"
    # the longest first, so that the sequences still running are the first n
    order = sorted(range(N), key=lambda i: -lens[i])
    at = torch.tensor([start[i] for i in order], device=DEV)
    last = torch.tensor([start[i] + lens[i] - 1 for i in order], device=DEV)
    ordt = torch.tensor(order, device=DEV)
    S = S[ordt].contiguous()
    alive = [sum(x > t for x in lens) for t in range(max(lens))]
    for t in range(max(lens)):
        n = alive[t]
        r = at[:n] + t
        Sn = S[:n]
        Sn.mul_(a).addcmul_(f["k"][r].unsqueeze(-1), f["v"][r].unsqueeze(-2))
        o[r] = torch.matmul(f["q"][r].unsqueeze(-2), Sn).squeeze(-2)
        if train:
            dq[r] = torch.matmul(Sn, f["do"][r].unsqueeze(-1)).squeeze(-1)
    inv = torch.argsort(ordt)
    out = dict(o=(o * scale).view(s["v"].shape), final_state=S[inv])
    if not train:
        return out
    E = s["dfinal"].double()[ordt].contiguous()
    for t in range(max(lens)):
        n = alive[t]
        r = last[:n] - t
        En = E[:n]
        En.addcmul_(f["q"][r].unsqueeze(-1), f["do"][r].unsqueeze(-2), value=scale)
        dv[r] = torch.matmul(f["k"][r].unsqueeze(-2), En).squeeze(-2)
        dk[r] = torch.matmul(En, f["v"][r].unsqueeze(-1)).squeeze(-1)
        En.mul_(a)
    out.update(dq=(dq * scale).view(s["q"].shape), dk=dk.view(s["k"].shape),
               dv=dv.view(s["v"].shape))
    if c["init"]:
        out["dh0"] = E[inv]
    return out


def _exact_norm(s, c):
    """Gradients by the chain rule on each row's own terms, in 64 bits."""
    d = {n: t.double() for n, t in s.items() if isinstance(t, torch.Tensor)}
    u = d["x"]
    if c["res"]:
        u = u + d["residual_scale"].view(1, -1, 1) * d["residual"]
    D = u.shape[-1]
    ms = (u * u).sum(-1, keepdim=True) / D + EPS
    sig = torch.special.expit(d["gate"])
    g = sig if c["act"] == "sigmoid" else sig * d["gate"]
    y = u / ms.sqrt() * d["weight"] * g
    out = dict(y=y)
    if c["op"] == "norm_fwd":
        return out
    dy = d["dy"]
    t = dy * d["weight"] * g                       # dL/d(u / sqrt(ms))
    du = t / ms.sqrt() - u * (t * u).sum(-1, keepdim=True) / (D * ms * ms.sqrt())
    dg = sig * (1 - sig)
    if c["act"] == "silu":
        dg = sig + d["gate"] * dg
    out.update(dx=du, dgate=dy * u / ms.sqrt() * d["weight"] * dg,
               dweight=(dy * u / ms.sqrt() * g).sum((0, 1)))
    if c["res"]:
        out.update(dresidual=du * d["residual_scale"].view(1, -1, 1),
                   dresidual_scale=(du * d["residual"]).sum((0, 2)))
    return out
