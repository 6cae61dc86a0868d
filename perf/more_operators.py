"""Cases of what stands around an attention block of this family: the gated
linear recurrence over channels, the short causal convolution in front of it
(and of q, k and v), and the layer norm in front of the block, with their
plain forms.

A case is a dict of plain values; ``op`` says which call it makes:
  scan_fwd    the recurrence over prompts
  scan_train  its forward and backward pass
  scan_decode one token for each of ``N`` sequences, the state updated
  conv_fwd    the convolution over prompts
  conv_train  its forward and backward pass
  conv_decode one token for each of ``N`` sequences, the state updated
  ln_fwd      the layer norm
  ln_train    its forward and backward pass
Packed batches (``seqs`` > 0) hold ``seqs`` sequences of ``lo`` to ``hi``
tokens (drawn from ``lens``, so that sizes are the case's own) and ``tail``
rows behind the last one, whose outputs are zeros.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def _tokens(op, **kw):
    c = dict(op=op, dtype="bf16", B=1, T=0, C=8, seqs=0, lo=0, hi=0, lens=0, tail=0, init=False)
    if op.startswith("conv"):
        c.update(W=4, bias=False, act="silu")
    c.update(kw)
    return c


def listed():
    return [
        # one short prompt of a small model: the call's latency
        dict(_tokens("scan_fwd", T=256, C=256), name="scan prompt short"),
        # a serving batch of unequal prompts without padding, the states kept for decoding
        dict(_tokens("scan_fwd", C=4096, seqs=16, lo=256, hi=4096, lens=2, init=True),
             name="scan prompts packed"),
        # one very long document: a long chain of tokens over few channels
        dict(_tokens("scan_fwd", T=131072, C=2048, init=True), name="scan prompt 131072"),
        # a training step's share of one layer
        dict(_tokens("scan_train", B=2, T=2048, C=4096, init=True), name="scan train 2x2048"),
        # training in 32 bits on odd sizes: packed documents, one-token ones among them, with
        # padding behind them and channels that fill no wavefront
        dict(_tokens("scan_train", dtype="fp32", C=360, seqs=24, lo=1, hi=1024, lens=7, tail=37),
             name="scan train odd"),
        # a serving batch's next tokens
        dict(op="scan_decode", dtype="bf16", N=64, C=4096, name="scan tokens"),
        # q, k and v of 32 heads over packed prompts, the states kept for decoding
        dict(_tokens("conv_fwd", C=12288, seqs=16, lo=256, hi=4096, lens=2, init=True),
             name="conv prompts packed"),
        # a training step's share of one layer, with a bias
        dict(_tokens("conv_train", B=2, T=2048, C=4096, bias=True), name="conv train 2x2048"),
        # a serving batch's next tokens
        dict(op="conv_decode", dtype="bf16", N=64, C=12288, W=4, bias=False, act="silu",
             name="conv tokens"),
        # the norm in front of a decode step, with the skip: the call's latency
        dict(op="ln_fwd", dtype="bf16", rows=64, D=4096, res=True, bias=True, name="norm tokens"),
        # the norm of a training step
        dict(op="ln_train", dtype="bf16", rows=16384, D=4096, res=True, bias=True,
             name="norm train"),
        # a residual stream in 32 bits, rows and channels that fill no tile
        dict(op="ln_train", dtype="fp32", rows=3001, D=1000, res=False, bias=False,
             name="norm train odd"),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_train", "scan_decode", "conv_fwd", "conv_train",
                     "conv_decode", "ln_fwd", "ln_train"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op.startswith("ln"):
        D = 8 * _spread(rng, 1, 2048)
        return dict(op=op, dtype=dtype, rows=_spread(rng, 1, max(1, min(65536, 2 ** 25 // D))),
                    D=D, res=rng.random() < 0.5, bias=rng.random() < 0.5)
    C = 8 * _spread(rng, 1, 1536)
    conv = dict(W=rng.randint(2, 4), bias=rng.random() < 0.5, act=rng.choice(["silu", "none"]))
    if op.endswith("decode"):
        c = dict(op=op, dtype=dtype, N=_spread(rng, 1, 512), C=C)
        return dict(c, **conv) if op == "conv_decode" else c
    most = max(1, (1 << 26 if op.endswith("fwd") else 1 << 24) // C)  # tokens
    c = dict(dtype=dtype, C=C, init=rng.random() < 0.5)
    if op.startswith("conv"):
        c.update(conv)
    if rng.random() < 0.5:
        n = _spread(rng, 1, min(64, most))
        hi = _spread(rng, 1, max(1, min(8192, most // n)))
        lo = rng.randint(0, hi)
        c.update(seqs=n, lo=1 if lo == 0 and hi < 64 else lo, hi=hi, lens=rng.randint(1, 10 ** 6),
                 tail=rng.choice([0, 0, rng.randint(1, 100)]))
    else:
        T = _spread(rng, 1, min(131072, most))
        c.update(B=_spread(rng, 1, max(1, min(32, most // T))), T=T)
    return _tokens(op, **c)


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
    size = TYPES[c["dtype"]].itemsize
    if c["op"].startswith("ln"):
        e, fwd = c["rows"] * c["D"], 2 + 2 * c["res"]
        if c["op"] == "ln_fwd":
            return {"bytes": size * e * fwd, "flops": 8 * e}
        return {"bytes": size * e * (fwd + 3 + c["res"]), "flops": 22 * e}
    if c["op"] == "scan_decode":
        e = c["N"] * c["C"]
        return {"bytes": e * (4 * size + 8), "flops": 24 * e}
    if c["op"] == "conv_decode":
        e = c["N"] * c["C"]
        return {"bytes": e * size * 2 * c["W"], "flops": (2 * c["W"] + 4) * e}
    n, e = len(_lengths(c)) * c["C"], sum(_lengths(c)) * c["C"]
    if c["op"].startswith("scan"):
        by, fl = 4 * size * e + 4 * n * (1 + c["init"]), 24 * e
        if c["op"] == "scan_train":  # x, g, gate, do read; three gradients written
            by, fl = by + 7 * size * e + 4 * n * (1 + c["init"]), fl + 50 * e
        return {"bytes": by, "flops": fl}
    state = (c["W"] - 1) * size * n
    by, fl = 2 * size * e + state * (1 + c["init"]), (2 * c["W"] + 4) * e
    if c["op"] == "conv_train":
        by, fl = by + 3 * size * e + state * (1 + c["init"]), fl + (6 * c["W"] + 8) * e
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    tt = TYPES[c["dtype"]]

    def normal(*shape, dtype=tt, std=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)

    def uniform(n, lo, hi):
        return torch.rand(n, generator=g, device=DEV, dtype=torch.float64) * (hi - lo) + lo

    s = dict(case=c)
    if c["op"].startswith("ln"):
        R, D = c["rows"], c["D"]
        s["x"] = normal(R, D) + 0.25  # a residual stream's rows have a mean
        s["residual"] = normal(R, D) if c["res"] else None
        s["weight"] = 1.0 + normal(D, dtype=torch.float32, std=0.1)
        s["bias"] = normal(D, dtype=torch.float32, std=0.1) if c["bias"] else None
        if c["op"] == "ln_train":
            s["dy"] = normal(R, D)
            s["dsum"] = normal(R, D) if c["res"] else None  # what the skip itself passes back
        return s
    C = c["C"]
    if c["op"].startswith("scan"):
        # from channels that forget within a few tokens to ones that remember thousands
        s["A_log"] = torch.log(uniform(C, 1.0, 16.0)).float()
        s["dt_bias"] = torch.log(torch.expm1(torch.exp(uniform(C, math.log(1e-3),
                                                               math.log(1e-1))))).float()
    else:
        s["weight"] = normal(C, c["W"], dtype=torch.float32, std=0.5)
        s["bias"] = normal(C, dtype=torch.float32, std=0.1) if c["bias"] else None
    if c["op"].endswith("decode"):
        N = c["N"]
        s["x"] = normal(N, C)
        if c["op"] == "scan_decode":
            s["g"], s["gate"] = normal(N, C), normal(N, C)
            s["state"] = normal(N, C, dtype=torch.float32)
        else:
            s["state"] = normal(N, c["W"] - 1, C)
        s["new_state"] = torch.empty_like(s["state"])
        return s
    B, T = _rows(c)
    lens = _lengths(c)
    s["x"] = normal(B, T, C)
    state = (C,) if c["op"].startswith("scan") else (c["W"] - 1, C)
    stype = torch.float32 if c["op"].startswith("scan") else tt
    if c["op"].startswith("scan"):
        s["g"], s["gate"] = normal(B, T, C), normal(B, T, C)
    s["h0"] = normal(len(lens), *state, dtype=stype) if c["init"] else None
    s["cu"] = None
    if c["seqs"]:
        at = [0]
        for n in lens:
            at.append(at[-1] + n)
        s["cu"] = torch.tensor(at, dtype=torch.int32, device=DEV)
    if c["op"].endswith("train"):
        s["do"] = normal(B, T, C)
        s["dfinal"] = normal(len(lens), *state, dtype=stype)
    return s


# ------------------------------------------------------------------ the calls
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return _PLAIN[op](state)


def _own(op, s):
    import chunked_gated_delta_kda_amd as kda

    c = s["case"]
    if op.startswith("ln"):
        y, total = kda.layer_norm_fwd(s["x"], s["weight"], s["bias"], EPS, residual=s["residual"])
        out = dict(y=y)
        if c["res"]:
            out["sum"] = total
        if op == "ln_fwd":
            return out
        r = kda.layer_norm_bwd(total, s["weight"], s["dy"], EPS, dsum=s["dsum"],
                               need_dbias=c["bias"])
        out.update(dx=r["dx"], dweight=r["dweight"])
        if c["bias"]:
            out["dbias"] = r["dbias"]
        return out
    if op == "scan_decode":
        o, new = kda.gated_scan_decode(s["x"], s["g"], s["gate"], s["A_log"], s["dt_bias"],
                                       state=s["state"], state_out=s["new_state"])
        return dict(o=o, state=new)
    if op == "conv_decode":
        y, new = kda.short_conv_decode(s["x"], s["weight"], s["state"], s["bias"],
                                       activation=c["act"], state_out=s["new_state"])
        return dict(y=y, state=new)
    if op.startswith("scan"):
        a = (s["x"], s["g"], s["gate"], s["A_log"], s["dt_bias"])
        kw = dict(initial_state=s["h0"], cu_seqlens=s["cu"])
        if op == "scan_fwd":
            o, final = kda.gated_scan_fwd(*a, **kw)
            return dict(o=o, final_state=final)
        o, final, states = kda.gated_scan_fwd_save(*a, **kw)
        r = kda.gated_scan_bwd(*a, s["do"], states, dfinal=s["dfinal"], need_dh0=c["init"], **kw)
        out = dict(o=o, final_state=final, dx=r["dx"], dg=r["dg"], dgate=r["dinput_gate"],
                   dA_log=r["dA_log"], ddt_bias=r["ddt_bias"])
    else:
        kw = dict(activation=c["act"], initial_state=s["h0"], cu_seqlens=s["cu"])
        y, final = kda.short_conv_fwd(s["x"], s["weight"], s["bias"], **kw)
        if op == "conv_fwd":
            return dict(y=y, final_state=final)
        r = kda.short_conv_bwd(s["x"], s["weight"], s["do"], s["bias"], dfinal=s["dfinal"],
                               need_dh0=c["init"], **kw)
        out = dict(y=y, final_state=final, dx=r["dx"], dweight=r["dweight"])
        if c["bias"]:
            out["dbias"] = r["dbias"]
    if c["init"]:
        out["dh0"] = r["dh0"]
    return out


# ------------------------------------------------------------------ plain forms
def _places(c):
    """Of every token row [B, T]: its sequence, its place in it, and the tokens
    left behind it (-1 where the row is no token)."""
    B, T = _rows(c)
    lens = torch.tensor(_lengths(c), device=DEV)
    if not c["seqs"]:
        pos = torch.arange(T, device=DEV).expand(B, T)
        return torch.arange(B, device=DEV)[:, None].expand(B, T), pos, T - 1 - pos
    ends = torch.cumsum(lens, 0)
    t = torch.arange(T, device=DEV)
    n = torch.bucketize(t, ends, right=True)
    there = n < len(lens)
    n = n.clamp(max=len(lens) - 1)
    pos = t - (ends - lens)[n]
    left = torch.where(there, ends[n] - 1 - t, -1)
    return n[None], pos[None], left[None]


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1, by doubling (a and b are used up)."""
    d = 1
    while d < a.shape[1]:
        b[:, d:] = b[:, d:] + a[:, d:] * b[:, :-d]
        a[:, d:] = a[:, d:] * a[:, :-d]
        d *= 2
    return b


def _gates(s):
    x, g, i = s["x"].float(), s["g"].float(), s["gate"].float()
    z = g + s["dt_bias"]
    L = torch.exp(s["A_log"]) * (z.clamp(min=0) + torch.log1p(torch.exp(-z.abs())))
    m = torch.sqrt(-torch.expm1(-2 * L))
    return x, z, L, torch.exp(-L), m, 1 / (1 + torch.exp(-i))


def _plain_scan(s):
    c = s["case"]
    train = c["op"] == "scan_train"
    n, pos, left = _places(c)
    there, first, last = (left >= 0)[..., None], (pos == 0) & (left >= 0), left == 0
    tt, h0 = s["x"].dtype, s["h0"]
    N = len(_lengths(c))
    x, z, L, a, m, sg = _gates(s)
    b = torch.where(there, m * sg * x, 0.0)
    if h0 is not None:
        b[first] += a[first] * h0[n[first]]
    keep = torch.where(there & ~first[..., None], a, 0.0)
    h = _scan(keep, b)
    del keep
    final = torch.zeros(N, c["C"], device=DEV)
    if h0 is not None:
        final += h0  # (of sequences without a token)
    final[n[last]] = h[last]
    out = dict(o=h.to(tt), final_state=final)
    if not train:
        return out
    before = torch.zeros_like(h)
    before[:, 1:] = h[:, :-1]
    before[first] = 0.0 if h0 is None else h0[n[first]]
    del h
    do = torch.where(there, s["do"].float(), 0.0)
    do[last] += s["dfinal"][n[last]]
    # back_t = a_t (do_t + back_{t+1}): the gradient that reaches the state before t
    keep = torch.where(there & ~last[..., None], a, 0.0).flip(1).contiguous()
    back = _scan(keep, torch.where(there, a * do, 0.0).flip(1).contiguous()).flip(1)
    del keep
    e = do
    e[:, :-1] += torch.where(last[:, :-1, None], 0.0, back[:, 1:])
    e = torch.where(there, e, 0.0)
    dh0 = s["dfinal"].clone()
    dh0[n[first]] = back[first]
    u = sg * x
    p = torch.where(there, a * e * (torch.where(m > 0, a * u / m, 0.0) - before), 0.0)
    dg = p * torch.exp(s["A_log"]) / (1 + torch.exp(-z))
    out.update(dx=(e * m * sg).to(tt), dg=dg.to(tt), dgate=(e * m * u * (1 - sg)).to(tt),
               dA_log=(p * L).sum((0, 1), dtype=torch.float64).float(),
               ddt_bias=dg.sum((0, 1), dtype=torch.float64).float())
    if c["init"]:
        out["dh0"] = dh0
    return out


def _plain_scan_decode(s):
    x, _, _, a, m, sg = _gates(s)
    new = a * s["state"] + m * sg * x
    return dict(o=new.to(s["x"].dtype), state=new)


def _act(z, act):
    """The activation and its slope."""
    if act == "none":
        return z, torch.ones_like(z)
    sg = 1 / (1 + torch.exp(-z))
    return z * sg, sg * (1 + z * (1 - sg))


def _plain_conv(s):
    c = s["case"]
    train = c["op"] == "conv_train"
    W, w, tt, h0 = c["W"], s["weight"], s["x"].dtype, s["h0"]
    n, pos, left = _places(c)
    there = (left >= 0)[..., None]
    x = s["x"].float()
    lens = torch.tensor(_lengths(c), device=DEV)
    N = len(lens)

    def earlier(k):
        """The value k tokens before each (of the state where the sequence has none)."""
        if k == 0:
            return x
        v = torch.zeros_like(x)
        v[:, k:] = x[:, :-k] if k < x.shape[1] else v[:, k:]
        out = (pos < k) & (left >= 0)
        v[out] = 0.0 if h0 is None else h0[n[out], W - 1 + pos[out] - k].float()
        return v

    z = torch.zeros_like(x) if s["bias"] is None else s["bias"].expand_as(x).clone()
    for j in range(W):
        z += w[:, j] * earlier(W - 1 - j)
    y, slope = _act(z, c["act"])
    # the state behind a sequence: its last W - 1 values, the oldest first
    final = torch.zeros(N, W - 1, c["C"], device=DEV, dtype=tt)
    b, t = torch.nonzero((left >= 0) & (left < W - 1), as_tuple=True)
    final[n[b, t], W - 2 - left[b, t]] = s["x"][b, t]
    if h0 is not None:
        for r in range(W - 1):  # what is older than a sequence shorter than the state
            old = lens <= W - 2 - r
            final[old, r] = h0[old, r + lens[old]]
    out = dict(y=torch.where(there, y, 0.0).to(tt), final_state=final)
    del y
    if not train:
        return out
    dz = torch.where(there, s["do"].float() * slope, 0.0)
    del slope
    dx = torch.zeros_like(x)
    dh0 = torch.zeros(N, W - 1, c["C"], device=DEV)
    dw = []
    for j in range(W):
        k = W - 1 - j
        dw.append((dz * earlier(k)).sum((0, 1), dtype=torch.float64).float())
        part = dz * w[:, j]
        own_row = (pos >= k) & (left >= 0)
        if k < x.shape[1]:
            dx[:, :x.shape[1] - k] += torch.where(own_row[..., None], part, 0.0)[:, k:]
        b, t = torch.nonzero((pos < k) & (left >= 0), as_tuple=True)
        dh0[n[b, t], W - 1 + pos[b, t] - k] += part[b, t]
    df = s["dfinal"].float()
    b, t = torch.nonzero((left >= 0) & (left < W - 1), as_tuple=True)
    dx[b, t] += df[n[b, t], W - 2 - left[b, t]]
    for r in range(W - 1):
        old = lens <= W - 2 - r
        dh0[old, r + lens[old]] += df[old, r]
    out.update(dx=dx.to(tt), dweight=torch.stack(dw, 1))
    if c["bias"]:
        out["dbias"] = dz.sum((0, 1), dtype=torch.float64).float()
    if c["init"]:
        out["dh0"] = dh0.to(tt)
    return out


def _plain_conv_decode(s):
    rows = torch.cat([s["state"], s["x"][:, None]], 1)
    z = (rows.float() * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        z = z + s["bias"]
    return dict(y=_act(z, s["case"]["act"])[0].to(s["x"].dtype), state=rows[:, 1:].contiguous())


def _plain_ln(s):
    c = s["case"]
    tt = s["x"].dtype
    total = s["x"]
    if c["res"]:
        total = (s["x"].float() + s["residual"].float()).to(tt)
    v = total.float()
    v = v - v.mean(-1, keepdim=True)
    rho = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    n = v * rho
    y = n * s["weight"] if s["bias"] is None else n * s["weight"] + s["bias"]
    out = dict(y=y.to(tt))
    if c["res"]:
        out["sum"] = total
    if c["op"] == "ln_fwd":
        return out
    dy = s["dy"].float()
    t = dy * s["weight"]
    dx = rho * (t - t.mean(-1, keepdim=True) - n * (t * n).mean(-1, keepdim=True))
    if c["res"]:
        dx = dx + s["dsum"].float()
    out.update(dx=dx.to(tt), dweight=(dy * n).sum(0, dtype=torch.float64).float())
    if c["bias"]:
        out["dbias"] = dy.sum(0, dtype=torch.float64).float()
    return out


_PLAIN = dict(scan_fwd=_plain_scan, scan_train=_plain_scan, scan_decode=_plain_scan_decode,
              conv_fwd=_plain_conv, conv_train=_plain_conv, conv_decode=_plain_conv_decode,
              ln_fwd=_plain_ln, ln_train=_plain_ln)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    d = {n: t.double() if t.is_floating_point() else t for n, t in s.items()
         if isinstance(t, torch.Tensor)}
    if c["op"].startswith("ln"):
        return _exact_ln(s, d, c)
    if c["op"].startswith("conv"):
        return _exact_conv(d, c)
    return _exact_scan(d, c)


def _spans(c):
    """(batch row, first token, end) of every sequence."""
    lens = _lengths(c)
    if not c["seqs"]:
        return [(b, 0, n) for b, n in enumerate(lens)]
    return [(0, sum(lens[:i]), sum(lens[:i + 1])) for i in range(len(lens))]


def _exact_scan(d, c):
    """The recurrence, token by token."""
    amount = torch.exp(d["A_log"])
    softplus = torch.logaddexp(d["g"] + d["dt_bias"], torch.zeros((), device=DEV,
                                                                  dtype=torch.float64))
    L = softplus * amount
    a = torch.exp(-L)
    root = (-torch.expm1(-2 * L)).sqrt()
    sg = torch.special.expit(d["gate"])
    inp = root * sg * d["x"]
    if c["op"] == "scan_decode":
        new = a * d["state"] + inp
        return dict(o=new, state=new)
    train = c["op"] == "scan_train"
    h = torch.zeros_like(inp)
    prev = torch.zeros_like(inp) if train else None
    spans = _spans(c)
    final = torch.zeros(len(spans), c["C"], device=DEV, dtype=torch.float64)
    if not c["seqs"]:  # all rows of the batch at once
        spans = [(slice(None), 0, c["T"])]
    for n, (b, t0, t1) in enumerate(spans):
        which = slice(None) if not c["seqs"] else n
        S = final[which].clone() if "h0" not in d else d["h0"][which].clone()
        if train and t1 > t0:
            prev[b, t0] = S
        for t in range(t0, t1):
            torch.addcmul(inp[b, t], a[b, t], S, out=h[b, t])
            S = h[b, t]
        if train and t1 > t0:
            prev[b, t0 + 1:t1] = h[b, t0:t1 - 1]
        final[which] = S
    out = dict(o=h, final_state=final)
    if not train:
        return out
    e = torch.zeros_like(inp)
    dh0 = d["dfinal"].clone()
    for n, (b, t0, t1) in enumerate(spans):
        which = slice(None) if not c["seqs"] else n
        E = dh0[which].clone()
        for t in range(t1 - 1, t0 - 1, -1):
            torch.add(d["do"][b, t], E, out=e[b, t])
            E = a[b, t] * e[b, t]
        dh0[which] = E
    # the chain rule on h = a before + root sg x
    droot = e * sg * d["x"]
    dL = -a * e * prev + droot * torch.where(root > 0, a * a / root, torch.zeros_like(root))
    dg = dL * amount * torch.special.expit(d["g"] + d["dt_bias"])
    out.update(dx=e * root * sg, dg=dg, dgate=e * root * d["x"] * sg * torch.special.expit(-d["gate"]),
               dA_log=(dL * L).sum((0, 1)), ddt_bias=dg.sum((0, 1)))
    if c["init"]:
        out["dh0"] = dh0
    return out


def _exact_conv(d, c):
    """Each sequence with its state in front."""
    W, w = c["W"], d["weight"]

    def act(z):
        return z if c["act"] == "none" else z * torch.special.expit(z)

    if c["op"] == "conv_decode":
        rows = torch.cat([d["state"], d["x"][:, None]], 1)
        z = torch.einsum("nwc,cw->nc", rows, w)
        return dict(y=act(z + d["bias"] if c["bias"] else z), state=rows[:, 1:])
    train = c["op"] == "conv_train"
    y = torch.zeros_like(d["x"])
    dx = torch.zeros_like(y) if train else None
    final, dh0 = [], []
    dw = torch.zeros(c["C"], W, device=DEV, dtype=torch.float64)
    db = torch.zeros(c["C"], device=DEV, dtype=torch.float64)
    for n, (b, t0, t1) in enumerate(_spans(c)):
        front = d["h0"][n] if c["init"] else torch.zeros(W - 1, c["C"], device=DEV,
                                                         dtype=torch.float64)
        ext = torch.cat([front, d["x"][b, t0:t1]])
        T = t1 - t0
        z = sum(ext[j:j + T] * w[:, j] for j in range(W))
        if c["bias"]:
            z = z + d["bias"]
        y[b, t0:t1] = act(z)
        final.append(ext[T:])
        if not train:
            continue
        dz = d["do"][b, t0:t1]
        if c["act"] == "silu":
            sg = torch.special.expit(z)
            dz = dz * (sg + z * sg * torch.special.expit(-z))
        dext = torch.zeros_like(ext)
        for j in range(W):
            dext[j:j + T] += dz * w[:, j]
            dw[:, j] += (dz * ext[j:j + T]).sum(0)
        db += dz.sum(0)
        dext[T:] += d["dfinal"][n]
        dx[b, t0:t1] = dext[W - 1:]
        dh0.append(dext[:W - 1])
    out = dict(y=y, final_state=torch.stack(final))
    if train:
        out.update(dx=dx, dweight=dw)
        if c["bias"]:
            out["dbias"] = db
        if c["init"]:
            out["dh0"] = torch.stack(dh0)
    return out


def _exact_ln(s, d, c):
    """Gradients by the chain rule on each row's own terms.  The sum that is
    normalised is the one that is handed on: rounded to the tokens' type."""
    total = d["x"] + d["residual"] if c["res"] else d["x"]
    v = total.to(s["x"].dtype).double()
    D = v.shape[-1]
    mean = v.sum(-1, keepdim=True) / D
    dev = v - mean
    std = ((dev * dev).sum(-1, keepdim=True) / D + EPS).sqrt()
    y = dev / std * d["weight"]
    out = dict(y=y + d["bias"] if c["bias"] else y)
    if c["res"]:
        out["sum"] = total
    if c["op"] == "ln_fwd":
        return out
    t = d["dy"] * d["weight"]
    ddev = t / std - dev * (t * dev).sum(-1, keepdim=True) / (D * std ** 3)
    dx = ddev - ddev.sum(-1, keepdim=True) / D
    out.update(dx=dx + d["dsum"] if c["res"] else dx, dweight=(d["dy"] * dev / std).sum(0))
    if c["bias"]:
        out["dbias"] = d["dy"].sum(0)
    return out
