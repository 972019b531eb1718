"""The token mixer's operators on one GPU: the short causal convolution, the selective state
space scan and the head norm with position rotation, each for prompts, for training and for
single tokens. ``run`` computes them with elementary torch operations in 32 bits (``own``
false) or through this repository's package (``own`` true)."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # the lm workload's 4 heads of 256 channels through the convolution before the layer
        {"name": "conv prompt", "op": "conv", "pass": "fwd", "type": "bf16", "B": 2, "N": 32768,
         "D": 1024, "width": 4, "act": True, "state": False, "ragged": False},
        # one training micro-batch of a mid-sized model
        {"name": "conv training", "op": "conv", "pass": "bwd", "type": "bf16", "B": 4, "N": 4096,
         "D": 2048, "width": 4, "act": True, "state": False, "ragged": False},
        # full-precision training on padded sequences of odd sizes that continue a state
        {"name": "conv ragged fp32", "op": "conv", "pass": "bwd", "type": "fp32", "B": 3, "N": 1023,
         "D": 515, "width": 3, "act": False, "state": True, "ragged": True},
        # serving: the next token of 64 sequences
        {"name": "conv token", "op": "conv", "pass": "step", "type": "bf16", "B": 64, "N": 1,
         "D": 2048, "width": 4, "act": True, "state": True, "ragged": False},
        # one long prompt, few channels: the sequence itself has to be split
        {"name": "scan long prompt", "op": "scan", "pass": "fwd", "type": "bf16", "B": 1, "N": 32768,
         "D": 1024, "S": 16, "G": 1, "gate": True, "state": False, "ragged": False},
        # a batch of prompts that fills the GPU by its channels
        {"name": "scan batch", "op": "scan", "pass": "fwd", "type": "bf16", "B": 8, "N": 2048,
         "D": 4096, "S": 16, "G": 1, "gate": True, "state": False, "ragged": False},
        # the same training micro-batch as the convolution's
        {"name": "scan training", "op": "scan", "pass": "bwd", "type": "bf16", "B": 4, "N": 4096,
         "D": 2048, "S": 16, "G": 1, "gate": True, "state": False, "ragged": False},
        # full precision, two groups, an odd state, padded sequences that continue a state
        {"name": "scan ragged fp32", "op": "scan", "pass": "bwd", "type": "fp32", "B": 2, "N": 777,
         "D": 330, "S": 11, "G": 2, "gate": False, "state": True, "ragged": True},
        # serving: the next token of 64 sequences
        {"name": "scan token", "op": "scan", "pass": "step", "type": "bf16", "B": 64, "N": 1,
         "D": 4096, "S": 16, "G": 1, "gate": True, "state": True, "ragged": False},
        # the lm workload's q, k and v from the fused projection to the layer's layout
        {"name": "heads prompt", "op": "heads", "pass": "fwd", "type": "bf16", "B": 2, "N": 32768,
         "Hq": 4, "Hk": 4, "Hv": 4, "h": 256, "norm": "l2", "weight": False, "rot": 256,
         "pairs": "halves", "far": 0},
        # half of the long workload's sequence in training, with norm weights
        {"name": "heads training", "op": "heads", "pass": "bwd", "type": "bf16", "B": 1, "N": 65536,
         "Hq": 8, "Hk": 8, "Hv": 8, "h": 128, "norm": "rms", "weight": True, "rot": 128,
         "pairs": "interleaved", "far": 0},
        # serving: one token of 32 sequences, far positions, fewer key than query heads
        {"name": "heads token", "op": "heads", "pass": "fwd", "type": "bf16", "B": 32, "N": 1,
         "Hq": 16, "Hk": 4, "Hv": 4, "h": 128, "norm": "rms", "weight": True, "rot": 64,
         "pairs": "halves", "far": 1000000},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "heads"])
    mode = rng.choice(["fwd", "bwd", "step"])
    case = {"op": op, "pass": "fwd" if op == "heads" and mode == "step" else mode,
            "type": rng.choice(["bf16", "bf16", "fp32"])}
    step = mode == "step"
    B = _log(rng, 1, 256 if step else 16)
    N = 1 if step else _log(rng, 1, 32768)
    if op == "heads":
        h = rng.choice([16, 24, 64, 80, 96, 128, 128, 256, _log(rng, 3, 256)])
        H = [_log(rng, 1, 16) for _ in range(3)]
        rot = rng.choice([h // 2 * 2, h // 4 * 2, 0])
        N = max(1, min(N, 40_000_000 // (B * sum(H) * h)))
        case.update(B=B, N=N, Hq=H[0], Hk=H[1], Hv=rng.choice([0, H[2]]), h=h,
                    norm=rng.choice(["l2", "rms", "none"]), weight=rng.random() < 0.5, rot=rot,
                    pairs=rng.choice(["halves", "interleaved"]),
                    far=rng.choice([0, _log(rng, 1, 2000000)]))
        return case
    more = {"state": step or rng.random() < 0.5, "ragged": not step and rng.random() < 0.4}
    if op == "conv":
        D = _log(rng, 1, 8192)
        N = max(1, min(N, 30_000_000 // (B * D)))
        case.update(B=B, N=N, D=D, width=rng.choice([2, 3, 4, 4, 5, 7]), act=rng.random() < 0.7,
                    **more)
        return case
    G = rng.choice([1, 1, 1, 2, 4])
    D = G * _log(rng, 1, 4096 // G)
    S = rng.choice([16, 16, 16, 8, 32, 64, _log(rng, 1, 64)])
    N = max(1, min(N, (64_000_000 if mode == "bwd" else 250_000_000) // (B * D * S)))
    case.update(B=B, N=N, D=D, S=S, G=G, gate=rng.random() < 0.6, **more)
    return case


# ----------------------------------------------------------------------------- the inputs
def prepare(case, seed):
    dt = DTYPES[case["type"]]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=dt, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo

    f32 = torch.float32
    B, N = case["B"], case["N"]
    s = {"case": case}
    if case["op"] == "heads":
        h, heads = case["h"], [case["Hq"], case["Hk"], case["Hv"]]
        rows = normal(B, N, sum(heads) * h)      # the fused projection's output
        parts = rows.split([n * h for n in heads], dim=-1)
        s["q"], s["k"], s["v"] = (p.unflatten(-1, (n, h)) if n else None
                                  for p, n in zip(parts, heads))
        s["wq"], s["wk"] = ((1 + normal(h, dtype=f32, std=0.1) for _ in range(2))
                            if case["weight"] else (None, None))
        s["inv_freq"] = None
        if case["rot"]:
            i = torch.arange(case["rot"] // 2, device="cuda", dtype=f32)
            s["inv_freq"] = 10000.0 ** (-2 * i / case["rot"])
        start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda")
        s["positions"] = (start + torch.arange(N, device="cuda")).to(torch.int32)
        if case["pass"] == "bwd":
            s["dq"], s["dk"], s["dv"] = (normal(B, n, N, h) if n else None for n in heads)
        return s
    D = case["D"]
    s["lens"] = None
    if case["ragged"]:
        s["lens"] = torch.randint(0, N + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    if case["op"] == "conv":
        K = case["width"]
        rows = (B, D) if case["pass"] == "step" else (B, N, D)
        s["x"] = normal(*rows)
        s["w"] = normal(K, D, dtype=f32, std=K ** -0.5)
        s["bias"] = normal(D, dtype=f32, std=0.1)
        s["state"] = normal(B, K - 1, D) if case["state"] else None
        if case["pass"] == "bwd":
            s["dy"] = normal(B, N, D)
            s["dstate"] = normal(B, K - 1, D) if case["state"] else None
        return s
    S, G = case["S"], case["G"]
    rows = (B,) if case["pass"] == "step" else (B, N)
    s["u"] = normal(*rows, D)
    s["dt"] = normal(*rows, D, std=0.5)
    s["A"] = -torch.arange(1, S + 1, device="cuda", dtype=f32) * uniform(0.7, 1.4, D, S)
    s["Bm"], s["Cm"] = normal(*rows, G, S), normal(*rows, G, S)
    s["D"] = 1 + normal(D, dtype=f32, std=0.1)
    step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), D))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))     # softplus(dt_bias) = step
    s["z"] = normal(*rows, D) if case["gate"] else None
    s["state"] = normal(B, D, S, dtype=f32) if case["state"] else None
    if case["pass"] == "bwd":
        s["dy"] = normal(B, N, D)
        s["dstate"] = normal(B, D, S, dtype=f32) if case["state"] else None
    return s


# ----------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    if c["op"] == "heads":
        return _heads_bwd(s, c) if c["pass"] == "bwd" else _heads_fwd(s, c)
    if c["op"] == "conv":
        return {"fwd": _conv_fwd, "bwd": _conv_bwd, "step": _conv_step}[c["pass"]](s, c)
    return {"fwd": _scan_fwd, "bwd": _scan_bwd, "step": _scan_step}[c["pass"]](s, c)


def _own(s, c):
    from test_weight_layers_ttt_b200 import layer
    if c["op"] == "heads":
        kw = dict(wq=s["wq"], wk=s["wk"], norm=None if c["norm"] == "none" else c["norm"], eps=1e-6,
                  inv_freq=s["inv_freq"], positions=s["positions"], pairs=c["pairs"])
        if c["pass"] == "fwd":
            return layer.head_norm_rope_fwd(s["q"], s["k"], s["v"], **kw)
        return layer.head_norm_rope_bwd(s["q"], s["k"], s["v"], s["dq"], s["dk"], s["dv"], **kw)
    if c["op"] == "conv":
        act = "silu" if c["act"] else None
        if c["pass"] == "step":
            return layer.short_conv_step(s["x"], s["w"], s["state"], bias=s["bias"], act=act), s["state"]
        kw = dict(bias=s["bias"], act=act, state=s["state"], lens=s["lens"])
        if c["pass"] == "fwd":
            return layer.short_conv_fwd(s["x"], s["w"], **kw)
        return layer.short_conv_bwd(s["x"], s["w"], s["dy"], dstate=s["dstate"], **kw)
    kw = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    a = (s["u"], s["dt"], s["A"], s["Bm"], s["Cm"])
    if c["pass"] == "step":
        return layer.selective_scan_step(*a, s["state"], **kw), s["state"]
    kw.update(state=s["state"], lens=s["lens"])
    if c["pass"] == "fwd":
        return layer.selective_scan_fwd(*a, **kw)
    return layer.selective_scan_bwd(*a, s["dy"], dstate=s["dstate"], **kw)


# ------------------------------------------------------- the plain forms: convolution
def _keep(s, N):
    """1 for the tokens of a sequence, 0 behind its end: [B, N, 1] (None: all)."""
    if s["lens"] is None:
        return None
    return (torch.arange(N, device="cuda")[None, :] < s["lens"][:, None]).float()[..., None]


def _before(s, c):
    """The inputs with the width - 1 tokens before them: [B, width - 1 + N, D] in 32 bits."""
    x = s["x"].float()
    k = _keep(s, c["N"])
    if k is not None:
        x = torch.where(k > 0, x, 0.0)
    st = s["state"]
    st = x.new_zeros(c["B"], c["width"] - 1, c["D"]) if st is None else st.float()
    return torch.cat([st, x], dim=1)


def _last(s, c, x):
    """Row numbers, in _before's axis, of the state after the last token: [B, width - 1, D]."""
    n = torch.full((c["B"],), c["N"], device="cuda") if s["lens"] is None else s["lens"]
    at = n.long()[:, None] + torch.arange(c["width"] - 1, device="cuda")[None, :]
    return at[..., None].expand(-1, -1, c["D"])


def _taps(x, s, c):
    """bias + sum_j w[j] x[t - j]"""
    K, N = c["width"], c["N"]
    wins = torch.stack([x[:, K - 1 - j:K - 1 - j + N] for j in range(K)])     # [K, B, N, D]
    return s["bias"] + (wins * s["w"][:, None, None, :]).sum(0), wins


def _conv_fwd(s, c):
    x = _before(s, c)
    y, _ = _taps(x, s, c)
    y = y * torch.sigmoid(y) if c["act"] else y
    k = _keep(s, c["N"])
    y = y if k is None else y * k
    return y.to(s["x"].dtype), x.gather(1, _last(s, c, x)).to(s["x"].dtype)


def _conv_bwd(s, c):
    K, N = c["width"], c["N"]
    x = _before(s, c)
    g = s["dy"].float()
    y, wins = _taps(x, s, c)
    if c["act"]:
        sg = torch.sigmoid(y)
        g = g * (sg * (1 + y * (1 - sg)))
    k = _keep(s, N)
    g = g if k is None else torch.where(k > 0, g, 0.0)
    dw = (wins * g).sum((1, 2))
    dx = torch.zeros_like(x)
    if s["dstate"] is not None:
        dx.scatter_add_(1, _last(s, c, x), s["dstate"].float())
    pad = torch.nn.functional.pad(g, (0, 0, K - 1, K - 1))                    # [B, N + 2K - 2, D]
    outs = torch.stack([pad[:, j:j + N + K - 1] for j in range(K)])           # g[t' - (K-1) + j]
    dx = dx + (outs * s["w"][:, None, None, :]).sum(0)
    dt = s["x"].dtype
    dxs = dx[:, K - 1:]
    dxs = dxs if k is None else dxs * k
    return (dxs.to(dt), dw, g.sum((0, 1)),
            dx[:, :K - 1].to(dt) if s["state"] is not None else None)


def _conv_step(s, c):
    x = torch.cat([s["state"].float(), s["x"].float()[:, None]], dim=1)       # [B, width, D]
    y = s["bias"] + (x * s["w"].flip(0)).sum(1)
    y = y * torch.sigmoid(y) if c["act"] else y
    s["state"].copy_(x[:, 1:])
    return y.to(s["x"].dtype), s["state"]


# ------------------------------------------------------- the plain forms: scan
def _doubling(a, x):
    """h[t] = a[t] h[t - 1] + x[t] along axis 1, h[-1] = 0, in log2(N) rounds."""
    N, n = a.shape[1], 1
    while n < N:
        x = torch.cat([x[:, :n], torch.addcmul(x[:, n:], a[:, n:], x[:, :-n])], dim=1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], dim=1) if 2 * n < N else None
        n *= 2
    return x


def _delta(s, keep=None):
    raw = s["dt"].float() + s["dt_bias"]
    d = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw.clamp(max=20))))
    return (d if keep is None else torch.where(keep > 0, d, 0.0)), raw


def _grouped(m, c):
    """[..., G, S] for each channel: [..., D, S] in 32 bits."""
    return m.float().repeat_interleave(c["D"] // c["G"], dim=-2)


def _states(s, c):
    k = _keep(s, c["N"])
    delta, raw = _delta(s, k)
    u = s["u"].float()
    u = u if k is None else torch.where(k > 0, u, 0.0)
    Bm, Cm = _grouped(s["Bm"], c), _grouped(s["Cm"], c)
    if k is not None:
        Bm, Cm = torch.where(k[..., None] > 0, Bm, 0.0), torch.where(k[..., None] > 0, Cm, 0.0)
    a = torch.exp(delta[..., None] * s["A"])                                  # [B, N, D, S]
    x = (delta * u)[..., None] * Bm
    if s["state"] is not None:
        x[:, 0] += a[:, 0] * s["state"]
    return k, delta, raw, u, Bm, Cm, a, _doubling(a, x)


def _scan_fwd(s, c):
    k, _, _, u, _, Cm, _, h = _states(s, c)
    y = (h * Cm).sum(-1) + s["D"] * u
    if s["z"] is not None:
        z = s["z"].float()
        z = z if k is None else torch.where(k > 0, z, 0.0)
        y = y * (z * torch.sigmoid(z))
    return y.to(s["u"].dtype), h[:, -1]


def _scan_bwd(s, c):
    k, delta, raw, u, Bm, Cm, a, h = _states(s, c)
    B, N, D, S, G = (c[n] for n in ("B", "N", "D", "S", "G"))
    g = s["dy"].float()
    g = g if k is None else torch.where(k > 0, g, 0.0)
    dz = None
    if s["z"] is not None:
        z = s["z"].float()
        z = z if k is None else torch.where(k > 0, z, 0.0)
        sg = torch.sigmoid(z)
        dz = g * ((h * Cm).sum(-1) + s["D"] * u) * (sg * (1 + z * (1 - sg)))
        g = g * (z * sg)
    # dh[t] = C[t] g[t] + a[t + 1] dh[t + 1]: the same recurrence from the end
    x = g[..., None] * Cm
    if s["dstate"] is not None:
        x[:, -1] += s["dstate"]
    nxt = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], dim=1)
    dh = _doubling(nxt.flip(1), x.flip(1)).flip(1)
    start = torch.zeros_like(h[:, :1]) if s["state"] is None else s["state"][:, None]
    dlog = dh * a * torch.cat([start, h[:, :-1]], dim=1)      # gradient of delta A
    dxs = (dh * Bm).sum(-1)
    du = g * s["D"] + dxs * delta
    ddt = ((dlog * s["A"]).sum(-1) + dxs * u) / (1 + torch.exp(-raw))
    ddt = ddt if k is None else torch.where(k > 0, ddt, 0.0)
    dA = (dlog * delta[..., None]).sum((0, 1))
    dB = (dh * (delta * u)[..., None]).view(B, N, G, D // G, S).sum(3)
    dC = (h * g[..., None]).view(B, N, G, D // G, S).sum(3)
    dt = s["u"].dtype
    return (du.to(dt), ddt.to(dt), dA, dB.to(dt), dC.to(dt), (g * u).sum((0, 1)),
            None if dz is None else dz.to(dt), ddt.sum((0, 1)),
            dh[:, 0] * a[:, 0] if s["state"] is not None else None)


def _scan_step(s, c):
    delta, _ = _delta(s)
    u = s["u"].float()
    Bm, Cm = _grouped(s["Bm"], c), _grouped(s["Cm"], c)
    h = torch.exp(delta[..., None] * s["A"]) * s["state"] + (delta * u)[..., None] * Bm
    s["state"].copy_(h)
    y = (h * Cm).sum(-1) + s["D"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    return y.to(s["u"].dtype), s["state"]


# ------------------------------------------------------- the plain forms: heads
def _angles(s, c):
    """cos and sin [B, N, 1, rot / 2]; the angles of far positions need 64 bits."""
    ang = s["positions"].double()[:, :, None, None] * s["inv_freq"].double()
    return torch.cos(ang).float(), torch.sin(ang).float()


def _rotate(x, cs, sn, c):
    r = c["rot"]
    if c["pairs"] == "halves":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat([a * cs - b * sn, b * cs + a * sn, x[..., r:]], dim=-1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat([torch.stack([a * cs - b * sn, b * cs + a * sn], dim=-1).flatten(-2), x[..., r:]], dim=-1)


def _inv_norm(x, c):
    if c["norm"] == "none":
        return torch.ones_like(x[..., :1])
    sq = (x * x).sum(-1, keepdim=True)
    return torch.rsqrt((sq / c["h"] if c["norm"] == "rms" else sq) + 1e-6)


def _weighted(x, w):
    return x if w is None else x * w


def _heads_fwd(s, c):
    cs, sn = _angles(s, c) if c["rot"] else (None, None)

    def one(x, w):
        y = x.float()
        y = _weighted(y * _inv_norm(y, c), w)
        y = _rotate(y, cs, sn, c) if c["rot"] else y
        return y.transpose(1, 2).contiguous().to(x.dtype)

    return (one(s["q"], s["wq"]), one(s["k"], s["wk"]),
            None if s["v"] is None else s["v"].transpose(1, 2).contiguous())


def _heads_bwd(s, c):
    cs, sn = _angles(s, c) if c["rot"] else (None, None)

    def one(x, w, dout):
        g = dout.transpose(1, 2).float()
        g = _rotate(g, cs, -sn, c) if c["rot"] else g
        y = x.float()
        r = _inv_norm(y, c)
        dw = None if w is None else (g * y * r).sum((0, 1, 2))
        g = _weighted(g, w)
        dx = g * r
        if c["norm"] != "none":
            dot = (g * y).sum(-1, keepdim=True)
            dx = dx - y * (r * r * r) * (dot / c["h"] if c["norm"] == "rms" else dot)
        return dx.contiguous().to(x.dtype), dw

    (dq, dwq), (dk, dwk) = one(s["q"], s["wq"], s["dq"]), one(s["k"], s["wk"], s["dk"])
    dv = None if s["v"] is None else s["dv"].transpose(1, 2).contiguous()
    return dq, dk, dv, dwq, dwk


# ----------------------------------------------------------------------------- the work
def work(case):
    el = 2 if case["type"] == "bf16" else 4
    B, N, mode = case["B"], case["N"], case["pass"]
    if case["op"] == "heads":
        qk, v = B * N * (case["Hq"] + case["Hk"]) * case["h"], B * N * case["Hv"] * case["h"]
        extra = 4 * B * N + (8 * case["h"] if case["weight"] else 0) + 2 * case["rot"]
        if mode == "fwd":
            return {"bytes": el * 2 * (qk + v) + extra, "flops": 8 * qk}
        return {"bytes": el * (3 * qk + 2 * v) + extra + (8 * case["h"] if case["weight"] else 0),
                "flops": 16 * qk}
    D, t = case["D"], B * N * case["D"]
    if case["op"] == "conv":
        K = case["width"]
        st = B * (K - 1) * D * el if case["state"] else 0
        small = 4 * (K + 1) * D
        if mode == "bwd":
            return {"bytes": el * 3 * t + 2 * st + 2 * small, "flops": (6 * K + 8) * t}
        out = B * (K - 1) * D * el
        return {"bytes": el * 2 * t + st + out + small, "flops": (2 * K + 4) * t}
    S, G = case["S"], case["G"]
    st = 4 * B * D * S
    bc, small = 2 * B * N * G * S * el, 4 * D * (S + 2)
    gate = 1 if case["gate"] else 0
    if mode == "bwd":
        return {"bytes": el * (5 + 2 * gate) * t + 2 * bc + 2 * small + (3 * st if case["state"] else 0),
                "flops": (20 * S + 30) * t}
    return {"bytes": el * (3 + gate) * t + bc + small + st * (2 if case["state"] else 1),
            "flops": (7 * S + 12) * t}


# ----------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    d = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    B, N = c["B"], c["N"]
    if c["op"] == "heads":
        return _exact_heads(d, c)
    live = None
    if s["lens"] is not None:
        live = torch.arange(N, device="cuda")[None, :] < s["lens"][:, None]
    return _exact_conv(d, c, live) if c["op"] == "conv" else _exact_scan(d, c, live)


def _exact_conv(d, c, live):
    B, N, D, K = c["B"], c["N"], c["D"], c["width"]
    x = d["x"].view(B, N, D).clone()
    if live is not None:
        x[~live] = 0
    old = torch.zeros(B, K - 1, D, device="cuda", dtype=torch.float64) if d["state"] is None else d["state"]
    n = [N] * B if d["lens"] is None else d["lens"].tolist()
    hist = torch.cat([old, x], dim=1)
    pre = d["bias"].expand(B, N, D).clone()
    for j in range(K):
        pre += d["w"][j] * hist[:, K - 1 - j:K - 1 - j + N]
    last = torch.stack([hist[b, n[b]:n[b] + K - 1] for b in range(B)])
    if c["pass"] != "bwd":
        y = pre / (1 + torch.exp(-pre)) if c["act"] else pre
        if live is not None:
            y[~live] = 0
        return (y[:, 0] if c["pass"] == "step" else y), last
    g = d["dy"].clone()
    if c["act"]:
        sg = 1 / (1 + torch.exp(-pre))
        g = g * (sg + pre * sg * (1 - sg))
    if live is not None:
        g[~live] = 0
    dh = torch.zeros_like(hist)
    dw = torch.zeros_like(d["w"])
    for j in range(K):
        dh[:, K - 1 - j:K - 1 - j + N] += d["w"][j] * g
        dw[j] = (g * hist[:, K - 1 - j:K - 1 - j + N]).sum((0, 1))
    if d["dstate"] is not None:
        for b in range(B):
            dh[b, n[b]:n[b] + K - 1] += d["dstate"][b]
    dx = dh[:, K - 1:].clone()
    if live is not None:
        dx[~live] = 0
    return dx, dw, g.sum((0, 1)), dh[:, :K - 1] if d["state"] is not None else None


def _exact_scan(d, c, live):
    B, N, D, S, G = (c[n] for n in ("B", "N", "D", "S", "G"))
    if N > 70000 or B * N * D * S > 6e8 and c["pass"] == "bwd":
        return None
    view = lambda t: None if t is None else t.view(B, N, *t.shape[-1:])  # noqa: E731
    u, dt, z = view(d["u"]), view(d["dt"]), view(d["z"])
    Bm, Cm = d["Bm"].view(B, N, G, S), d["Cm"].view(B, N, G, S)
    raw = dt + d["dt_bias"]
    delta = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    if live is not None:
        delta = torch.where(live[..., None], delta, 0.0)
    A = d["A"].view(G, D // G, S)
    h = torch.zeros(B, G, D // G, S, device="cuda", dtype=torch.float64)
    if d["state"] is not None:
        h = d["state"].view(B, G, D // G, S).clone()
    per = lambda t, i: t[:, i].view(B, G, D // G, 1)  # noqa: E731
    back = c["pass"] == "bwd"
    hs, y = [h], torch.empty(B, N, D, device="cuda", dtype=torch.float64)
    for i in range(N):
        h = torch.exp(per(delta, i) * A) * h + per(delta * u, i) * Bm[:, i, :, None] if N == 1 else \
            torch.addcmul(torch.exp(per(delta, i) * A) * h, per(delta, i) * per(u, i), Bm[:, i, :, None])
        y[:, i] = torch.matmul(h, Cm[:, i, :, :, None]).view(B, D)
        if back:
            hs.append(h)
    y += d["D"] * u
    if live is not None:
        y[~live] = 0
    gate = None if z is None else z / (1 + torch.exp(-z))
    if not back:
        out = y if z is None else y * gate
        if live is not None:
            out[~live] = 0
        return (out[:, 0] if c["pass"] == "step" else out), h.reshape(B, D, S)
    g = d["dy"].clone()
    dz = None
    if z is not None:
        sg = 1 / (1 + torch.exp(-z))
        dz = g * y * (sg + z * sg * (1 - sg))
        g = g * gate
    if live is not None:
        g[~live] = 0
        if dz is not None:
            dz[~live] = 0
    dh = torch.zeros_like(h) if d["dstate"] is None else d["dstate"].view_as(h).clone()
    du, dde = torch.empty_like(u), torch.empty_like(u)
    dA, dB, dC = torch.zeros_like(A), torch.zeros_like(Bm), torch.zeros_like(Cm)
    for i in range(N - 1, -1, -1):
        if live is None or bool(live[:, i].any()):
            on = 1.0 if live is None else live[:, i].double().view(B, 1, 1, 1)
            gi = per(g, i)
            dh = dh + gi * Cm[:, i, :, None] * on
            dC[:, i] = (gi * hs[i + 1]).sum(2)
            a = torch.exp(per(delta, i) * A)
            through = dh * a * hs[i]
            x = (dh * Bm[:, i, :, None]).sum(-1, keepdim=True)
            dB[:, i] = (dh * per(delta, i) * per(u, i) * on).sum(2)
            du[:, i] = (x * per(delta, i)).reshape(B, D)
            dde[:, i] = ((through * A).sum(-1, keepdim=True) + x * per(u, i)).reshape(B, D)
            dA += (through * per(delta, i)).sum(0)
            dh = a * dh
        else:
            du[:, i], dde[:, i] = 0, 0
    du = du + g * d["D"]
    ddt = dde / (1 + torch.exp(-raw))
    if live is not None:
        du[~live], ddt[~live] = 0, 0
        u = torch.where(live[..., None], u, 0.0)
    return (du, ddt, dA.reshape(D, S), dB, dC, (g * u).sum((0, 1)), dz, ddt.sum((0, 1)),
            dh.reshape(B, D, S) if d["state"] is not None else None)


def _exact_heads(d, c):
    r, h = c["rot"], c["h"]
    if r:
        ang = d["positions"].double()[..., None] * d["inv_freq"]
        turn = torch.polar(torch.ones_like(ang), ang)[:, :, None]

    def spin(x, t):
        if not r:
            return x
        if c["pairs"] == "halves":
            p = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * t
            return torch.cat([p.real, p.imag, x[..., r:]], dim=-1)
        p = torch.view_as_complex(x[..., :r].contiguous().unflatten(-1, (r // 2, 2))) * t
        return torch.cat([torch.view_as_real(p).flatten(-2), x[..., r:]], dim=-1)

    def scale(x):
        if c["norm"] == "none":
            return torch.ones_like(x[..., :1])
        n = (x ** 2).sum(-1, keepdim=True)
        return 1 / torch.sqrt((n / h if c["norm"] == "rms" else n) + 1e-6)

    one = torch.ones(h, device="cuda", dtype=torch.float64)
    wq, wk = (one if w is None else w for w in (d["wq"], d["wk"]))
    lay = lambda t: None if t is None else t.transpose(1, 2).contiguous()  # noqa: E731
    if c["pass"] == "fwd":
        q, k = (spin(x * scale(x) * w, turn if r else None) for x, w in ((d["q"], wq), (d["k"], wk)))
        return lay(q), lay(k), lay(d["v"])
    got = []
    for x, w, do in ((d["q"], wq, d["dq"]), (d["k"], wk, d["dk"])):
        g = spin(do.transpose(1, 2), turn.conj() if r else None)
        n = x * scale(x)                     # the normed row: its own direction leaves the gradient
        dw = (g * n).sum((0, 1, 2))
        g = g * w
        if c["norm"] != "none":
            m = n / h if c["norm"] == "rms" else n
            g = (g - m * (g * n).sum(-1, keepdim=True)) * scale(x)
        got.append((g, dw if c["weight"] else None))
    return got[0][0], got[1][0], lay(d["dv"]), got[0][1], got[1][1]
