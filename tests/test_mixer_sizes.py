"""The token-mixer operators at the sizes where their launch rules change: runs of 16, 32 and 64
tokens in the convolution, several tokens per block in the head norm, whole sequences and pieces of
several staged tiles in the scan. The references are the definitions in 64 bits with torch (tensors
of the operators' layouts), held against the oracle's loops on the CPU."""
import numpy as np
import pytest
import torch

from oracle import mixer_oracle as M
from test_weight_layers_ttt_b200 import abi, layer

from gpu_helpers import dev, host, torch_dtype
from test_mixer_gpu import U, conv_case, heads_case, near, rand, scan_case, scan_roundings


# ----------------------------------------------------------------------------- 64-bit references
def alive(lens, B, N, device):
    n = torch.full((B,), N) if lens is None else torch.as_tensor(lens)
    return torch.arange(N, device=device)[None] < n.to(device)[:, None]


def conv64(x, w, bias, act, state, lens, dy, dstate):
    """y, state, dx, dw, dbias, dstate_in and the sums of magnitudes behind dw and dbias."""
    B, N, D = x.shape
    K = w.shape[0]
    on = alive(lens, B, N, x.device)[..., None]
    n = on.sum(1)
    hist = torch.cat([torch.zeros_like(x[:, :1]).expand(-1, K - 1, -1) if state is None else state,
                      torch.where(on, x, 0.0)], 1)
    rows = (n + torch.arange(K - 1, device=x.device))[..., None].expand(-1, -1, D)
    pre = bias + sum(w[j] * hist[:, K - 1 - j:K - 1 - j + N] for j in range(K))
    s = torch.sigmoid(pre)
    y = torch.where(on, pre * s if act else pre, 0.0)
    g = torch.where(on, dy * (s * (1 + pre * (1 - s))) if act else dy, 0.0)
    dh = torch.zeros_like(hist).scatter_(1, rows, dstate)
    dw, size = [], []
    for j in range(K):
        part = hist[:, K - 1 - j:K - 1 - j + N]
        dh[:, K - 1 - j:K - 1 - j + N] += w[j] * g
        dw.append((g * part).sum((0, 1)))
        size.append((g * part).abs().sum((0, 1)).max())
    return (y, hist.gather(1, rows), torch.where(on, dh[:, K - 1:], 0.0), torch.stack(dw), g.sum((0, 1)),
            dh[:, :K - 1], max(size), g.abs().sum((0, 1)).max())


def scan64(u, dt, A, Bm, Cm, D, z, dt_bias, state, lens, dy, dstate):
    """y, last state, the gradients by name and the sums of magnitudes behind them."""
    B, N, d = u.shape
    G, S = Bm.shape[2:]
    on = alive(lens, B, N, u.device)[..., None]
    u, dt, dy = (torch.where(on, t, 0.0) for t in (u, dt, dy))
    z = None if z is None else torch.where(on, z, 0.0)
    Bm, Cm = (torch.where(on[..., None], t, 0.0) for t in (Bm, Cm))
    raw = dt + dt_bias
    delta = torch.where(on, torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs())), 0.0)
    wide = lambda m, t: m[:, t].repeat_interleave(d // G, 1)                                # noqa: E731
    hs = [torch.zeros_like(u[:, 0, :, None].expand(-1, -1, S)) if state is None else state]
    y = torch.empty_like(u)
    for t in range(N):
        hs.append(torch.exp(delta[:, t, :, None] * A) * hs[-1] + (delta * u)[:, t, :, None] * wide(Bm, t))
        y[:, t] = (wide(Cm, t) * hs[-1]).sum(-1)
    y = torch.where(on, y + D * u, 0.0)
    g, o, size = dy, {}, {}
    if z is not None:
        s = torch.sigmoid(z)
        o["dz"] = dy * y * (s * (1 + z * (1 - s)))
        g, y = dy * (z * s), y * (z * s)
    dh = torch.zeros_like(hs[0]) if dstate is None else dstate
    du, dd, dA, absA = torch.empty_like(u), torch.empty_like(u), torch.zeros_like(A), torch.zeros_like(A)
    dB, dC, size["dB"], size["dC"] = torch.empty_like(Bm), torch.empty_like(Cm), 0.0, 0.0
    groups = lambda v: v.view(B, G, d // G, S)                                              # noqa: E731
    for t in range(N - 1, -1, -1):
        a = torch.exp(delta[:, t, :, None] * A)
        dh = dh + g[:, t, :, None] * wide(Cm, t)
        p, x = dh * a * hs[t], (dh * wide(Bm, t)).sum(-1)
        dA += (delta[:, t, :, None] * p).sum(0)
        absA += (delta[:, t, :, None] * p).abs().sum(0)
        for name, out, v in (("dB", dB, groups(dh * (delta * u)[:, t, :, None])),
                             ("dC", dC, groups(g[:, t, :, None] * hs[t + 1]))):
            out[:, t] = v.sum(2)
            size[name] = max(size[name], float(v.abs().sum(2).max()))
        du[:, t], dd[:, t] = delta[:, t] * x, (A * p).sum(-1) + u[:, t] * x
        dh = a * dh
    ddt = torch.where(on, dd * torch.sigmoid(raw), 0.0)
    o.update(du=du + g * D, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(g * u).sum((0, 1)), ddt_bias=ddt.sum((0, 1)),
             dstate=dh)
    size.update(dA=float(absA.max()), dD=float((g * u).abs().sum((0, 1)).max()),
                ddt_bias=float(ddt.abs().sum((0, 1)).max()))
    return y, hs[-1], o, size


def f64(v, device):
    return torch.as_tensor(v, dtype=torch.float64, device=device) if isinstance(v, np.ndarray) else v


@pytest.mark.parametrize("act,lens", [(True, [0, 5, 7]), (False, None)])
def test_conv64_is_the_oracle(act, lens):
    rng = np.random.default_rng(0)
    x, w, bias = rng.normal(size=(3, 7, 4)), rng.normal(size=(3, 4)), rng.normal(size=4)
    st, dy, ds = rng.normal(size=(3, 2, 4)), rng.normal(size=(3, 7, 4)), rng.normal(size=(3, 2, 4))
    got = conv64(*(f64(v, "cpu") for v in (x, w, bias)), act, f64(st, "cpu"), lens, f64(dy, "cpu"), f64(ds, "cpu"))
    ref = M.short_conv(x, w, bias, act, st, lens) + M.short_conv_backward(x, w, dy, bias, act, st, lens, ds)
    for g, r in zip(got, ref):
        assert np.allclose(g.numpy(), r, rtol=0, atol=1e-12)


@pytest.mark.parametrize("gate,lens,G", [(True, [6, 0, 3], 2), (False, None, 1)])
def test_scan64_is_the_oracle(gate, lens, G):
    rng = np.random.default_rng(1)
    B, N, D, S = 3, 6, 4, 3
    v = dict(u=rng.normal(size=(B, N, D)), dt=rng.normal(size=(B, N, D)), A=-rng.uniform(0.2, 2, size=(D, S)),
             Bm=rng.normal(size=(B, N, G, S)), Cm=rng.normal(size=(B, N, G, S)), D=rng.normal(size=D),
             z=rng.normal(size=(B, N, D)) if gate else None, dt_bias=rng.normal(size=D),
             state=rng.normal(size=(B, D, S)), lens=lens)
    dy, ds = rng.normal(size=(B, N, D)), rng.normal(size=(B, D, S))
    y, last, grads, _ = scan64(**{k: f64(x, "cpu") for k, x in v.items()}, dy=f64(dy, "cpu"), dstate=f64(ds, "cpu"))
    ry, hs = M.selective_scan(**v)
    ref = M.selective_scan_backward(**v, dy=dy, dstate=ds)
    assert np.allclose(y, ry, rtol=0, atol=1e-12) and np.allclose(last, hs[:, -1], rtol=0, atol=1e-12)
    for name, g in grads.items():
        assert np.allclose(g, ref[name], rtol=0, atol=1e-12), name


def close(got, ref, roundings, what, terms=0.0):
    """near() of test_mixer_gpu on the GPU: half a step of got's type at ref, plus ``roundings`` fp32
    half steps at the array's largest value or at ``terms``, the sum of the magnitudes behind it."""
    half = torch.finfo(got.dtype).eps / 2
    off = (got.double() - ref).abs()
    worst = float((off - half * ref.abs()).max()) - roundings * U * max(float(ref.abs().max()), float(terms))
    assert got.shape == ref.shape and bool(torch.isfinite(got).all()) and worst <= 0, \
        f"{what}: {float(off.max())} off, {worst} too much"


# ----------------------------------------------------------------------------- convolution
CONV = [  # dtype, B, N, D, width, act, state, lens, pad; tokens of a run in the backward
    (("bf16", 2, 2401, 8192, 4, "silu", True, [2401, 1111], 0), 64),
    (("bf16", 2, 500, 8192, 4, "silu", False, None, 8), 32),
    (("bf16", 2, 250, 8192, 3, None, True, [250, 33], 0), 16),
    (("fp32", 1, 1300, 4099, 5, "silu", True, [1299], 0), 32),
    (("bf16", 1, 2400, 4099, 2, "silu", False, None, 0), 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case,run", CONV)
def test_short_conv_runs(case, run):
    dtype, B, N, D, width, act, state, lens, pad = case
    x, w, bias, st, xg, wg, g, rng = conv_case(*case)
    td = torch_dtype(dtype)
    dy, ds = dev(rand(rng, B, N, D, dtype=dtype), td), dev(rand(rng, B, width - 1, D, dtype=dtype), td)
    desc = abi.ttt_conv_desc(B, N, D, width, abi.TTT_DTYPE_BF16 if dtype == "bf16" else abi.TTT_DTYPE_FP32, 1)
    assert abi.ttt_short_conv_bwd_workspace_bytes(desc) == B * -(-N // run) * (width + 1) * D * 4
    del x
    y, new = layer.short_conv_fwd(xg, wg, **g)
    got = layer.short_conv_bwd(xg, wg, dy, dstate=ds, **g)
    ref = conv64(xg.double(), wg.double(), g["bias"].double(), act == "silu",
                 None if st is None else g["state"].double(), lens, dy.double(), ds.double())
    close(y, ref[0], 4 * width + 32, "y")
    assert torch.equal(new.double(), ref[1])
    close(got[0], ref[2], 4 * width + 48, "dx")
    # a sum of B N terms, each off by some 48 roundings: a run, a sixteenth of the runs, their join
    chain = 48 + run + B * -(-N // run) // 16 + 32
    close(got[1], ref[3], chain, "dw", ref[6])
    close(got[2], ref[4], chain, "dbias", ref[7])
    if state:
        close(got[3], ref[5], 4 * width + 48, "dstate")


# ----------------------------------------------------------------------------- heads
# A block takes 2^k tokens from 592 * 2^k tokens on, as many as its lane groups (128 for rows of one
# access, 4 for the widest); the backward's blocks go through several such tiles.
HEADS = [  # dtype, B, N, (Hq, Hk, Hv), h, norm, weight, rot, pairs, far, pad
    ("bf16", 1, 1201, (3, 2, 1), 256, "l2", True, 256, "halves", 0, 0),
    ("bf16", 2, 1250, (2, 1, 0), 33, "rms", True, 32, "halves", 100, 0),
    ("fp32", 3, 2501, (1, 3, 2), 64, "rms", True, 30, "interleaved", 5000, 4),
    ("bf16", 1, 20011, (2, 1, 1), 128, "rms", True, 64, "interleaved", 0, 8),
    ("bf16", 1, 80001, (1, 2, 1), 16, "l2", True, 16, "halves", 0, 0),
    ("fp32", 1, 40003, (2, 1, 0), 7, None, True, 4, "interleaved", 3, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", HEADS)
def test_heads_of_many_tokens(case):
    dtype, B, N, H, h, norm = case[:6]
    xs, ws, xg, kw, ok, rng = heads_case(*case)
    td = torch_dtype(dtype)
    out = layer.head_norm_rope_fwd(*xg, **kw)
    dg = [None if not n else dev(rand(rng, B, n, N, h, dtype=dtype), td) for n in H]
    got = layer.head_norm_rope_bwd(*xg, *dg, **kw)
    for i in range(2):
        near(out[i], M.head_norm_rope(xs[i], ws[i], **ok), h + 32, "qk"[i])
        do = host(dg[i])
        dx, dw = M.head_norm_rope_backward(xs[i], do, ws[i], **ok)
        # dx: two terms of at most r sqrt(h) max |g| (by Cauchy-Schwarz, either norm), |R^T dout| <= 2 |dout|
        sq = (xs[i] ** 2).sum(-1)
        r = {"l2": 1 / np.sqrt(sq + 1e-6), "rms": 1 / np.sqrt(sq / h + 1e-6), None: np.ones_like(sq)}[norm]
        g = 2 * np.abs(do).max()
        near(got[i], dx, 4 * h + 64, "dqk"[i + 1], terms=np.sqrt(h) * g * np.abs(ws[i]).max() * r.max())
        # dw: B N H terms of at most g |x| r, of two sums over h and some roundings each, added one
        # after another in a lane (at most all heads of a group's every 148th token), then over its
        # block's groups and the rows of at most 1184 blocks by sixteenths
        rows = B * N
        chain = h + 64 + H[i] * (rows // 148 + 1) + 16 + 1184 // 16
        near(got[3 + i], dw, chain, "dw", terms=g * (np.abs(xs[i]) * r[..., None]).sum((0, 1, 2)).max())
    if xs[2] is not None:
        assert torch.equal(out[2], xg[2].transpose(1, 2)) and torch.equal(got[2], dg[2].transpose(1, 2))


# ----------------------------------------------------------------------------- selective scan
def pieces(case, backward):
    """Pieces that the library cuts a sequence into, from the size of their states in the workspace."""
    dtype, B, N, D, S, G = case[:6]
    desc = abi.ttt_scan_desc(B, N, D, S, G, abi.TTT_DTYPE_BF16 if dtype == "bf16" else abi.TTT_DTYPE_FP32, 1)
    size = abi.ttt_selective_scan_workspace_bytes(desc, int(backward))
    lanes = 2 if S <= 8 else 4 if S <= 16 else 8 if S <= 32 else 16
    states = 4 * lanes
    if not backward:
        return size // (4 * B * D * (states + 1)) if size else 1
    blocks = -(-(D // G) // (256 // lanes))
    marks = 4 * B * -(-N // 8) * D * (states + 1)
    return (size - marks - 4 * blocks * B * N * G * 2 * states) // (4 * B * D * (2 * states + 1 + S + 2))


SCAN_FWD = [  # dtype, B, N, D, S, G, gate, state, lens, softplus, pad; pieces
    (("bf16", 9, 150, 1024, 64, 1, True, True, [150, 149, 33, 0, 1, 32, 64, 65, 97], True, 0), 1),
    (("fp32", 9, 150, 2048, 24, 1, True, True, None, True, 0), 1),
    (("bf16", 17, 100, 4096, 8, 1, False, True, None, True, 8), 1),
    (("bf16", 9, 120, 4096, 16, 2, True, False, None, True, 0), 1),
    (("fp32", 9, 100, 1001, 64, 1, True, True, None, True, 0), 1),
    (("fp32", 3, 1500, 512, 24, 1, True, True, [1500, 1000, 97], True, 0), 16),
    (("bf16", 3, 1500, 512, 64, 2, True, True, None, True, 0), 10),
    (("bf16", 2, 2000, 2048, 8, 1, True, False, [2000, 1777], True, 0), 32),
    (("fp32", 2, 2000, 1024, 16, 1, False, True, None, True, 3), 32),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case,cut", SCAN_FWD)
def test_selective_scan_of_several_tiles(case, cut):
    dtype, B, N, D, S = case[:5]
    assert pieces(case, False) == cut and N / cut > 32
    h, g, _ = scan_case(*case)
    y, st = layer.selective_scan_fwd(**g)
    v = {k: f64(x, "cuda") for k, x in h.items() if k != "softplus"}
    ry, last = forward64({"z": None, "state": None, **v})
    close(y, ry, scan_roundings(N, S), "y")
    close(st, last, scan_roundings(N, S), "state")


def forward64(v):
    """scan64's forward half (without the states of all tokens)."""
    u, dt, A, Bm, Cm, D, z, dt_bias, state, lens = (v[k] for k in (
        "u", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "state", "lens"))
    ys, n = [], u.shape[1]
    for t0 in range(0, n, 64):
        cut = slice(t0, t0 + 64)
        left = None if lens is None else [min(max(x - t0, 0), 64) for x in lens]
        y, state, _, _ = scan64(u[:, cut], dt[:, cut], A, Bm[:, cut], Cm[:, cut], D, None if z is None else z[:, cut],
                                dt_bias, state, left, torch.zeros_like(u[:, cut]), None)
        ys.append(y)
    return torch.cat(ys, 1), state


SCAN_BWD = [  # as above
    (("bf16", 6, 100, 8192, 16, 1, True, True, None, True, 0), 1),
    (("fp32", 6, 100, 4096, 24, 1, True, False, [100, 99, 8, 0, 57, 64], True, 0), 1),
    (("bf16", 6, 100, 2048, 64, 1, True, True, [100, 33, 72, 1, 80, 95], True, 0), 1),
    (("fp32", 6, 70, 2041, 40, 1, False, True, None, True, 0), 1),
    (("bf16", 2, 700, 2048, 16, 1, True, True, [700, 333], True, 0), 11),
    (("fp32", 2, 1000, 1024, 24, 2, True, True, None, True, 0), 11),
    (("bf16", 2, 900, 1024, 64, 1, False, True, None, True, 16), 6),
    (("bf16", 3, 1100, 4096, 8, 1, True, False, [1100, 1099, 500], True, 0), 9),
    (("fp32", 3, 700, 2051, 8, 1, True, True, None, True, 0), 11),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case,cut", SCAN_BWD)
def test_selective_scan_backward_of_several_tiles(case, cut):
    dtype, B, N, D, S, G = case[:6]
    assert pieces(case, True) == cut and N / cut > 32
    h, g, rng = scan_case(*case)
    dy, ds = rand(rng, B, N, D, dtype=dtype), rand(rng, B, D, S)
    got = layer.selective_scan_bwd(**g, dy=dev(dy, torch_dtype(dtype)), dstate=dev(ds))
    v = {k: f64(x, "cuda") for k, x in h.items() if k != "softplus"}
    _, _, ref, size = scan64(**{"z": None, "state": None, **v}, dy=f64(dy, "cuda"), dstate=f64(ds, "cuda"))
    # two recurrences; the sums over tokens or channels have terms with those roundings, and add
    n = 2 * scan_roundings(N, S)
    for t, name in zip(got, ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate")):
        if t is None:
            assert name == "dz" and "z" not in g or name == "dstate" and "state" not in g
        else:
            close(t, ref[name], n + {"dB": D // G, "dC": D // G}.get(name, N + B), name, size.get(name, 0.0))


@pytest.mark.gpu
def test_selective_scan_backward_past_32_bits():
    """Tensors of more than 2^31 elements: the last sequence equals a call of its own, cut at other
    places, up to the roundings of a memory of some 2000 tokens (the decays below)."""
    B, N, D = 3, 1 << 20, 768
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((B, N, D), dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        x[b].normal_(generator=gen)
    assert x.numel() > 1 << 31
    A = -torch.rand((D, 8), generator=gen, device="cuda") - 0.1
    Bm = torch.randn((B, N, 1, 8), generator=gen, device="cuda").to(torch.bfloat16)
    bias = torch.full((D,), -4.0, device="cuda")
    state = torch.randn((B, D, 8), generator=gen, device="cuda")
    got = layer.selective_scan_bwd(x, x, A, Bm, Bm, x, z=x, dt_bias=bias, state=state)
    last = [got[i][2:].clone() for i in (0, 1, 3, 4, 6, 8)]
    del got
    x1, B1 = x[2:].clone(), Bm[2:].clone()
    del x
    one = layer.selective_scan_bwd(x1, x1, A, B1, B1, x1, z=x1, dt_bias=bias, state=state[2:].clone())
    for a, b, name in zip(last, (one[i] for i in (0, 1, 3, 4, 6, 8)), ("du", "ddt", "dB", "dC", "dz", "dstate")):
        top, off = float(b.float().abs().max()), float((a.float() - b.float()).abs().max())
        step = 2.0 ** -7 if a.dtype == torch.bfloat16 else 2 * 8 * 2000 * U
        assert off <= step * top, name
