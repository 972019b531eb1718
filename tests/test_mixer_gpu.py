"""GPU parity of the token-mixer operators (short convolution, head norm with rotation,
selective scan) against the fp64 oracle, at the sizes, strides and masks where they can go
wrong, and a run of them together with the layer."""
import numpy as np
import pytest
import torch

from oracle import mixer_oracle as M
from oracle import ttt_oracle as O
from test_weight_layers_ttt_b200 import abi, layer

from gpu_helpers import TOL, dev, host, rel, torch_dtype

pytestmark = pytest.mark.gpu

U = 2.0 ** -24      # half a step of fp32


def near(got, ref, roundings, what="", terms=0.0):
    """|got - ref| is at most half a step of got's type at ref, plus ``roundings`` fp32 half
    steps at the largest value of the array (the terms of its sums are of that size) or at
    ``terms`` where its terms are larger than itself."""
    ref = np.asarray(ref, dtype=np.float64)
    g = host(got) if got.dtype != torch.float64 else got.cpu().numpy()
    assert g.shape == ref.shape, what
    if not ref.size:
        return
    half = torch.finfo(got.dtype).eps / 2
    allowed = half * np.abs(ref) + roundings * U * max(np.abs(ref).max(), terms)
    worst = np.max(np.abs(g - ref) - allowed)
    assert np.isfinite(g).all() and worst <= 0, f"{what}: {np.abs(g - ref).max()} off, {worst} too much"


def rand(rng, *shape, dtype="fp32", std=1.0):
    """Host values that the type holds exactly."""
    t = torch.from_numpy(rng.normal(size=shape) * std).float()
    return t.to(torch_dtype(dtype)).float().numpy()


def sliced(x, dtype, pad):
    """x on the GPU as a slice of a wider buffer: ``pad`` more elements per token, in front."""
    flat = x.reshape(*x.shape[:2], -1)
    wide = np.full(flat.shape[:2] + (flat.shape[2] + pad + 3,), np.nan)
    wide[..., pad:pad + flat.shape[2]] = flat
    t = dev(wide, torch_dtype(dtype))[..., pad:pad + flat.shape[2]]
    return t.unflatten(-1, x.shape[2:]) if x.ndim > 3 else t


# ----------------------------------------------------------------------------- convolution
# A convolution adds width products and the bias, and silu has some 10 roundings; its weight
# gradients add B * N products.
CONV = [  # dtype, B, N, D, width, act, state, lens, pad
    ("fp32", 1, 1, 1, 2, "silu", False, None, 0),
    ("fp32", 2, 70, 33, 4, "silu", True, [70, 3], 0),
    ("fp32", 3, 129, 64, 3, None, True, [0, 129, 64], 0),
    ("bf16", 2, 200, 48, 4, "silu", True, None, 16),
    ("bf16", 1, 9, 1032, 8, "silu", True, None, 0),
    ("bf16", 2, 65, 40, 5, None, False, [1, 64], 5),
    ("bf16", 4, 3, 24, 7, "silu", True, [0, 1, 2, 3], 8),
    ("bf16", 1, 300, 7, 4, "silu", False, None, 0),
    ("fp32", 1, 40, 20, 6, "silu", False, [17], 4),
    ("bf16", 2, 0, 16, 4, "silu", True, None, 0),
]


def conv_case(dtype, B, N, D, width, act, state, lens, pad, seed=0):
    rng = np.random.default_rng(seed)
    x, w, bias = rand(rng, B, N, D, dtype=dtype), rand(rng, width, D, std=0.5), rand(rng, D)
    st = rand(rng, B, width - 1, D, dtype=dtype) if state else None
    if lens is not None:        # what is behind a sequence's end is not read
        for b, n in enumerate(lens):
            x[b, n:] = np.nan
    xg = sliced(x, dtype, pad) if pad else dev(x, torch_dtype(dtype))
    g = dict(bias=dev(bias), act=act, state=None if st is None else dev(st, torch_dtype(dtype)),
             lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"))
    return x, w, bias, st, xg, dev(w), g, rng


@pytest.mark.parametrize("case", CONV)
def test_short_conv_forward(case):
    dtype, B, N, D, width, act, state, lens, pad = case
    x, w, bias, st, xg, wg, g, _ = conv_case(*case)
    y, new = layer.short_conv_fwd(xg, wg, **g)
    ry, rnew = M.short_conv(x, w, bias, act == "silu", st, lens)
    near(y, ry, 4 * width + 32, "y")
    assert np.array_equal(host(new), rnew)
    # the state written over the one it continues
    if state:
        y2, same = layer.short_conv_fwd(xg, wg, **g, state_out=g["state"])
        assert same is g["state"] and np.array_equal(host(same), rnew) and torch.equal(y, y2)


@pytest.mark.parametrize("case", CONV)
def test_short_conv_backward(case):
    dtype, B, N, D, width, act, state, lens, pad = case
    x, w, bias, st, xg, wg, g, rng = conv_case(*case)
    dy, ds = rand(rng, B, N, D, dtype=dtype), rand(rng, B, width - 1, D, dtype=dtype)
    got = layer.short_conv_bwd(xg, wg, dev(dy, torch_dtype(dtype)), dstate=dev(ds, torch_dtype(dtype)), **g)
    ref = M.short_conv_backward(x, w, dy, bias, act == "silu", st, lens, ds)
    near(got[0], ref[0], 4 * width + 48, "dx")
    near(got[1], ref[1], B * N + 64, "dw")
    near(got[2], ref[2], B * N + 64, "dbias")
    if state:
        near(got[3], ref[3], 4 * width + 48, "dstate")
    assert (got[3] is None) == (not state)


@pytest.mark.parametrize("dtype,B,D,width", [("bf16", 3, 64, 4), ("fp32", 2, 13, 3), ("bf16", 1, 5, 8)])
def test_short_conv_steps_equal_the_prompt(dtype, B, D, width):
    x, w, bias, st, xg, wg, g, _ = conv_case(dtype, B, 11, D, width, "silu", True, None, 0, seed=3)
    state = g["state"].clone()
    y, new = layer.short_conv_fwd(xg, wg, **g)
    for t in range(11):
        # a token of a wider buffer: its rows are 11 * D apart
        yt = layer.short_conv_step(xg[:, t], wg, state, bias=g["bias"])
        assert torch.equal(yt, y[:, t])
    assert torch.equal(state, new)


def test_short_conv_without_bias_and_state():
    x, w, _, _, xg, wg, _, rng = conv_case("bf16", 2, 50, 24, 4, "silu", False, None, 0, seed=5)
    y, none = layer.short_conv_fwd(xg, wg, return_state=False)
    near(y, M.short_conv(x, w)[0], 48)
    dy = rand(rng, 2, 50, 24, dtype="bf16")
    dx, dw, db, ds = layer.short_conv_bwd(xg, wg, dev(dy, torch.bfloat16))
    ref = M.short_conv_backward(x, w, dy)
    near(dx, ref[0], 64)
    near(dw, ref[1], 164)
    assert none is None and db is None and ds is None


# ----------------------------------------------------------------------------- heads
HEADS = [  # dtype, B, N, (Hq, Hk, Hv), h, norm, weight, rot, pairs, far, pad
    ("bf16", 2, 37, (4, 2, 2), 128, "l2", False, 128, "halves", 0, 0),
    ("bf16", 1, 5, (3, 1, 0), 64, "rms", True, 32, "interleaved", 1000000, 0),
    ("bf16", 2, 33, (2, 2, 1), 256, "rms", True, 256, "interleaved", 7, 24),
    ("bf16", 3, 1, (16, 4, 4), 128, "rms", True, 64, "halves", 2000000000, 0),
    ("bf16", 1, 19, (1, 1, 1), 76, "l2", True, 38, "halves", 0, 1),
    ("fp32", 2, 21, (2, 3, 1), 33, "l2", True, 20, "halves", 5, 0),
    ("fp32", 1, 17, (5, 1, 2), 80, "rms", True, 80, "halves", 50000, 12),
    ("fp32", 2, 9, (1, 2, 1), 512, "l2", False, 512, "interleaved", 0, 0),
    ("fp32", 1, 40, (2, 1, 0), 7, None, True, 6, "interleaved", 3, 0),
    ("fp32", 1, 12, (2, 2, 2), 16, "rms", False, 0, "halves", 0, 4),
    ("bf16", 1, 3, (1, 1, 1), 511, "rms", True, 510, "halves", 0, 0),
    ("bf16", 1, 2, (2, 1, 1), 1, "rms", True, 0, "halves", 0, 0),
    ("bf16", 1, 700, (2, 1, 1), 16, "rms", True, 16, "halves", 0, 0),
]


def heads_case(dtype, B, N, H, h, norm, weight, rot, pairs, far, pad, seed=0):
    rng = np.random.default_rng(seed)
    xs = [rand(rng, B, N, n, h, dtype=dtype) if n else None for n in H]
    ws = [rand(rng, h) + 1 if weight else None for _ in range(2)]
    inv = (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32) if rot else None
    pos = (rng.integers(0, far + 1, size=(B, 1)) + np.arange(N)).astype(np.int64)
    td = torch_dtype(dtype)
    xg = [None if x is None else sliced(x, dtype, pad) if pad else dev(x, td) for x in xs]
    kw = dict(norm=norm, eps=1e-6, inv_freq=None if inv is None else dev(inv), pairs=pairs,
              wq=None if ws[0] is None else dev(ws[0]), wk=None if ws[1] is None else dev(ws[1]),
              positions=torch.from_numpy(pos.astype(np.int32)).cuda())
    ok = dict(norm=norm, eps=1e-6, inv_freq=inv, pairs=pairs, positions=pos)
    return xs, ws, xg, kw, ok, rng


# A norm adds h squares; the rotation's angle is within 2^-25 of a turn (7 * 2^-24 radian).
@pytest.mark.parametrize("case", HEADS)
def test_head_norm_rope_forward(case):
    xs, ws, xg, kw, ok, _ = heads_case(*case)
    out = layer.head_norm_rope_fwd(*xg, **kw)
    for i in range(2):
        near(out[i], M.head_norm_rope(xs[i], ws[i], **ok), case[4] + 32, "qk"[i])
    if xs[2] is None:
        assert out[2] is None
    else:
        assert torch.equal(out[2], xg[2].transpose(1, 2))


@pytest.mark.parametrize("case", HEADS)
def test_head_norm_rope_backward(case):
    dtype, B, N, H, h = case[:5]
    xs, ws, xg, kw, ok, rng = heads_case(*case)
    td = torch_dtype(dtype)
    do = [rand(rng, B, n, N, h, dtype=dtype) if n else None for n in H]
    dg = [None if d is None else dev(d, td) for d in do]
    got = layer.head_norm_rope_bwd(*xg, *dg, **kw)
    for i in range(2):
        dx, dw = M.head_norm_rope_backward(xs[i], do[i], ws[i], **ok)
        # dx = g r - x r^3 <g, x> [/ h] with g = w R^T dout: two terms that may cancel (at h = 1
        # to eps / (x^2 + eps) of themselves), each with a relative error of some roundings and
        # two sums over h. |R^T dout| <= 2 max |dout|, |x| r <= 1 (L2) or sqrt(h) (RMS), and
        # |<g, x>| r <= |g|_2 (L2) or sqrt(h) |g|_2 (RMS, over h): by Cauchy-Schwarz the second
        # term is at most r |g|_2 <= r sqrt(h) max |g| in either norm.
        x = xs[i].astype(np.float64)
        sq = (x * x).sum(-1)
        r = {"l2": 1 / np.sqrt(sq + 1e-6), "rms": 1 / np.sqrt(sq / h + 1e-6), None: np.ones_like(sq)}[case[5]]
        g = 2 * np.abs(do[i]).max() * (1.0 if ws[i] is None else np.abs(ws[i]).max())
        near(got[i], dx, 4 * h + 64, "dqk"[i + 1], terms=np.sqrt(h) * g * r.max())
        if ws[i] is not None:
            near(got[3 + i], dw, B * N * H[i] + h + 64, "dw")
        else:
            assert got[3 + i] is None
    if xs[2] is not None:
        assert torch.equal(got[2], dg[2].transpose(1, 2))


def test_head_norm_rope_default_positions_and_zero_rows():
    rng = np.random.default_rng(5)
    x = rand(rng, 2, 6, 3, 32)
    x[1, 2, 1] = 0.0
    inv = np.array([1.0, 0.1, 0.01], dtype=np.float32)
    q, k, v = layer.head_norm_rope_fwd(dev(x), None, None, norm="l2", inv_freq=dev(inv), pos0=4)
    pos = np.broadcast_to(np.arange(6) + 4, (2, 6))
    near(q, M.head_norm_rope(x, None, "l2", 1e-6, inv, pos), 64)
    assert k is None and v is None and host(q)[1, 1, 2].max() == 0.0


@pytest.mark.parametrize("which", [(False, True, False), (False, False, True), (True, False, True)])
def test_head_norm_rope_of_some_tensors(which):
    xs, ws, xg, kw, ok, rng = heads_case("bf16", 2, 23, (3, 2, 4), 64, "rms", True, 32, "halves", 9, 0)
    xg = [x if on else None for x, on in zip(xg, which)]
    out = layer.head_norm_rope_fwd(*xg, **kw)
    back = layer.head_norm_rope_bwd(*xg, *out, **kw)
    for i, on in enumerate(which):
        assert (out[i] is not None) == on and (back[i] is not None) == on
        if on and i < 2:
            near(out[i], M.head_norm_rope(xs[i], ws[i], **ok), 96)
            dx, dw = M.head_norm_rope_backward(xs[i], host(out[i]), ws[i], **ok)
            near(back[i], dx, 320, terms=8 * 2 * 4)      # sqrt(64) 2 |dout| |w| r, all below 2
            near(back[3 + i], dw, 2 * 23 * 4 + 128)
        elif on:
            assert torch.equal(out[i], xg[i].transpose(1, 2)) and torch.equal(back[i], xg[i])


# ----------------------------------------------------------------------------- selective scan
SCAN = [  # dtype, B, N, D, S, G, gate, state, lens, softplus, pad
    ("fp32", 1, 1, 1, 1, 1, False, False, None, True, 0),
    ("fp32", 2, 9, 5, 3, 1, True, True, [9, 4], True, 0),
    ("fp32", 1, 33, 64, 16, 1, True, False, None, True, 0),
    ("bf16", 2, 100, 130, 16, 1, True, True, None, True, 24),
    ("bf16", 3, 40, 96, 16, 2, False, True, [0, 40, 17], True, 0),
    ("fp32", 1, 700, 6, 11, 2, True, True, None, True, 5),
    ("bf16", 1, 520, 64, 16, 1, True, False, [300], True, 0),
    ("fp32", 2, 300, 20, 8, 1, False, True, [300, 129], False, 0),
    ("bf16", 1, 70, 48, 24, 1, True, True, None, True, 0),
    ("fp32", 1, 260, 18, 33, 3, True, False, None, True, 0),
    ("bf16", 2, 65, 32, 64, 1, True, True, None, True, 16),
    ("fp32", 1, 8, 300, 2, 1, True, True, None, True, 0),
    ("bf16", 2, 0, 16, 16, 1, True, True, None, True, 0),
]


def scan_case(dtype, B, N, D, S, G, gate, state, lens, softplus, pad, seed=0):
    rng = np.random.default_rng(seed)
    x = {"u": rand(rng, B, N, D, dtype=dtype), "Bm": rand(rng, B, N, G, S, dtype=dtype),
         "Cm": rand(rng, B, N, G, S, dtype=dtype)}
    x["dt"] = rand(rng, B, N, D, dtype=dtype)
    if not softplus:
        x["dt"] = np.abs(x["dt"]) / 16
    if gate:
        x["z"] = rand(rng, B, N, D, dtype=dtype)
    p = {"A": -(np.arange(1, S + 1) * rng.uniform(0.7, 1.4, size=(D, S))).astype(np.float32),
         "D": rand(rng, D), "dt_bias": (rng.uniform(-5, -1, size=D) if softplus else
                                        rng.uniform(0, 0.1, size=D)).astype(np.float32)}
    if state:
        p["state"] = rand(rng, B, D, S)
    if lens is not None:
        for v in x.values():
            for b, n in enumerate(lens):
                v[b, n:] = np.nan
    td = torch_dtype(dtype)
    g = {k: sliced(v, dtype, pad) if pad else dev(v, td) for k, v in x.items()}
    g.update({k: dev(v) for k, v in p.items()})
    if lens is not None:
        g["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    h = {**x, **p, "lens": lens, "softplus": softplus}
    return h, {**g, "softplus": softplus}, rng


def scan_roundings(N, S):
    """A step of the recurrence rounds its exponent, exponential (2^-22), two products and the
    sum: 8 half steps, for each of N tokens; the output adds S products and the gate."""
    return 8 * N + 4 * S + 64


@pytest.mark.parametrize("case", SCAN)
def test_selective_scan_forward(case):
    dtype, B, N, D, S = case[:5]
    h, g, _ = scan_case(*case)
    y, st = layer.selective_scan_fwd(**g)
    ry, hs = M.selective_scan(**h)
    near(y, ry, scan_roundings(N, S), "y")
    near(st, hs[:, -1], scan_roundings(N, S), "state")
    if "state" in g:     # written over the state it continues
        y2, same = layer.selective_scan_fwd(**g, state_out=g["state"])
        assert same is g["state"] and torch.equal(y, y2) and torch.equal(same, st)


@pytest.mark.parametrize("case", SCAN)
def test_selective_scan_backward(case):
    dtype, B, N, D, S, G = case[:6]
    h, g, rng = scan_case(*case)
    dy, ds = rand(rng, B, N, D, dtype=dtype), rand(rng, B, D, S)
    lens = h["lens"]
    got = layer.selective_scan_bwd(**g, dy=dev(dy, torch_dtype(dtype)), dstate=dev(ds))
    ref = M.selective_scan_backward(**h, dy=dy, dstate=ds)
    # two recurrences, one in the states and one in their gradients; the sums over tokens or
    # channels add that many terms
    n = 2 * scan_roundings(N, S)
    names = ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate")
    more = {"dA": B * N, "dB": D // G, "dC": D // G, "dD": B * N, "ddt_bias": B * N}
    for t, name in zip(got, names):
        if t is None:
            assert name == "dz" and "z" not in g or name == "dstate" and "state" not in g
        else:
            near(t, ref[name], n + more.get(name, 0), name)


@pytest.mark.parametrize("dtype,D,S,G", [("bf16", 64, 16, 1), ("fp32", 10, 5, 2), ("bf16", 8, 64, 1),
                                         ("fp32", 33, 24, 1)])
def test_selective_scan_steps_continue_the_prompt(dtype, D, S, G):
    B, N, split = 2, 15, 6
    h, g, _ = scan_case(dtype, B, N, D, S, G, True, True, None, True, 0, seed=7)
    ry, hs = M.selective_scan(**h)
    tokens = ("u", "dt", "z", "Bm", "Cm")
    first = {k: v[:, :split].contiguous() if k in tokens else v for k, v in g.items()}
    y, state = layer.selective_scan_fwd(**first)
    near(y, ry[:, :split], scan_roundings(N, S))
    rest = {k: v for k, v in g.items() if k not in tokens + ("state",)}
    for t in range(split, N):
        yt = layer.selective_scan_step(state=state, **{k: g[k][:, t] for k in tokens}, **rest)
        near(yt, ry[:, t], scan_roundings(N, S), f"token {t}")
    near(state, hs[:, -1], scan_roundings(N, S))


def test_a_split_sequence_equals_two_calls():
    """The state of a first call continues in a second one, over pieces that the library itself
    splits at other places."""
    h, g, _ = scan_case("fp32", 1, 900, 8, 16, 1, True, True, None, True, 0, seed=9)
    ry, hs = M.selective_scan(**h)
    tokens = ("u", "dt", "z", "Bm", "Cm")
    state, ys = g.pop("state"), []
    for a, b in ((0, 401), (401, 402), (402, 900)):
        part = {k: v[:, a:b].contiguous() if k in tokens else v for k, v in g.items()}
        y, state = layer.selective_scan_fwd(**part, state=state)
        ys.append(y)
    near(torch.cat(ys, 1), ry, scan_roundings(900, 16))
    near(state, hs[:, -1], scan_roundings(900, 16))


def test_selective_scan_without_options():
    """No skip, gate, bias or state, and delta as it is."""
    h, g, rng = scan_case("fp32", 2, 70, 12, 16, 1, False, False, None, False, 0, seed=13)
    for k in ("D", "dt_bias"):
        h.pop(k), g.pop(k)
    y, none = layer.selective_scan_fwd(**g, return_state=False)
    near(y, M.selective_scan(**h)[0], scan_roundings(70, 16))
    dy = rand(rng, 2, 70, 12)
    got = layer.selective_scan_bwd(**g, dy=dev(dy))
    ref = M.selective_scan_backward(**h, dy=dy)
    for t, name in zip(got, ("du", "ddt", "dA", "dB", "dC")):
        near(t, ref[name], 2 * scan_roundings(70, 16) + 140, name)
    assert none is None and all(t is None for t in got[5:])


@pytest.mark.parametrize("dtype,B,D,S", [("bf16", 77, 2048, 16), ("fp32", 131, 1100, 7), ("bf16", 5, 9, 64)])
def test_selective_scan_step_of_many_sequences(dtype, B, D, S):
    rng = np.random.default_rng(17)
    h, g, _ = scan_case(dtype, B, 1, D, S, 1, True, True, None, True, 3, seed=17)
    ry, hs = M.selective_scan(**h)
    tokens = ("u", "dt", "z", "Bm", "Cm")
    g.pop("softplus")
    y = layer.selective_scan_step(**{k: v[:, 0] if k in tokens else v for k, v in g.items()})
    near(y, ry[:, 0], scan_roundings(1, S))
    near(g["state"], hs[:, -1], scan_roundings(1, S))


@pytest.mark.parametrize("n", [1, 30, 257])
def test_padded_sequences_equal_their_own_calls(n):
    """A padded batch against calls of the sequences alone (which may be cut elsewhere)."""
    h, g, rng = scan_case("fp32", 2, 300, 40, 16, 1, True, True, [n, 300], True, 0, seed=21)
    y, st = layer.selective_scan_fwd(**g)
    one = {k: v[:1] if k in ("state",) else v[:1, :n].contiguous() if k in ("u", "dt", "z", "Bm", "Cm") else v
           for k, v in g.items() if k != "lens"}
    y1, st1 = layer.selective_scan_fwd(**one)
    top = float(y1.abs().max())
    assert float((y[:1, :n] - y1).abs().max()) <= scan_roundings(n, 16) * U * top
    assert float((st[:1] - st1).abs().max()) <= scan_roundings(n, 16) * U * float(st1.abs().max())
    assert float(y[0, n:].abs().max()) == 0.0 if n < 300 else True


def test_a_step_of_zero_keeps_the_state_exactly():
    """delta = 0 decays by exp(0) = 1 and adds nothing, in the prompt, its pieces and a token."""
    h, g, _ = scan_case("fp32", 2, 600, 24, 16, 1, False, True, None, False, 0, seed=23)
    g["dt"].zero_()
    g["dt_bias"].zero_()
    before = g["state"].clone()
    _, st = layer.selective_scan_fwd(**g)
    assert torch.equal(st, before)
    one = {k: v[:, 0].contiguous() if k in ("u", "dt", "Bm", "Cm") else v for k, v in g.items()}
    layer.selective_scan_step(**one)
    assert torch.equal(g["state"], before)
    ds = torch.randn_like(before)
    got = layer.selective_scan_bwd(**g, dy=torch.zeros_like(g["u"]), dstate=ds)
    assert torch.equal(got[8], ds)


def test_nan_and_inf_stay_where_they_belong():
    h, g, _ = scan_case("fp32", 2, 300, 70, 16, 1, True, True, None, True, 0, seed=25)
    y, st = layer.selective_scan_fwd(**g)
    bad = {**g, "u": g["u"].clone()}
    bad["u"][1, 100, 33] = float("nan")
    y2, st2 = layer.selective_scan_fwd(**bad)
    assert torch.isnan(y2[1, 100:, 33]).all() and torch.isnan(st2[1, 33]).all()
    y2[1, 100:, 33], st2[1, 33] = y[1, 100:, 33], st[1, 33]
    assert torch.equal(y, y2) and torch.equal(st, st2)
    x, w, bias, _, xg, wg, c, _ = conv_case("bf16", 1, 40, 24, 4, "silu", False, None, 0, seed=26)
    y, _ = layer.short_conv_fwd(xg, wg, **c)
    xg[0, 20, 5] = float("inf")
    y2, _ = layer.short_conv_fwd(xg, wg, **c)
    ref = torch.nn.functional.silu(torch.where(wg[:, 5] > 0, float("inf"), -float("inf")))   # taps in turn
    assert torch.equal(torch.isnan(y2[0, 20:24, 5]), torch.isnan(ref)) and torch.isinf(y2[0, 20:24, 5]).equal(torch.isinf(ref))
    y2[0, 20:24, 5] = y[0, 20:24, 5]
    assert torch.equal(y, y2)
    q = torch.randn((2, 5, 3, 64), device="cuda")
    o, _, _ = layer.head_norm_rope_fwd(q, None, None)
    q[1, 2, 1, 7] = float("nan")
    o2, _, _ = layer.head_norm_rope_fwd(q, None, None)
    assert torch.isnan(o2[1, 1, 2]).all()
    o2[1, 1, 2] = o[1, 1, 2]
    assert torch.equal(o, o2)


# ----------------------------------------------------------------------------- how they are called
def together(g):
    """Projection -> short convolution -> heads -> the layer's linear attention and, beside it,
    the selective scan of the convolved channels; then both backward passes."""
    x, proj, w, S0, eta, A, inv = (g[k] for k in ("x", "proj", "w", "S0", "eta", "A", "inv"))
    B, N, _ = x.shape
    rows = x @ proj                                   # [B, N, 3 * 128 + 128 + 32 + 64]
    qkv, dt, Bm, Cm = rows[..., :384], rows[..., 384:512], rows[..., 512:528], rows[..., 528:544]
    c, conv_state = layer.short_conv_fwd(qkv, w)
    q, k, v = c.view(B, N, 3, 2, 64).unbind(2)
    heads = layer.head_norm_rope_fwd(q, k, v, inv_freq=inv)
    o, S = layer.linear_attn_fwd(*heads, eta, S0, 64)
    y, h = layer.selective_scan_fwd(c[..., :128], dt, A, Bm.unsqueeze(2), Cm.unsqueeze(2))
    grads = layer.selective_scan_bwd(c[..., :128], dt, A, Bm.unsqueeze(2), Cm.unsqueeze(2), y)
    dq = layer.head_norm_rope_bwd(q, k, v, *heads, inv_freq=inv)
    dc = layer.short_conv_bwd(qkv, w, torch.cat([t.reshape(B, N, 128) for t in dq[:3]], -1))
    return [t for t in (rows, c, conv_state, *heads, o, S, y, h, *grads, *dq, *dc) if t is not None]


def together_inputs(B=2, N=300):
    rng = np.random.default_rng(11)
    b = torch.bfloat16
    return dict(x=dev(rand(rng, B, N, 96, dtype="bf16"), b), proj=dev(rand(rng, 96, 544, dtype="bf16", std=0.1), b),
                w=dev(rand(rng, 4, 384, std=0.5)), S0=dev(rand(rng, 2, 64, 64, std=0.1)),
                eta=dev(np.abs(rand(rng, B, 2, N, std=0.1))), A=dev(-np.abs(rand(rng, 128, 16)) - 0.1),
                inv=dev((10000.0 ** (-np.arange(32) / 32)).astype(np.float32)))


def test_the_operators_run_together():
    g = together_inputs()
    got = together(g)
    rows = host(got[0])
    B, N = rows.shape[:2]
    c, cs = M.short_conv(rows[..., :384], host(g["w"]))
    near(got[1], c, 64)
    cg = host(got[1]).reshape(B, N, 3, 2, 64)          # what the next operators were given
    pos = np.broadcast_to(np.arange(N), (B, N))
    q, k = (M.head_norm_rope(cg[:, :, i], None, "l2", 1e-6, host(g["inv"]), pos) for i in range(2))
    near(got[3], q, 128)
    near(got[4], k, 128)
    ref, Sref = O.linear_attention_batched(host(got[3]), host(got[4]), host(got[5]), host(g["eta"]),
                                           host(g["S0"]), 64)
    assert rel(host(got[6]), ref) <= TOL["bf16"] and rel(host(got[7]), Sref) <= TOL["bf16"]
    u = cg.reshape(B, N, 384)[..., :128]
    y, hs = M.selective_scan(u, rows[..., 384:512], host(g["A"]), rows[..., None, 512:528], rows[..., None, 528:544])
    near(got[8], y, scan_roundings(N, 16))
    near(got[9], hs[:, -1], scan_roundings(N, 16))
    abi.ttt_last_device_status()


def test_the_same_call_gives_the_same_bits_on_streams_and_in_graphs():
    g = together_inputs()
    first = together(g)
    again = together(g)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    # another stream than the tensors' own, two calls in flight
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            runs.append(together(g))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in runs for a, b in zip(first, r))
    # two captured graphs, replayed in turn on changed inputs
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = together(g)
        graphs.append((graph, out))
    old = g["x"].clone()
    g["x"].mul_(0.5)
    changed = together(g)
    for graph, out in graphs:
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for _, out in graphs for a, b in zip(changed, out))
    g["x"].copy_(old)
    for graph, out in graphs:
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for _, out in graphs for a, b in zip(first, out))


def test_a_given_stream_is_used():
    """stream= as a torch stream and as a raw handle; the results are ready when it is."""
    g = together_inputs()
    x, w = g["x"], g["w"][:, :96].contiguous()
    y0, s0 = layer.short_conv_fwd(x, w)
    u, A = x[..., :64].contiguous(), g["A"][:64].contiguous()
    bc = x[..., 64:80].unsqueeze(2).contiguous()
    r0 = layer.selective_scan_bwd(u, u, A, bc, bc, u)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        y1, s1 = layer.short_conv_fwd(x, w, stream=stream)
        r1 = layer.selective_scan_bwd(u, u, A, bc, bc, u, stream=stream)
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]   # on the other stream
        s.synchronize()
        assert torch.equal(y0, y1) and torch.equal(s0, s1)
        assert all(torch.equal(a, b) for a, b in zip(r0[:5], r1[:5]))
        del junk


def test_debug_checks_cover_the_operators():
    g = together_inputs()
    plain = together(g)
    abi.ttt_set_debug_checks(abi.TTT_CHECK_GUARDS | abi.TTT_CHECK_FINITE)
    try:
        guarded = together(g)
        abi.ttt_last_device_status()
        assert all(torch.equal(a, b) for a, b in zip(plain, guarded))
        g["x"][1, 7, 3] = float("nan")
        together(g)
        with pytest.raises(abi.TTTError) as ei:
            abi.ttt_last_device_status()
        assert ei.value.status == abi.TTT_ERR_DEVICE and "NaN" in str(ei.value)
    finally:
        abi.ttt_set_debug_checks(0)


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last sequence equals a call of its own."""
    B, N, D = 3, 1 << 20, 768
    x = torch.empty((B, N, D), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    for b in range(B):
        x[b].normal_(generator=gen)
    assert x.numel() > 1 << 31
    w = torch.randn((4, D), generator=gen, device="cuda")
    y, _ = layer.short_conv_fwd(x, w)
    y1, _ = layer.short_conv_fwd(x[2:].contiguous(), w)
    assert torch.equal(y[2:], y1)
    del y
    gy = layer.short_conv_bwd(x, w, x)[0]
    assert torch.equal(gy[2:], layer.short_conv_bwd(x[2:].contiguous(), w, y1.copy_(x[2:]))[0])
    del gy, y1
    q = x.view(B, N, 6, 128)
    inv = torch.ones(64, device="cuda")
    o, _, _ = layer.head_norm_rope_fwd(q, None, None, inv_freq=inv)
    o1, _, _ = layer.head_norm_rope_fwd(q[2:].contiguous(), None, None, inv_freq=inv)
    assert torch.equal(o[2:], o1)
    b1 = layer.head_norm_rope_bwd(q[2:].contiguous(), None, None, o1, None, None, inv_freq=inv)[0]
    b = layer.head_norm_rope_bwd(q, None, None, o, None, None, inv_freq=inv)[0]
    assert torch.equal(b[2:], b1)
    del o, o1, b, b1
    A = -torch.rand((D, 8), generator=gen, device="cuda") - 0.1
    Bm = torch.randn((B, N, 1, 8), generator=gen, device="cuda").to(torch.bfloat16)
    bias = torch.full((D,), -4.0, device="cuda")
    y, st = layer.selective_scan_fwd(x, x, A, Bm, Bm, z=x, dt_bias=bias)
    last = [t[2:].contiguous() for t in (x, Bm)]
    y1, st1 = layer.selective_scan_fwd(last[0], last[0], A, last[1], last[1], z=last[0], dt_bias=bias)
    # cut at other places for another batch: equal up to rounding, which decays after some
    # 1 / (1 - a) < 2000 tokens here
    assert float((y[2:].float() - y1.float()).abs().max()) <= 2.0 ** -7 * float(y1.float().abs().max())
    assert float((st[2:] - st1).abs().max()) <= 8 * 2000 * U * float(st1.abs().max())


def test_refusals_name_the_tensor():
    x = torch.zeros((2, 8, 16), device="cuda")
    w = torch.zeros((4, 16), device="cuda")
    A = torch.zeros((16, 4), device="cuda")
    bc = torch.zeros((2, 8, 1, 4), device="cuda")
    for err, text, call in [
        (ValueError, "CUDA", lambda: layer.short_conv_fwd(x.cpu(), w)),
        (ValueError, "dimensions", lambda: layer.short_conv_fwd(x[0], w)),
        (ValueError, "w must", lambda: layer.short_conv_fwd(x, w[:, :8])),
        (TypeError, "w must", lambda: layer.short_conv_fwd(x, w.bfloat16())),
        (ValueError, "act", lambda: layer.short_conv_fwd(x, w, act="gelu")),
        (ValueError, "contiguous", lambda: layer.short_conv_fwd(x.transpose(1, 2).contiguous().transpose(1, 2), w)),
        (ValueError, "one stride", lambda: layer.short_conv_fwd(torch.zeros((2, 9, 16), device="cuda")[:, :8], w)),
        (ValueError, "one stride", lambda: layer.short_conv_fwd(x[:, :1].expand(2, 8, 16), w)),
        (ValueError, "overlap", lambda: layer.short_conv_fwd(x[:1, :1].expand(2, 8, 16), w)),
        (TypeError, "lens", lambda: layer.short_conv_fwd(x, w, lens=torch.zeros(2, device="cuda"))),
        (abi.TTTError, "overlaps", lambda: layer.short_conv_fwd(x, w, out=x)),
        (abi.TTTError, "width", lambda: layer.short_conv_fwd(x, torch.zeros((9, 16), device="cuda"))),
        (ValueError, "state", lambda: layer.short_conv_step(x[:, 0], w, x)),
        (ValueError, "dy", lambda: layer.short_conv_bwd(x, w, x[:, :4])),
        (ValueError, "one of", lambda: layer.head_norm_rope_fwd(None, None)),
        (ValueError, "k must", lambda: layer.head_norm_rope_fwd(x[:, :, None], x[:, :4, None])),
        (ValueError, "norm", lambda: layer.head_norm_rope_fwd(x[:, :, None], None, norm="layer")),
        (abi.TTTError, "rot", lambda: layer.head_norm_rope_fwd(x[:, :, None], None, inv_freq=w[0, :9])),
        (ValueError, "dk", lambda: layer.head_norm_rope_bwd(x[:, :, None], x[:, :, None], None, x[:, None], None, None)),
        (ValueError, "Cm must", lambda: layer.selective_scan_fwd(x, x, A, bc, bc[:, :4])),
        (ValueError, "A must", lambda: layer.selective_scan_fwd(x, x, A[0], bc, bc)),
        (ValueError, "Bm must", lambda: layer.selective_scan_fwd(x, x, A, bc[:, :, 0], bc)),
        (abi.TTTError, "multiple of G", lambda: layer.selective_scan_fwd(
            x, x, A, bc.expand(2, 8, 3, 4).contiguous(), bc.expand(2, 8, 3, 4).contiguous())),
        (TypeError, "z must", lambda: layer.selective_scan_fwd(x, x, A, bc, bc, z=x.bfloat16())),
        (ValueError, "state", lambda: layer.selective_scan_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0], A)),
    ]:
        with pytest.raises(err) as ei:
            call()
        assert text in str(ei.value), (text, str(ei.value))
