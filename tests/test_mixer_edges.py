"""Values at the edges of the token-mixer operators' range: infinities and the largest decays next
to padded tokens, tiny norms, and elements that an operator passes on untouched."""
import numpy as np
import pytest
import torch

from oracle import mixer_oracle as M
from test_weight_layers_ttt_b200 import layer

from gpu_helpers import dev, host, torch_dtype
from test_mixer_gpu import conv_case, near, rand, scan_case, scan_roundings

pytestmark = pytest.mark.gpu

INF = float("inf")


# ----------------------------------------------------------------------------- convolution
@pytest.mark.parametrize("dtype,D,width", [("bf16", 48, 4), ("fp32", 33, 8), ("bf16", 7, 2)])
@pytest.mark.parametrize("act", ["silu", None])
def test_short_conv_gradients_behind_an_infinite_last_token_are_zeros(dtype, D, width, act):
    lens, N = [17, 40, 0, 41], 41
    _, _, _, _, xg, wg, g, rng = conv_case(dtype, 4, N, D, width, act, True, lens, 0, seed=31)
    dy = dev(rand(rng, 4, N, D, dtype=dtype), torch_dtype(dtype))
    ref = layer.short_conv_bwd(xg, wg, dy, **g)
    xg[0, 16, 3] = INF
    xg[1, 39, 5] = -INF
    got = layer.short_conv_bwd(xg, wg, dy, **g)
    for b, n in enumerate(lens):
        assert float(got[0][b, n:].abs().sum()) == 0.0
    # an infinite input reaches its own channel's gradients of the tokens up to it, no others
    same = torch.ones_like(got[0], dtype=torch.bool)
    same[0, 17 - width:17, 3] = same[1, 40 - width:40, 5] = False
    assert torch.equal(got[0][same], ref[0][same])


def test_short_conv_gradients_behind_the_end_are_zeros_for_infinite_weights():
    _, _, _, _, xg, wg, g, rng = conv_case("fp32", 1, 20, 16, 4, "silu", False, [11], 0, seed=32)
    wg[1, 2] = INF
    got = layer.short_conv_bwd(xg, wg, dev(rand(rng, 1, 20, 16)), **g)
    assert float(got[0][0, 11:].abs().sum()) == 0.0


# ----------------------------------------------------------------------------- heads
@pytest.mark.parametrize("dtype,h,rot", [("fp32", 64, 32), ("fp32", 33, 20), ("bf16", 128, 128), ("bf16", 81, 0)])
@pytest.mark.parametrize("norm", ["l2", "rms"])
@pytest.mark.parametrize("weight", [True, False])
def test_head_norm_backward_of_tiny_rows_with_a_small_eps(dtype, h, rot, norm, weight):
    """dx = r (g - n <g, n>) with n = x r, r up to eps^(-1/2): in range where r^3 is not."""
    eps, td = float(np.float32(1e-30)), torch_dtype(dtype)
    rng = np.random.default_rng(33)
    x, do = rand(rng, 1, 4, 3, h, dtype=dtype), rand(rng, 1, 3, 4, h, dtype=dtype)
    x[0, 1, 1] = 0.0
    x[0, 2] = host(dev(x[0, 2] * 1e-15, td))        # of eps' size
    x[0, 3] = host(dev(x[0, 3] * 1e-19, td))        # far below it
    w = rand(rng, h) + 1 if weight else None
    inv = (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32) if rot else None
    kw = dict(norm=norm, eps=eps, inv_freq=None if inv is None else dev(inv))
    got = layer.head_norm_rope_bwd(dev(x, td), None, None, dev(do, td), None, None,
                                   wq=None if w is None else dev(w), **kw)
    pos = np.arange(4)[None]
    dx, dw = M.head_norm_rope_backward(x, do, w, norm, eps, inv, pos)
    # the terms of a row's dx are at most r sqrt(h) max |g| (Cauchy-Schwarz, either norm), each with
    # two sums over h and some roundings; |R^T dout| <= 2 max |dout|
    sq = (x * x).sum(-1)
    r = 1 / np.sqrt((sq if norm == "l2" else sq / h) + eps)
    g = 2 * np.abs(do).max() * (1.0 if w is None else np.abs(w).max())
    for t in range(4):
        near(got[0][:, t], dx[:, t], 4 * h + 64, f"token {t}", terms=np.sqrt(h) * g * r[0, t].max())
    if weight:
        near(got[3], dw, 12 + h + 64, "dw", terms=12 * np.sqrt(h) * g)


@pytest.mark.parametrize("dtype,h,rot,pairs", [("fp32", 64, 64, "halves"), ("bf16", 80, 40, "interleaved"),
                                               ("fp32", 7, 0, "halves")])
def test_head_gradients_without_a_norm_do_not_depend_on_the_input(dtype, h, rot, pairs):
    td = torch_dtype(dtype)
    rng = np.random.default_rng(34)
    x, do = rand(rng, 2, 5, 2, h, dtype=dtype), rand(rng, 2, 2, 5, h, dtype=dtype)
    inv = dev((10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)) if rot else None
    xg, dg = dev(x, td), dev(do, td)
    ref = layer.head_norm_rope_bwd(xg, None, None, dg, None, None, norm=None, inv_freq=inv, pairs=pairs)[0]
    xg[0, 1, 1, 2], xg[1, 4, 0, 5], xg[1, 0, 0] = INF, float("nan"), -INF
    got = layer.head_norm_rope_bwd(xg, None, None, dg, None, None, norm=None, inv_freq=inv, pairs=pairs)[0]
    assert torch.equal(got, ref)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("h,rot", [(64, 32), (80, 20), (96, 0), (33, 20), (128, 6)])
@pytest.mark.parametrize("pairs", ["halves", "interleaved"])
def test_elements_behind_the_rotation_stay_apart(dtype, h, rot, pairs):
    """Without a norm an element behind the rotated ones is passed on alone, forward and backward:
    an infinite neighbour does not reach it."""
    td = torch_dtype(dtype)
    rng = np.random.default_rng(35)
    x = dev(rand(rng, 2, 3, 2, h, dtype=dtype), td)
    inv = dev((10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)) if rot else None
    kw = dict(norm=None, inv_freq=inv, pairs=pairs, pos0=5)
    for at in (rot, rot + (h - rot) // 2, h - 1):
        bad = x.clone()
        bad[1, 2, 0, at] = INF
        want = layer.head_norm_rope_fwd(x, None, **kw)[0]
        want[1, 0, 2, at] = INF
        assert torch.equal(layer.head_norm_rope_fwd(bad, None, **kw)[0], want)
        do = x.transpose(1, 2).contiguous()
        want = layer.head_norm_rope_bwd(x, None, None, do, None, None, **kw)[0]
        want[1, 2, 0, at] = INF
        do[1, 0, 2, at] = INF
        assert torch.equal(layer.head_norm_rope_bwd(x, None, None, do, None, None, **kw)[0], want)


# ----------------------------------------------------------------------------- selective scan
@pytest.mark.parametrize("value", [-3e38, -INF])
@pytest.mark.parametrize("N,lens", [(37, None), (37, [37, 20]), (300, [299, 45]), (300, [0, 1])])
def test_a_decay_beyond_the_range_of_its_exponent_forgets_at_once(value, N, lens):
    """exp(delta A) = 0 for each of a sequence's tokens; the padded tokens of a tile and whole pieces
    behind the end step by 0."""
    S, D = 16, 24
    h, g, rng = scan_case("fp32", 2, N, D, S, 1, True, True, lens, True, 0, seed=36)
    dy, ds = rand(rng, 2, N, D), rand(rng, 2, D, S)
    h["A"][3, 5] = h["A"][10] = -1e30               # as good as infinite: delta > 1e-3 here
    g["A"][3, 5] = g["A"][10] = value
    y, st = layer.selective_scan_fwd(**g)
    ry, hs = M.selective_scan(**h)
    near(y, ry, scan_roundings(N, S), "y")
    near(st, hs[:, -1], scan_roundings(N, S), "state")
    if value != -INF:                               # the gradient of delta has the factor A
        got = layer.selective_scan_bwd(**g, dy=dev(dy), dstate=dev(ds))
        ref = M.selective_scan_backward(**h, dy=dy, dstate=ds)
        for t, name in zip(got, ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate")):
            near(t, ref[name], 2 * scan_roundings(N, S) + 2 * N + D, name)


def test_a_step_takes_a_decay_beyond_the_range_of_its_exponent():
    h, g, _ = scan_case("fp32", 3, 1, 10, 16, 1, True, True, None, True, 0, seed=37)
    h["A"][2] = -1e30
    g["A"][2] = -3e38
    ry, hs = M.selective_scan(**h)
    g.pop("softplus")
    one = {k: v[:, 0].contiguous() if k in ("u", "dt", "z", "Bm", "Cm") else v for k, v in g.items()}
    near(layer.selective_scan_step(**one), ry[:, 0], scan_roundings(1, 16))
    near(one["state"], hs[:, -1], scan_roundings(1, 16))
    # a step of zero is no decay
    g["dt"].zero_(), g["dt_bias"].zero_()
    one["dt"], before = one["dt"].zero_(), one["state"].clone()
    layer.selective_scan_step(**one, softplus=False)
    assert torch.equal(one["state"], before)


@pytest.mark.parametrize("dtype,N,n,D,S", [("fp32", 60, 45, 40, 16), ("bf16", 300, 130, 64, 16),
                                           ("fp32", 30, 30, 18, 33), ("bf16", 300, 300, 9, 8)])
def test_an_infinite_last_input_reaches_no_gradient_in_front_of_it(dtype, N, n, D, S):
    """The last token's u is in its own state, output and gradients only: du (which is without u) and
    what other tokens and channels have stay what they are. Its own channel's dA is a sum that it
    may spoil, as it does those of dD and ddt_bias."""
    _, g, rng = scan_case(dtype, 2, N, D, S, 1, True, True, [n, max(n - 9, 0)], True, 0, seed=38)
    dy = dev(rand(rng, 2, N, D, dtype=dtype), torch_dtype(dtype))
    ref = layer.selective_scan_bwd(**g, dy=dy)
    g["u"][0, n - 1, 4] = INF
    got = layer.selective_scan_bwd(**g, dy=dy)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[8], ref[8])
    for i in (1, 3, 4, 6):                           # ddt, dB, dC, dz of all other tokens
        ref[i][0, n - 1], got[i][0, n - 1] = 0, 0
        assert torch.equal(got[i], ref[i])
    for i in (2, 5, 7):                              # dA, dD, ddt_bias of all other channels
        ref[i][4], got[i][4] = 0, 0
        assert torch.equal(got[i], ref[i])
