"""CPU checks of the token-mixer operators: the oracle's gradients against central differences,
and the library's refusals (nothing here reaches the CUDA driver)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import mixer_oracle as M
from test_weight_layers_ttt_b200 import abi, layer
from test_weight_layers_ttt_b200 import build as tbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    tbuild.build()
    return abi.lib()


# ----------------------------------------------------------------------------- the oracle
def differences(loss, x, eps=1e-6):
    """Central differences of a scalar function in every element of x (changed in place)."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + eps
        hi = loss()
        x[i] = old - eps
        lo = loss()
        x[i] = old
        g[i] = (hi - lo) / (2 * eps)
    return g


# A central difference of a smooth function is off by about eps^2 of its third derivative plus
# the rounding 2^-53 |loss| / eps: below 1e-8 for losses around 10.
FD_TOL = 1e-7


@pytest.mark.parametrize("act,lens", [(True, None), (False, [4, 0])])
def test_short_conv_oracle_gradients(act, lens):
    rng = np.random.default_rng(1)
    x, w, bias = rng.normal(size=(2, 5, 3)), rng.normal(size=(3, 3)), rng.normal(size=3)
    st, dy, ds = rng.normal(size=(2, 2, 3)), rng.normal(size=(2, 5, 3)), rng.normal(size=(2, 2, 3))

    def loss():
        y, new = M.short_conv(x, w, bias, act, st, lens)
        return (y * dy).sum() + (new * ds).sum()

    got = M.short_conv_backward(x, w, dy, bias, act, st, lens, ds)
    for g, v in zip(got, (x, w, bias, st)):
        assert np.abs(g - differences(loss, v)).max() < FD_TOL


@pytest.mark.parametrize("norm,pairs,weight", [("l2", "halves", True), ("rms", "interleaved", True),
                                               (None, "halves", False)])
def test_head_norm_rope_oracle_gradients(norm, pairs, weight):
    rng = np.random.default_rng(2)
    x, dout = rng.normal(size=(2, 3, 2, 7)), rng.normal(size=(2, 2, 3, 7))
    w = rng.normal(size=7) if weight else None
    kw = dict(norm=norm, eps=1e-3, inv_freq=np.array([1.0, 0.3]), pairs=pairs,
              positions=np.array([[0, 1, 2], [50, 3, 9]]))

    def loss():
        return (M.head_norm_rope(x, w, **kw) * dout).sum()

    dx, dw = M.head_norm_rope_backward(x, dout, w, **kw)
    assert np.abs(dx - differences(loss, x)).max() < FD_TOL
    if weight:
        assert np.abs(dw - differences(loss, w)).max() < FD_TOL


@pytest.mark.parametrize("softplus,gate,lens", [(True, True, None), (False, False, [3, 0]),
                                                (True, True, [4, 2])])
def test_selective_scan_oracle_gradients(softplus, gate, lens):
    rng = np.random.default_rng(3)
    B, N, D, S, G = 2, 4, 4, 3, 2
    v = {"u": rng.normal(size=(B, N, D)), "dt": rng.uniform(0.1, 1, size=(B, N, D)),
         "A": -rng.uniform(0.2, 2, size=(D, S)), "Bm": rng.normal(size=(B, N, G, S)),
         "Cm": rng.normal(size=(B, N, G, S)), "D": rng.normal(size=D), "dt_bias": rng.normal(size=D) * 0.1,
         "state": rng.normal(size=(B, D, S)), "z": rng.normal(size=(B, N, D)) if gate else None}
    dy, ds = rng.normal(size=(B, N, D)), rng.normal(size=(B, D, S))

    def loss():
        y, hs = M.selective_scan(**v, softplus=softplus, lens=lens)
        return (y * dy).sum() + (hs[:, -1] * ds).sum()

    got = M.selective_scan_backward(**v, dy=dy, softplus=softplus, lens=lens, dstate=ds)
    names = {"u": "du", "dt": "ddt", "A": "dA", "Bm": "dB", "Cm": "dC", "D": "dD", "z": "dz",
             "dt_bias": "ddt_bias", "state": "dstate"}
    for n, g in names.items():
        if v[n] is not None:
            assert np.abs(got[g] - differences(loss, v[n])).max() < FD_TOL, n


def test_scan_with_one_state_and_no_decay_is_a_running_sum():
    rng = np.random.default_rng(4)
    u = rng.normal(size=(1, 6, 2))
    one = np.ones((1, 6, 1, 1))
    y, _ = M.selective_scan(u, np.ones((1, 6, 2)), np.zeros((2, 1)), one, one, softplus=False)
    assert np.allclose(y, np.cumsum(u, axis=1), atol=1e-14)


# ----------------------------------------------------------------------------- refusals
P = [1 << (20 + i) for i in range(24)]     # distinct, aligned, far apart; never dereferenced


def refused(status, fn, *args, text=None):
    with pytest.raises(abi.TTTError) as ei:
        fn(*args, stream=0)
    assert ei.value.status == status, str(ei.value)
    if text:
        assert text in str(ei.value)


def conv_desc(**kw):
    return abi.ttt_conv_desc(**{**dict(B=2, N=16, D=32, width=4, dtype=abi.TTT_DTYPE_BF16, act=1), **kw})


def heads_desc(**kw):
    return abi.ttt_heads_desc(**{**dict(B=2, N=16, Hq=2, Hk=2, Hv=2, h=16, dtype=abi.TTT_DTYPE_BF16,
                                        norm=2, rot=16, pairs=0, eps=1e-6), **kw})


def scan_desc(**kw):
    return abi.ttt_scan_desc(**{**dict(B=2, N=16, D=32, S=16, G=1, dtype=abi.TTT_DTYPE_BF16, softplus=1), **kw})


def test_descriptors_match_the_header():
    assert ctypes.sizeof(abi.ttt_conv_desc) == 6 * 4 + 8
    assert ctypes.sizeof(abi.ttt_heads_desc) == 12 * 4 + 3 * 8
    assert ctypes.sizeof(abi.ttt_scan_desc) == 8 * 4 + 5 * 8


BAD, NOT = abi.TTT_ERR_INVALID_ARG, abi.TTT_ERR_UNSUPPORTED


@pytest.mark.parametrize("field,value,status", [
    ("B", -1, BAD), ("N", -1, BAD), ("D", 0, BAD), ("dtype", 2, BAD), ("act", 2, BAD), ("width", 0, BAD),
    ("x_row", 31, BAD), ("x_row", -32, BAD), ("width", 1, NOT), ("width", 9, NOT), ("B", 65536, NOT),
    ("N", (1 << 22) + 1, NOT), ("D", (1 << 20) + 1, NOT)])
def test_short_conv_refuses_descriptors(field, value, status):
    d = conv_desc(**{field: value})
    refused(status, abi.ttt_short_conv_fwd, d, P[0], P[1], P[2], None, None, P[3], P[4])
    refused(status, abi.ttt_short_conv_bwd, d, P[0], P[1], P[2], None, None, P[3], None, P[4], P[5],
            P[6], None, P[7], 1 << 19)
    assert abi.ttt_short_conv_bwd_workspace_bytes(d) == 0


def test_short_conv_refuses_buffers():
    d = conv_desc()
    fwd, bwd, step = abi.ttt_short_conv_fwd, abi.ttt_short_conv_bwd, abi.ttt_short_conv_step
    refused(BAD, fwd, d, None, P[1], None, None, None, P[3], None)
    refused(BAD, fwd, d, P[0], None, None, None, None, P[3], None)
    refused(BAD, fwd, d, P[0] + 1, P[1], None, None, None, P[3], None, text="aligned")
    refused(BAD, fwd, d, P[0], P[1] + 2, None, None, None, P[3], None, text="aligned")
    refused(BAD, fwd, d, P[0], P[1], None, None, None, P[0], None, text="overlaps")
    refused(BAD, fwd, d, P[0], P[1], None, None, None, P[0] + 2046, None, text="overlaps")
    # the rows of a wider projection reach further than the dense ones
    refused(BAD, fwd, conv_desc(x_row=64), P[0], P[1], None, None, None, P[0] + 3900, None, text="overlaps")
    refused(BAD, fwd, d, P[0], P[1], None, P[5], None, P[3], P[5] + 64, text="overlaps")
    refused(BAD, step, d, P[0], P[1], None, P[2], P[3], text="N = 1")
    refused(BAD, step, conv_desc(N=1), P[0], P[1], None, None, P[3])
    refused(BAD, step, conv_desc(N=1), P[0], P[1], None, P[2], P[2], text="overlaps")
    need = abi.ttt_short_conv_bwd_workspace_bytes(d)
    assert need > 0
    args = (d, P[0], P[1], P[2], None, None, P[3], None, P[4], P[5], P[6], None)
    refused(abi.TTT_ERR_WORKSPACE, bwd, *args, P[7], need - 1)
    refused(abi.TTT_ERR_WORKSPACE, bwd, *args, P[7] + 64, need)
    refused(abi.TTT_ERR_WORKSPACE, bwd, *args, None, 0)
    refused(BAD, bwd, d, P[0], P[1], P[2], None, None, P[3], None, P[3], P[5], P[6], None, P[7], need,
            text="overlaps")
    refused(BAD, bwd, d, P[0], P[1], P[2], None, None, P[3], None, P[4], None, P[6], None, P[7], need)


@pytest.mark.parametrize("field,value,status", [
    ("B", -1, BAD), ("N", -1, BAD), ("Hq", -1, BAD), ("h", 0, BAD), ("dtype", 7, BAD), ("norm", 3, BAD),
    ("pairs", 2, BAD), ("rot", 3, BAD), ("rot", 18, BAD), ("rot", -2, BAD), ("eps", 0.0, BAD),
    ("eps", -1.0, BAD), ("eps", float("nan"), BAD), ("pos0", -1, BAD), ("q_row", 31, BAD),
    ("h", 514, NOT), ("Hv", 65536, NOT), ("N", (1 << 22) + 1, NOT)])
def test_heads_refuse_descriptors(field, value, status):
    d = heads_desc(**{field: value})
    refused(status, abi.ttt_head_norm_rope_fwd, d, P[0], P[1], P[2], None, None, P[3], None, P[4], P[5], P[6])
    refused(status, abi.ttt_head_norm_rope_bwd, d, P[0], P[1], None, None, P[3], None, P[4], P[5], P[6],
            P[7], P[8], P[9], None, None, None, 0)
    assert abi.ttt_head_norm_rope_bwd_workspace_bytes(d) == 0


def test_heads_refuse_buffers():
    d = heads_desc()
    fwd, bwd = abi.ttt_head_norm_rope_fwd, abi.ttt_head_norm_rope_bwd
    refused(BAD, fwd, d, P[0], P[1], None, None, None, P[3], None, P[4], P[5], P[6])       # v missing
    refused(BAD, fwd, d, P[0], P[1], P[2], None, None, P[3], None, P[4], None, P[6])       # k_out missing
    refused(BAD, fwd, d, P[0], P[1], P[2], None, None, None, None, P[4], P[5], P[6], text="inv_freq")
    refused(BAD, fwd, d, P[0], P[1], P[2], None, None, P[3], None, P[0], P[5], P[6], text="overlaps")
    refused(BAD, fwd, d, P[0], P[1], P[2], None, None, P[3], None, P[4], P[4], P[6], text="overlaps")
    refused(BAD, fwd, d, P[0], P[1] + 1, P[2], None, None, P[3], None, P[4], P[5], P[6], text="aligned")
    tail = (P[4], P[5], P[6], P[7], P[8], P[9])
    refused(BAD, bwd, d, P[0], P[1], None, None, P[3], None, *tail, P[10], None, P[11], 1 << 18,
            text="needs its weight")
    refused(abi.TTT_ERR_WORKSPACE, bwd, d, P[0], P[1], P[2], None, P[3], None, *tail, P[10], None, None, 0)


@pytest.mark.parametrize("field,value,status", [
    ("B", -1, BAD), ("N", -1, BAD), ("D", 0, BAD), ("S", 0, BAD), ("G", 0, BAD), ("G", 3, BAD),
    ("dtype", 2, BAD), ("softplus", 2, BAD), ("reserved", 1, BAD), ("u_row", 16, BAD), ("b_row", 15, BAD),
    ("S", 65, NOT), ("D", (1 << 20) + 32, NOT), ("B", 65536, NOT)])
def test_scan_refuses_descriptors(field, value, status):
    d = scan_desc(**{field: value})
    ins = (P[0], P[1], P[2], P[3], P[4], None, None, None, None, None)
    refused(status, abi.ttt_selective_scan_fwd, d, *ins, P[5], P[6], P[7], 1 << 19)
    refused(status, abi.ttt_selective_scan_bwd, d, *ins, P[5], None, P[6], P[7], P[8], P[9], P[10], None,
            None, None, None, P[11], 1 << 19)
    assert abi.ttt_selective_scan_workspace_bytes(d, 0) == 0
    assert abi.ttt_selective_scan_workspace_bytes(d, 1) == 0


def test_scan_refuses_buffers():
    d = scan_desc()
    fwd, bwd, step = abi.ttt_selective_scan_fwd, abi.ttt_selective_scan_bwd, abi.ttt_selective_scan_step
    none = (None,) * 5
    refused(BAD, fwd, d, None, P[1], P[2], P[3], P[4], *none, P[5], P[6], None, 0)
    refused(BAD, fwd, d, P[0], P[1], None, P[3], P[4], *none, P[5], P[6], None, 0)
    refused(BAD, fwd, d, P[0], P[1], P[2], P[3], P[4], *none, P[0], P[6], None, 0, text="overlaps")
    refused(BAD, fwd, d, P[0], P[1], P[2] + 2, P[3], P[4], *none, P[5], P[6], None, 0, text="aligned")
    refused(BAD, fwd, d, P[0], P[1], P[2], P[3], P[4], None, None, None, P[6] + 4, None, P[5], P[6], None, 0,
            text="overlaps")
    # few channels and a long sequence: split over the time axis, in a workspace
    long = scan_desc(B=1, N=4096)
    need = abi.ttt_selective_scan_workspace_bytes(long, 0)
    assert need > 0
    refused(abi.TTT_ERR_WORKSPACE, fwd, long, P[0], P[1], P[2], P[3], P[4], *none, P[5], P[6], P[7], need - 1)
    # many channels: one pass, no workspace
    assert abi.ttt_selective_scan_workspace_bytes(scan_desc(B=64, D=4096, N=4096), 0) == 0
    refused(BAD, step, d, P[0], P[1], P[2], P[3], P[4], None, None, None, P[5], P[6], text="N = 1")
    refused(BAD, step, scan_desc(N=1), P[0], P[1], P[2], P[3], P[4], None, None, None, None, P[6])
    need = abi.ttt_selective_scan_workspace_bytes(d, 1)
    outs = (P[6], P[7], P[8], P[9], P[10], None)
    refused(BAD, bwd, d, P[0], P[1], P[2], P[3], P[4], None, P[12], None, None, None, P[5], None, *outs,
            None, None, None, P[11], need, text="z and dz")
    refused(abi.TTT_ERR_WORKSPACE, bwd, d, P[0], P[1], P[2], P[3], P[4], *none, P[5], None, *outs, None,
            None, None, P[11], need - 1)


def test_empty_calls_enqueue_nothing():
    abi.ttt_short_conv_fwd(conv_desc(B=0), None, P[0], None, None, None, None, None, stream=0)
    abi.ttt_short_conv_fwd(conv_desc(N=0), None, P[0], None, None, None, None, None, stream=0)
    abi.ttt_head_norm_rope_fwd(heads_desc(N=0), *(None,) * 10, stream=0)
    abi.ttt_head_norm_rope_fwd(heads_desc(Hq=0, Hk=0, Hv=0), *(None,) * 10, stream=0)
    abi.ttt_selective_scan_fwd(scan_desc(B=0), *(None,) * 13, 0, stream=0)
    abi.ttt_selective_scan_fwd(scan_desc(N=0), None, None, P[0], *(None,) * 10, 0, stream=0)


def test_backward_workspaces_grow_with_guards():
    sizes = {}
    for flags in (0, abi.TTT_CHECK_GUARDS):
        abi.ttt_set_debug_checks(flags)
        try:
            sizes[flags] = (abi.ttt_short_conv_bwd_workspace_bytes(conv_desc()),
                            abi.ttt_head_norm_rope_bwd_workspace_bytes(heads_desc()),
                            abi.ttt_selective_scan_workspace_bytes(scan_desc(), 1))
        finally:
            abi.ttt_set_debug_checks(0)
    assert all(g >= n + 512 for n, g in zip(sizes[0], sizes[1]))


# ----------------------------------------------------------------------------- strides
def stride_between_tokens(t, lead, width):
    """What the descriptor says of ``t``: checked against the address of every token's first
    and last element."""
    row = layer._rows(t, "t", lead, width, t.dtype, t.device)
    n = int(np.prod(width))
    r = row or n
    last = tuple(w - 1 for w in width)
    for i, at in enumerate(np.ndindex(*lead)):
        assert t[at + (0,) * len(width)].data_ptr() == t.data_ptr() + i * r * t.element_size()
        assert t[at + last].data_ptr() == t.data_ptr() + (i * r + n - 1) * t.element_size()
    return row


@pytest.mark.parametrize("make,lead,width,row", [
    (lambda z: z(2, 5, 6), (2, 5), (6,), 0),
    (lambda z: z(2, 5, 16)[..., 3:9], (2, 5), (6,), 16),
    (lambda z: z(2, 5, 16)[..., 4:12].unflatten(-1, (2, 4)), (2, 5), (2, 4), 16),
    (lambda z: z(3, 1, 16)[..., :6], (3, 1), (6,), 16),
    (lambda z: z(1, 5, 16)[..., :6], (1, 5), (6,), 16),
    (lambda z: z(1, 9, 6)[:, :5], (1, 5), (6,), 0),
    (lambda z: z(1, 10, 6)[:, ::2], (1, 5), (6,), 12),
    (lambda z: z(4, 7, 6)[:, 3], (4,), (6,), 42),
    (lambda z: z(4, 7, 12)[:, 3, 2:8].unflatten(-1, (3, 2)), (4,), (3, 2), 84),
    (lambda z: z(1, 1, 6).expand(1, 1, 6), (1, 1), (6,), 0),
    (lambda z: z(2, 5, 3, 8)[..., 1:2, :], (2, 5), (1, 8), 24),
])
def test_row_strides_reach_every_token(make, lead, width, row):
    assert stride_between_tokens(make(torch.zeros), lead, width) == row


@pytest.mark.parametrize("make,lead,width,text", [
    (lambda z: z(2, 6, 5).transpose(1, 2), (2, 5), (6,), "contiguous"),
    (lambda z: z(2, 5, 12)[..., ::2], (2, 5), (6,), "contiguous"),
    (lambda z: z(2, 5, 4, 2).transpose(2, 3), (2, 5), (2, 4), "contiguous"),
    (lambda z: z(2, 5, 3, 8)[..., :6], (2, 5), (3, 6), "contiguous"),
    (lambda z: z(2, 9, 6)[:, :5], (2, 5), (6,), "one stride"),
    (lambda z: z(5, 2, 6).transpose(0, 1), (2, 5), (6,), "one stride"),
    (lambda z: z(1, 5, 6).expand(2, 5, 6), (2, 5), (6,), "one stride"),
    (lambda z: z(2, 1, 6).expand(2, 5, 6), (2, 5), (6,), "one stride"),
    (lambda z: z(1, 1, 6).expand(1, 5, 6), (1, 5), (6,), "overlap"),
    (lambda z: z(1, 1, 6).expand(2, 5, 6), (2, 5), (6,), "overlap"),
    (lambda z: z(1, 6).expand(4, 6), (4,), (6,), "overlap"),
    (lambda z: z(64).as_strided((1, 5, 6), (30, 5, 1)), (1, 5), (6,), "overlap"),
    (lambda z: z(2, 5, 6), (2, 4), (6,), "must be"),
])
def test_other_strides_are_refused(make, lead, width, text):
    t = make(torch.zeros)
    with pytest.raises(ValueError) as ei:
        layer._rows(t, "t", lead, width, t.dtype, t.device)
    assert text in str(ei.value)


def test_sizes_beyond_32_bits_are_refused():
    big, f32 = 2**32 + 1, torch.float32
    x = torch.empty(1, big, 1, dtype=torch.bfloat16, device="meta")
    w = torch.empty(4, 1, device="meta")
    with pytest.raises(ValueError, match="below 2"):
        layer._conv_desc(x, w, None, "silu", None, None, (1, big))
    bc = torch.empty(1, big, 1, 1, dtype=torch.bfloat16, device="meta")
    A = torch.empty(1, 1, dtype=f32, device="meta")
    with pytest.raises(ValueError, match="below 2"):
        layer._scan_desc(x, x, A, bc, bc, None, None, None, True, None, None, (1, big))
    assert layer._sizes(0, 2**31 - 1) == (0, 2**31 - 1)


def test_a_workspace_must_span_its_elements():
    cpu = torch.device("cpu")
    ws = torch.empty(64, dtype=torch.uint8)
    assert layer._scratch(ws, 64, cpu) is ws
    with pytest.raises(ValueError, match="contiguous"):
        layer._scratch(ws[:1].expand(64), 64, cpu)


@pytest.mark.parametrize("pos0", [2**31, 2**32 + 5, -1, -2**32 + 5])
def test_positions_beyond_32_bits_are_refused(pos0):
    """In front of every other check, for the descriptor's 32 bits would wrap them."""
    q = torch.empty(1, 2, 1, 8)
    for call in (lambda: layer.head_norm_rope_fwd(q, None, pos0=pos0),
                 lambda: layer.head_norm_rope_bwd(q, None, None, q, None, None, pos0=pos0)):
        with pytest.raises(ValueError, match="pos0"):
            call()
    with pytest.raises(ValueError, match="CUDA"):
        layer.head_norm_rope_fwd(q, None, pos0=2**31 - 1)
