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
