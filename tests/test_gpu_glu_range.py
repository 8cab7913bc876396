"""The gated feed-forward at the ends of its range: gates that overflow to infinity."""
import pytest

pytestmark = pytest.mark.gpu


def _pkg():
    import attention_qkv_gemm_gb300 as pkg
    return pkg


def _stream():
    import torch
    return torch.cuda.current_stream().cuda_stream


# the few-token kernel, lone CTAs, CTAs that share a sum, pairs of narrow and of wide tiles
@pytest.mark.parametrize("tokens,d,f", [(3, 64, 64), (40, 64, 64), (40, 4096, 64), (7824, 216, 304), (6763, 136, 584)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_infinite_gates(tokens, d, f, act):
    """Gates of +-3e38 x 2, which overflow fp32, beside u = 2: act(inf) = inf; act(-inf) = -inf times 0,
    no number; the other rows' gates are 0."""
    import torch
    pkg = _pkg()
    inf = float("inf")
    x = torch.zeros(tokens, d, device="cuda").bfloat16()
    x[:, 1] = 1.0
    x[0, 0], x[1, 0], x[tokens - 1, 0] = 3e38, -3e38, 3e38
    wg, wu = torch.zeros(f, d, device="cuda").bfloat16(), torch.zeros(f, d, device="cuda").bfloat16()
    wg[:, 0], wu[:, 1] = 2.0, 2.0
    h = torch.full((tokens, f), 7.0, device="cuda").bfloat16()
    g = pkg.tfl_glu_create(d, f, pkg.TFL_BF16, pkg.TFL_BF16, {"silu": pkg.TFL_ACT_SILU, "gelu": pkg.TFL_ACT_GELU}[act])
    pkg.tfl_glu_forward(g, tokens, x.data_ptr(), None, wg.data_ptr(), None, wu.data_ptr(), None, h.data_ptr(), _stream())
    assert pkg.tfl_glu_status(g, _stream()) == 0
    pkg.tfl_glu_destroy(g)
    assert (h[0] == inf).all() and h[1].isnan().all() and (h[tokens - 1] == inf).all()
    assert (h[2:tokens - 1] == 0).all()
