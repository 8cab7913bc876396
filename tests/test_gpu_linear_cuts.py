"""The linear layer's weight gradient is cut by the call's tokens, not by what else its handle has room for."""
import pytest

import attention_qkv_gemm_gb300 as pkg
from tests.test_gpu_linear import _backward, _check_backward

pytestmark = pytest.mark.gpu


# (the first four take more shares of the tokens than the larger calls that the other handles have room for would)
@pytest.mark.parametrize("tokens,k,n,rooms", [(37343, 1032, 136, (8997,)), (28722, 400, 344, (158478,)), (23936, 80, 1144, (40673,)),
                                              (50544, 704, 736, (18833, 200000)), (6001, 128, 136, (700, 60000)),
                                              (700, 64, 72, (5000, 100000))])
def test_the_same_inputs_give_the_same_bits_in_any_handle(tokens, k, n, rooms):
    import torch
    own = _backward(tokens, k, n, "bf16", "gelu", "bf16", room=0)
    _check_backward(*own, "bf16", "gelu")
    for room in rooms:
        other = _backward(tokens, k, n, "bf16", "gelu", "bf16", room=room)[4]
        for name, want in own[4].items():
            assert torch.equal(other[name], want), (name, room)


def test_one_handle_serves_every_number_of_tokens_as_its_own():
    """Calls of all sizes in turn through one handle, each against a handle of its size."""
    import torch
    k, n, most = 120, 224, 50000
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, dy = torch.randn(most, k, generator=gen, device="cuda").half(), torch.randn(most, n, generator=gen, device="cuda").half()
    w = torch.randn(n, k, generator=gen, device="cuda").half()
    stream = torch.cuda.current_stream().cuda_stream
    P = lambda t: t.data_ptr()  # noqa: E731

    def run(op, tokens):
        dx, dw, db = torch.empty(tokens, k, device="cuda").half(), torch.empty_like(w), torch.empty(n, device="cuda")
        pkg.tfl_linear_backward(op, tokens, P(x), P(w), None, P(dy), P(dx), P(dw), P(db), stream)
        assert pkg.tfl_linear_status(op, stream) == 0
        return dx, dw, db

    make = lambda tokens: pkg.tfl_linear_create(k, n, pkg.TFL_F16, pkg.TFL_F16, pkg.TFL_ACT_NONE, pkg.TFL_F16, tokens)  # noqa: E731
    large = make(most)
    for tokens in (50000, 1, 63, 449, 512, 767, 1000, 2048, 4100, 9000, 20000, 33000, 49999):
        small = make(tokens)
        assert all(torch.equal(a, b) for a, b in zip(run(small, tokens), run(large, tokens))), tokens
        pkg.tfl_linear_destroy(small)
    pkg.tfl_linear_destroy(large)
