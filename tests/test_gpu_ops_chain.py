"""The norm and the feed-forward behind it, turn after turn on the same buffers without a pause, as
in generation: each kernel may start while the one before it still runs, so what it reads has to be
the newest.  Every turn has new values, and has to give the bits of a turn run alone."""
import pytest

pytestmark = pytest.mark.gpu

EPS = 1e-5
TURNS = 48


class Chain:
    """norm into y (and its scales), feed-forward from y; y and the scales are the same buffers every turn."""

    def __init__(self, tokens, d, f, e4m3):
        import torch
        import attention_qkv_gemm_gb300 as pkg
        self.pkg, self.tokens, self.e4m3 = pkg, tokens, e4m3
        gen = torch.Generator(device="cuda").manual_seed(tokens + d)
        self.rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
        self.x = self.rnd(TURNS, tokens, d).bfloat16()
        self.gamma = 1 + 0.1 * self.rnd(d)
        self.wg, self.sg = self._weights(f, d)
        self.wu, self.su = self._weights(f, d)
        self.n = pkg.tfl_rmsnorm_create(d, pkg.TFL_BF16, pkg.TFL_BF16, pkg.TFL_E4M3 if e4m3 else pkg.TFL_BF16, EPS)
        self.g = pkg.tfl_glu_create(d, f, pkg.TFL_E4M3 if e4m3 else pkg.TFL_BF16, pkg.TFL_BF16, pkg.TFL_ACT_SILU)
        self.y, self.ys = self.buffers()
        self.h = torch.empty(TURNS, tokens, f, dtype=torch.bfloat16, device="cuda")

    def _weights(self, f, d):
        import torch
        w = self.rnd(f, d) * d ** -0.5
        if not self.e4m3:
            return w.bfloat16(), None
        s = w.abs().amax(dim=1) / 448
        return (w / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), s

    def buffers(self):
        import torch
        y = torch.zeros(self.x.shape[1:], device="cuda").to(torch.float8_e4m3fn if self.e4m3 else torch.bfloat16)
        return y, torch.zeros(self.tokens, device="cuda") if self.e4m3 else None

    def turn(self, i, y, ys, h, stream):
        P = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self.pkg.tfl_rmsnorm_forward(self.n, self.tokens, P(self.x[i]), None, P(self.gamma), None, P(y), P(ys), stream)
        self.pkg.tfl_glu_forward(self.g, self.tokens, P(y), P(ys), P(self.wg), P(self.sg), P(self.wu), P(self.su), P(h),
                                 stream)

    def alone(self):
        """Every turn on buffers of its own, waited for after each call."""
        import torch
        out, s = torch.empty_like(self.h), torch.cuda.current_stream().cuda_stream
        for i in range(TURNS):
            y, ys = self.buffers()
            torch.cuda.synchronize()
            self.turn(i, y, ys, out[i], s)
            torch.cuda.synchronize()
        return out

    def close(self):
        rc = self.pkg.tfl_glu_status(self.g, 0)
        self.pkg.tfl_rmsnorm_destroy(self.n)
        self.pkg.tfl_glu_destroy(self.g)
        assert rc == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("tokens,d,f", [(1, 1024, 1040), (1, 4096, 4096), (8, 2048, 2080), (16, 512, 2048), (40, 4096, 2048),
                                        (200, 1024, 2048), (1500, 512, 2064)])
def test_turns_on_the_same_buffers_equal_turns_alone(tokens, d, f, e4m3):
    import torch
    c = Chain(tokens, d, f, e4m3)
    try:
        ref = c.alone()
        s = torch.cuda.current_stream().cuda_stream
        for i in range(TURNS):
            c.turn(i, c.y, c.ys, c.h[i], s)
        torch.cuda.synchronize()
        assert torch.equal(c.h, ref)
        # the same as one graph, replayed on other values
        st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            for i in range(TURNS):
                c.turn(i, c.y, c.ys, c.h[i], st.cuda_stream)
        for _ in range(2):
            c.x.copy_(c.rnd(*c.x.shape))
            ref = c.alone()
            c.h.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(c.h, ref)
    finally:
        c.close()
