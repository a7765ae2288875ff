"""The operators around a sparse block together, as one rank runs them: GEMM-ReduceScatter
slices, norm and residual, router, the experts (16-bit or 4-bit), the norm after; then the
backward of router and norms.  Each step is compared with the float64 definition on the
bits that the step before left.  Captured into a graph, the chain is replayed between eager
work and compared with the eager result; two chains run on two streams at once."""
import numpy as np
import pytest

import tile_gemm_communication_amd as fm
import workloads as wl
from gpu_util import say, side_stream
from oracle import block as ob

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
T, HID, FFN, E, TOPK, GROUP = 96, 512, 256, 16, 2, 64
EPS = 1e-5


@pytest.fixture(autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _host(t):
    return t.double().cpu().numpy()


class Chain:
    """One rank's buffers and the calls of a block."""

    def __init__(self, seed, four):
        import torch
        bf, dev = torch.bfloat16, "cuda:0"
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
        self.four = four
        self.a, self.w = r(T, 256).to(bf), (r(256, HID) / 16).to(bf)
        self.slices = torch.zeros(T, HID, device=dev)
        self.resid = r(T, HID).to(bf)
        self.w_post, self.w_pre, self.gate = ((1 + 0.1 * r(HID)).to(bf) for _ in range(3))
        self.gate = self.gate.view(1, HID)
        self.out, self.y = torch.empty_like(self.resid), torch.empty_like(self.resid)
        self.rq, self.rp = torch.empty(T, device=dev), torch.empty(T, device=dev)
        self.w_r = (r(HID, E) / 8).to(bf)
        self.logits = torch.empty(T, E, device=dev)
        self.ids = torch.empty(T, TOPK, dtype=torch.int32, device=dev)
        self.wts = torch.empty(T, TOPK, device=dev)
        self.counts = torch.empty(E + 1, dtype=torch.int32, device=dev)
        self.sums, self.loss = torch.empty(E, device=dev), torch.empty(1, device=dev)
        self.gws = fm.moe_gate_workspace(T, E)
        self.ws, self.w4ws = fm.moe_workspace(T, TOPK, HID, E), fm.moe_w4_workspace(T, TOPK, HID)
        self.h = torch.zeros(T * TOPK, FFN, device=dev, dtype=bf)
        self.sp = torch.zeros(T * TOPK, dtype=torch.int32, device=dev)
        self.off = torch.zeros(E + 1, dtype=torch.int32, device=dev)
        self.moe = torch.zeros(T, HID, device=dev)
        if four:
            self.m = []
            for K, N in ((HID, FFN), (FFN, HID)):
                c = torch.randint(0, 16, (E, K, N), generator=g, device=dev).to(torch.uint8)
                p = torch.empty(E, N, fm.fm_w4_row_bytes(K), dtype=torch.uint8, device=dev)
                fm.fm_w4_pack(c, p)
                self.m.append((p, ((0.5 + torch.rand(E, K // GROUP, N, generator=g, device=dev))
                                   / (5 * K ** 0.5)).to(bf)))
        else:
            self.w1, self.w2 = (r(E, HID, FFN) / HID ** 0.5).to(bf), (r(E, FFN, HID) / FFN ** 0.5).to(bf)
        self.out2, self.y2 = torch.empty_like(self.out), torch.empty_like(self.y)
        self.rq2, self.rp2 = torch.empty(T, device=dev), torch.empty(T, device=dev)
        self.d_y, self.d_out = r(T, HID).to(bf), r(T, HID).to(bf)
        self.d_wts, self.d_loss = r(T, TOPK), torch.full((1,), 3.0, device=dev)
        self.d_resid, self.d_moe = torch.empty_like(self.out), torch.empty_like(self.moe)
        self.d_w_post, self.d_w_pre = (torch.empty(HID, device=dev) for _ in range(2))
        self.d_gate = torch.empty(1, HID, device=dev)
        self.d_logits = torch.empty_like(self.logits)
        self.nws = fm.norm_residual_workspace(T, HID, 1)

    def run(self):
        self.slices.zero_()
        self.moe.zero_()
        fm.fm_gemm_rs(self.a, self.w, list(self.slices.view(4, T // 4, HID)), rank=1)
        fm.fm_norm_residual(self.out, self.y, block=self.slices, resid=self.resid,
                            w_post=self.w_post, w_pre=self.w_pre, eps=EPS, rstd_post=self.rq,
                            rstd_pre=self.rp)
        fm.fm_gemm(self.y, self.w_r, self.logits)
        fm.fm_moe_gate(self.logits, self.ids, self.wts, renormalize=True, counts=self.counts,
                       prob_sums=self.sums, loss=self.loss, ws=self.gws)
        if self.four:
            fm.fm_moe_gather_gemm_w4(self.y, self.ids, *self.m[0], self.h, self.sp, self.off, 0,
                                     GROUP, self.ws, act=fm.FM_ACT_SILU)
            fm.fm_moe_gemm_scatter_w4(self.h, *self.m[1], self.ids, self.sp, self.off, self.wts,
                                      self.moe, 0, GROUP, self.w4ws)
        else:
            fm.fm_moe_gather_gemm_act(self.y, self.ids, self.w1, self.h, self.sp, self.off, 0,
                                      fm.FM_ACT_SILU, self.ws)
            fm.fm_moe_gemm_scatter(self.h, self.w2, self.sp, self.off, self.wts, self.moe, self.ws)
        fm.fm_norm_residual(self.out2, self.y2, block=self.moe, resid=self.out, w_post=self.w_post,
                            w_pre=self.w_pre, gate=self.gate, scale=0.5, eps=EPS,
                            rstd_post=self.rq2, rstd_pre=self.rp2)
        fm.fm_norm_residual_bwd(self.d_resid, self.d_moe, out=self.out2, block=self.moe,
                                d_y=self.d_y, d_out=self.d_out, w_post=self.w_post,
                                w_pre=self.w_pre, gate=self.gate, scale=0.5, rstd_post=self.rq2,
                                rstd_pre=self.rp2, d_w_post=self.d_w_post, d_w_pre=self.d_w_pre,
                                d_gate=self.d_gate, ws=self.nws)
        fm.fm_moe_gate_bwd(self.logits, self.ids, self.d_logits, renormalize=True,
                           d_weights=self.d_wts, counts=self.counts, d_loss=self.d_loss)

    def results(self):
        return {k: getattr(self, k).clone() for k in
                ("out", "y", "logits", "ids", "wts", "counts", "sums", "loss", "moe", "out2", "y2",
                 "d_resid", "d_moe", "d_w_post", "d_w_pre", "d_gate", "d_logits")}


@pytest.mark.parametrize("four", [False, True])
def test_chain_against_definitions(four):
    import torch
    say(f"chain four={four}")
    c = Chain(3, four)
    c.run()
    torch.cuda.synchronize()
    ro, ry, rq, rp, mag = ob.norm(_host(c.slices), _host(c.resid), _host(c.w_post), _host(c.w_pre),
                                  None, 1.0, EPS)
    assert (np.abs(_host(c.out) - ro) <= 32 * U * mag + 2.0 ** -8 * np.abs(ro)).all()
    assert (np.abs(_host(c.y) - ry) <= 1e-5 * np.abs(ry).max() + 2.0 ** -8 * np.abs(ry)).all()
    ids, w, counts, sums, loss = ob.gate(_host(c.logits), TOPK, 0, True, 1.0)
    assert np.array_equal(c.ids.cpu().numpy(), ids) and np.array_equal(c.counts.cpu().numpy(), counts)
    np.testing.assert_allclose(_host(c.wts), w, rtol=1e-5)
    np.testing.assert_allclose(_host(c.sums), sums, rtol=1e-4)
    np.testing.assert_allclose(c.loss.item(), loss, rtol=1e-4)
    ro, ry, rq, rp, mag = ob.norm(_host(c.moe), _host(c.out), _host(c.w_post), _host(c.w_pre),
                                  _host(c.gate), 0.5, EPS)
    assert (np.abs(_host(c.out2) - ro) <= 32 * U * mag + 2.0 ** -8 * np.abs(ro)).all()
    ref, mag = ob.norm_bwd(_host(c.d_y), _host(c.d_out), _host(c.out2), _host(c.moe),
                           _host(c.w_post), _host(c.w_pre), _host(c.gate), 0.5, _host(c.rq2),
                           _host(c.rp2))
    for k, h in (("d_w_post", U), ("d_w_pre", U), ("d_gate", U), ("d_resid", 2.0 ** -8)):
        t = _host(getattr(c, k))
        assert (np.abs(t - ref[k]) <= 210 * U * mag[k] + h * np.abs(ref[k])).all(), k
    assert (np.abs(_host(c.d_moe) - ref["d_block"]) <= 129 * U * mag["d_block"]).all()
    dx, mg = ob.gate_bwd(_host(c.logits), ids, 0, True, 1.0, None, _host(c.d_wts), counts, 3.0)
    assert (np.abs(_host(c.d_logits) - dx) <= 400 * U * mg + 1e-37).all()


def _same(a, b):
    import torch
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("four", [False, True])
def test_chain_in_a_graph(four):
    import torch
    c = Chain(4, four)
    c.run()                                     # library warm-up outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    other = Chain(5, four)
    for i in range(4):
        c.resid.copy_(torch.randn_like(c.resid, dtype=torch.float32))
        c.a.copy_(torch.randn_like(c.a, dtype=torch.float32))
        for t in (c.y, c.ids, c.wts, c.moe, c.d_gate, c.gws, c.nws, c.w4ws):
            t.fill_(1)
        other.run()
        graph.replay()
        torch.cuda.synchronize()
        got = c.results()
        c.run()
        torch.cuda.synchronize()
        _same(got, c.results())


def test_two_chains_at_once():
    import torch
    a, b = Chain(6, True), Chain(7, True)
    a.run()
    b.run()
    torch.cuda.synchronize()
    ra, rb = a.results(), b.results()
    side = side_stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(side):
            b.run()
        a.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    _same(ra, a.results())
    _same(rb, b.results())
