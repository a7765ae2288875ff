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


def _codes(packed, K):
    """Codes [K, N] of packed bytes [N, row], one nibble at a time; packing them again gives the bytes."""
    words = packed.reshape(packed.shape[0], -1, 64).copy().view("<u4")     # [N, block, 16]
    out = np.zeros((words.shape[1] * 128, packed.shape[0]), np.uint8)
    for w in range(16):
        for p in range(8):
            k = 32 * (w % 4) + 8 * (w // 4) + (2 * p if p < 4 else 2 * (p - 4) + 1)
            out[k::128] = ((words[:, :, w] >> np.uint32(4 * p)) & 15).T
    assert np.array_equal(ob.w4_pack(out), packed)
    return out[:K]


def _norm_matches(out, y, rq, rp, block, resid, w_post, w_pre, gate, scale):
    """Stored stream, normed rows and both 1 / rms against the definition on the same inputs."""
    ro, ry, rrq, rrp, mag = ob.norm(*(_host(t) for t in (block, resid, w_post, w_pre)),
                                    None if gate is None else _host(gate), scale, EPS)
    assert (np.abs(_host(out) - ro) <= 32 * U * mag + 2.0 ** -8 * np.abs(ro)).all()
    np.testing.assert_allclose(_host(rq), rrq, rtol=24 * U)
    # the rms of out moves by at most the largest relative error of its rows' terms
    rel = 32 * U * np.linalg.norm(mag, axis=1) / np.linalg.norm(ro, axis=1)
    assert (np.abs(_host(rp) / rrp - 1) <= 24 * U + rel).all()
    lim = (32 * U * mag + (28 * U + rel)[:, None] * np.abs(ro)) * rrp[:, None] * np.abs(_host(w_pre))
    assert (np.abs(_host(y) - ry) <= lim + 2.0 ** -8 * np.abs(ry)).all()


@pytest.mark.parametrize("four", [False, True])
def test_products_and_norms_of_the_chain(oracle, four):
    """The steps between: both dense products, the route, both expert layers and both norms, each on
    the bits that the step before left.  A product of 16-bit numbers is exact in fp32 and each of its K
    additions is off by at most 2 u (if it truncates): 2 K u of sum |a| |b|.  The 4-bit ones, with base
    16: (K / 256 + 84) u * 62 of sum |x| scale."""
    import torch
    say(f"chain products four={four}")
    c = Chain(8, four)
    c.run()
    torch.cuda.synchronize()

    def near(got, a, b):
        return (np.abs(_host(got) - _host(a) @ _host(b)) <=
                2 * a.shape[1] * U * (np.abs(_host(a)) @ np.abs(_host(b))) + 1e-38).all()

    assert near(c.slices, c.a, c.w) and near(c.logits, c.y, c.w_r)
    _norm_matches(c.out, c.y, c.rq, c.rp, c.slices, c.resid, c.w_post, c.w_pre, None, 1.0)
    _norm_matches(c.out2, c.y2, c.rq2, c.rp2, c.moe, c.out, c.w_post, c.w_pre, c.gate, 0.5)
    ids = c.ids.cpu().numpy()
    roff, rsp = oracle.moe_route(ids, 0, E)
    assert np.array_equal(c.off.cpu().numpy(), roff) and np.array_equal(c.sp.cpu().numpy(), rsp)
    assert roff[-1] == T * TOPK

    def layer(i, x, e):
        """x [rows, K] times expert e's matrix of layer i, and the bound of its error."""
        K = x.shape[1]
        if not four:
            W = _host((c.w1, c.w2)[i][e])
            return x @ W, 2 * K * U * (np.abs(x) @ np.abs(W))
        packed, scales = c.m[i]
        s = _host(scales[e])
        W = ob.w4_matrix(_codes(packed[e].cpu().numpy(), K), s, None, GROUP)
        return x @ W, (K / 256 + 84) * U * 62 * (np.abs(x) @ s[np.arange(K) // GROUP])

    y, h, wts = _host(c.y), _host(c.h), _host(c.wts).reshape(-1)
    moe, lim_moe = np.zeros((T, HID)), np.zeros((T, HID))
    for e in range(E):
        rows = slice(roff[e], roff[e + 1])
        p = rsp[rows]
        if len(p) == 0:
            continue
        v, lim = layer(0, y[p // TOPK], e)
        ref = v / (1 + np.exp(-v))                                # slope at most 1.13
        assert (np.abs(h[rows] - ref) <= 1.13 * lim + 16 * U * np.abs(v) + 2.0 ** -8 * np.abs(ref) + 1e-38).all()
        v, lim = layer(1, h[rows], e)
        np.add.at(moe, p // TOPK, wts[p][:, None] * v)
        np.add.at(lim_moe, p // TOPK, wts[p][:, None] * (lim + (TOPK + 2) * U * np.abs(v)))
    assert (np.abs(_host(c.moe) - moe) <= lim_moe + 2 * U * np.abs(moe) + 1e-38).all()
