"""The operators of a dense block together, as a program runs them: an 8-bit MLP between
two norms (prefill and decode), a training step with dropout captured in a graph and
replayed, workspaces side by side on two streams, and tensors past 4 GiB.

Each step is compared with its float64 definition on the step's own inputs, so the
tolerances are those of the single operators: 16-bit outputs within half a step and 2^-17 of
the magnitudes they are made of (fp32 sums of at most 16384 terms in chains of 28, whose
errors add up to less than 2^-17)."""
import numpy as np
import pytest

import tile_gemm_communication_amd as fm
from gpu_util import say
from oracle import dense as od

pytestmark = pytest.mark.gpu

REL = 2.0 ** -17
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


@pytest.fixture(autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _h(t):
    return t.double().cpu().numpy()


def _near(got, ref, mag, dt, slope=1.0):
    lim = slope * REL * mag + HALF[dt] * np.abs(ref) + 1e-7
    assert (np.abs(_h(got) - ref) <= lim).all(), float((np.abs(_h(got) - ref) - lim).max())


@pytest.mark.parametrize("M,hidden,ffn,dt", [(1, 1024, 2816, "bf16"), (5, 512, 1024, "fp16"), (61, 1024, 2816, "bf16"),
                                             (300, 1024, 2816, "fp16")])
def test_mlp_in_8_bits(M, hidden, ffn, dt):
    """norm (8-bit rows) -> product, GELU -> linear layer -> bias and residual -> norm."""
    import torch
    say(f"8-bit MLP M={M} {hidden}x{ffn} {dt}")
    t = _dtype(dt)
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    e = lambda *s, d=t: torch.empty(s, dtype=d, device="cuda")  # noqa: E731
    resid, block, w, b, bias1, bias2 = (n(M, hidden).to(t), n(M, hidden), (1 + 0.2 * n(hidden)).to(t),
                                        (0.1 * n(hidden)).to(t), (0.1 * n(ffn)).to(t), (0.1 * n(hidden)).to(t))
    weights = []
    for N, K in ((ffn, hidden), (hidden, ffn)):       # once, when weights are loaded
        full, q, s = n(N, K) / K ** 0.5, e(N, K, d=torch.int8), e(N, d=torch.float32)
        fm.fm_quant_i8(full, q, s)
        weights.append((q, s))
    out, y, ys = e(M, hidden), e(M, hidden, d=torch.int8), e(M, d=torch.float32)
    fm.fm_layer_norm(out, y, block=block, resid=resid, w=w, b=b, y_scale=ys)
    act = e(M, ffn)
    fm.fm_gemm_i8(y, ys, *weights[0], act, bias=bias1, act=fm.FM_ACT_GELU_TANH)
    mlp = e(M, hidden, d=torch.float32)
    fm.fm_linear_i8(act, *weights[1], mlp, ws=fm.linear_i8_workspace(M, ffn))
    out2, y2 = e(M, hidden), e(M, hidden)
    fm.fm_layer_norm(out2, y2, block=mlp, resid=out, bias=bias2, w=w, b=b)

    z, ry, _, _, mag = od.layer_norm(_h(block), _h(resid), None, _h(w), _h(b), None, 1e-5)
    _near(out, z, mag, dt)
    s = _h(ys)[:, None]
    assert (np.abs(_h(y) * s - ry) <= 0.51 * s + REL * (np.abs(ry) + 1)).all()
    c, v, mag = od.gemm_i8(y.cpu().numpy(), _h(ys), weights[0][0].cpu().numpy(), _h(weights[0][1]), _h(bias1), 2)
    _near(act, c, mag, dt, slope=1.13)
    rq, rs = od.quant(_h(act))
    c, v, mag = od.gemm_i8(rq, rs, weights[1][0].cpu().numpy(), _h(weights[1][1]), None, 0)
    _near(mlp, c, mag, "fp32")
    z, ry, *_, mag = od.layer_norm(_h(mlp), _h(out), _h(bias2), _h(w), _h(b), None, 1e-5)
    _near(out2, z, mag, dt)
    _near(y2, ry, 8 * (np.abs(ry) + 1), dt)


def _step(M, N, t, seed=0):
    """A training step of one block's surroundings: buffers and the calls."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    v = dict(block=n(M, N), resid=n(M, N).to(t), bias=(0.1 * n(N)).to(t), w=(1 + 0.2 * n(N)).to(t), b=(0.1 * n(N)).to(t),
             d_y=n(M, N).to(t), d_out=n(M, N).to(t))
    o = {k: torch.zeros(M, N, dtype=t, device="cuda") for k in ("out", "y", "d_resid", "x", "dx")}
    o.update({k: torch.zeros(N, device="cuda") for k in ("d_bias", "d_w", "d_b")}, d_block=torch.zeros(M, N, device="cuda"))
    mean, rstd, ws = torch.zeros(M, device="cuda"), torch.zeros(M, device="cuda"), fm.layer_norm_workspace(M, N)
    rng = torch.tensor([77, 5], device="cuda")

    def calls():
        fm.fm_layer_norm(o["out"], o["y"], block=v["block"], resid=v["resid"], bias=v["bias"], w=v["w"], b=v["b"], p=0.2,
                         rng=rng, draw=1, mean=mean, rstd=rstd)
        fm.fm_dropout(o["y"], o["x"], 0.1, rng, draw=2)
        fm.fm_dropout(v["d_y"], o["dx"], 0.1, rng, draw=2)
        fm.fm_layer_norm_bwd(o["d_resid"], o["d_block"], out=o["out"], d_y=o["dx"], d_out=v["d_out"], w=v["w"], p=0.2,
                             rng=rng, draw=1, mean=mean, rstd=rstd, d_bias=o["d_bias"], d_w=o["d_w"], d_b=o["d_b"], ws=ws)

    return v, o, rng, calls, (mean, rstd)


@pytest.mark.parametrize("M,N", [(37, 1024), (300, 4096), (5, 12296)])
def test_training_step_in_a_graph(M, N):
    """Every replay draws its own mask, advanced on the GPU, and has an eager step's bits."""
    import torch
    t = torch.bfloat16
    v, o, rng, calls, stats = _step(M, N, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
        rng[1:] += 1
    rng.copy_(torch.tensor([77, 5], device="cuda"))
    seen = []
    for i in range(4):
        for x in o.values():
            x.fill_(-3)
        graph.replay()
        torch.cuda.synchronize()
        assert rng.tolist() == [77, 6 + i]
        got = {k: x.clone() for k, x in o.items()}
        rng[1:] -= 1
        calls()
        rng[1:] += 1
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], o[k]) for k in o)
        seen.append(got["d_block"])
    assert not any(torch.equal(seen[0], s) for s in seen[1:])
    # the first replay's step against the definitions
    f = od.keep_factor(M, N, 0.2, 77, 5 + 3, 1)
    z, ry, rm, rr, mag = od.layer_norm(*(_h(v[k]) for k in ("block", "resid", "bias", "w", "b")), f, 1e-5)
    _near(o["out"], z, mag, "bf16")
    _near(o["y"], ry, 16 * (np.abs(ry) + 1), "bf16")
    f2 = od.keep_factor(M, N, 0.1, 77, 8, 2)
    _near(o["x"], _h(o["y"]) * f2, np.abs(_h(o["y"])) * f2, "bf16")
    gr, m = od.layer_norm_bwd(_h(o["dx"]), _h(v["d_out"]), _h(o["out"]), _h(stats[0]), _h(stats[1]), _h(v["w"]), f)
    for k, dt in (("d_resid", "bf16"), ("d_block", "fp32"), ("d_bias", "fp32"), ("d_w", "fp32"), ("d_b", "fp32")):
        _near(o[k], gr[k], m[k], dt)


def test_linear_in_a_graph():
    import torch
    for M in (1, 3, 40, 200):
        K, N = 1024, 776
        x, q, s = torch.randn(M, K, device="cuda").half(), torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
        fm.fm_quant_i8(torch.randn(N, K, device="cuda"), q, s)
        C, ws = torch.zeros(M, N, dtype=torch.half, device="cuda"), fm.linear_i8_workspace(M, K)
        fm.fm_linear_i8(x, q, s, C, act=fm.FM_ACT_SILU, ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fm.fm_linear_i8(x, q, s, C, act=fm.FM_ACT_SILU, ws=ws)
        for i in range(3):
            x.copy_(torch.randn(M, K, device="cuda"))
            C.fill_(-3)
            graph.replay()
            torch.cuda.synchronize()
            got = C.clone()
            ws.fill_(0xFF)
            fm.fm_linear_i8(x, q, s, C, act=fm.FM_ACT_SILU, ws=ws)
            assert torch.equal(got, C), M


def test_two_streams_with_workspaces_of_their_own():
    import torch
    a, b = _step(400, 2048, torch.bfloat16, 1), _step(390, 4096, torch.bfloat16, 2)
    refs = []
    for s in (a, b):
        s[3]()
        torch.cuda.synchronize()
        refs.append({k: x.clone() for k, x in s[1].items()})
        for x in s[1].values():
            x.fill_(-3)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                s[3]()
    torch.cuda.synchronize()
    for s, ref in zip((a, b), refs):
        assert all(torch.equal(ref[k], s[1][k]) for k in ref)


def test_tensors_past_4_gib():
    """Rows behind the first 2^32 bytes and 2^31 elements have what the same rows alone have."""
    import torch
    t, N = torch.bfloat16, 4096
    M = (1 << 31) // N + 1001
    say(f"past 4 GiB: {M} x {N}")
    rng = torch.tensor([3, 4], device="cuda")
    x = torch.empty(M, N, dtype=t, device="cuda")
    for i in range(0, M, 65536):
        x[i:i + 65536] = torch.randn(min(65536, M - i), N, device="cuda").to(t)
    rows = [0, 1, (1 << 31) // N - 1, (1 << 31) // N, M - 1000, M - 1]
    w = torch.ones(N, dtype=t, device="cuda") + torch.rand(N, device="cuda").to(t)
    y = torch.empty_like(x)
    fm.fm_dropout(x, y, 0.3, rng)
    one = torch.empty(1, N, dtype=t, device="cuda")
    for r in rows:
        fm.fm_dropout(x[r:r + 1], one, 0.3, rng, row_begin=r)
        assert torch.equal(one, y[r:r + 1]), r
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    out = torch.empty_like(x)
    fm.fm_layer_norm(out, y, block=x, resid=x, w=w, p=0.3, rng=rng, mean=mean, rstd=rstd)
    d = torch.empty_like(x)
    fm.fm_layer_norm_bwd(None, d, out=out, d_y=y, w=w, p=0.3, rng=rng, mean=mean, rstd=rstd)
    o1, y1, d1 = (torch.empty(1, N, dtype=t, device="cuda") for _ in range(3))
    m1, r1 = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    for r in rows:
        fm.fm_layer_norm(o1, y1, block=x[r:r + 1], resid=x[r:r + 1], w=w, p=0.3, rng=rng, row_begin=r, mean=m1, rstd=r1)
        fm.fm_layer_norm_bwd(None, d1, out=o1, d_y=y1, w=w, p=0.3, rng=rng, row_begin=r, mean=m1, rstd=r1)
        assert torch.equal(o1, out[r:r + 1]) and torch.equal(y1, y[r:r + 1]) and torch.equal(d1, d[r:r + 1]), r
        assert m1[0] == mean[r] and r1[0] == rstd[r]
    del out, d, y
    # the same tensor's rows in 8 bits, 2^31 of them and more, and their product
    q, s = torch.empty(M, N, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    fm.fm_quant_i8(x, q, s)
    q1, s1 = torch.empty(1, N, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
    W = torch.randint(-127, 128, (72, N), dtype=torch.int8, device="cuda")
    ws = torch.rand(72, device="cuda")
    C, C1 = torch.empty(M, 72, device="cuda"), torch.empty(1, 72, device="cuda")
    fm.fm_gemm_i8(q, s, W, ws, C)
    for r in rows:
        fm.fm_quant_i8(x[r:r + 1], q1, s1)
        fm.fm_gemm_i8(q1, s1, W, ws, C1)
        assert torch.equal(q1, q[r:r + 1]) and s1[0] == s[r] and torch.equal(C1, C[r:r + 1]), r
    # weights and results past 4 GiB
    A, sa = W[:40].contiguous(), torch.rand(40, device="cuda")
    n = M // 8 * 8
    big = torch.empty(40, n, device="cuda")
    for rows_of_a in (3, 40):
        out = big[:rows_of_a]
        fm.fm_gemm_i8(A[:rows_of_a], sa[:rows_of_a], q[:n], s[:n], out)
        at = torch.tensor([0, (1 << 31) // N - 1, (1 << 31) // N, n - 8, n - 1], device="cuda")
        ref = (A[:rows_of_a].double() @ q[at].double().t().contiguous()) * (sa[:rows_of_a, None].double() * s[at].double())
        assert (out[:, at].double() - ref).abs().max() <= 2.0 ** -20 * ref.abs().max()
