"""fm_norm_residual and fm_norm_residual_bwd against the float64 definitions.

Tolerances, in units u = 2^-24.  rstd: a sum of squares in chains of at most 16, 6 and
16 additions, halved by the root, and v_rsq's ulp: 24 u.  out: that, three products
and two additions: 32 u of the magnitudes of its terms.  y: out's error, its own rstd
and two products.  The gradients take two such steps one after another, each with a
mean over the row (40 u) and six roundings: 128 u of their terms' magnitudes.  Column
sums add one rounding a row of the longest chain (rows of a block, 64-way joins): M u /
256 + 80 u at most.  An output of 16 bits rounds by eps / 2."""
import numpy as np
import pytest

import tile_gemm_communication_amd as fm
from gpu_util import say
from oracle import block as ob

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": U}
TINY = {"bf16": 1e-38, "fp16": 2.0 ** -25, "fp32": 1e-38}
EPS = 1e-5


@pytest.fixture(autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _dev(a, dt):
    import torch
    return None if a is None else torch.from_numpy(a).to("cuda:0").to(_dtype(dt))


def _host(t):
    return None if t is None else t.double().cpu().numpy()


def _buf(shape, dt):
    """A view of `shape` and the sentinels behind it."""
    import torch
    n = int(np.prod(shape))
    flat = torch.full((n + 8,), -7.0, device="cuda:0", dtype=_dtype(dt))
    return flat[:n].view(shape), flat[n:]


CASES = [  # M, N, dt, stream, block, post, pre, gates
    (1, 8, "bf16", "bf16", "fp32", 1, 1, 0),
    (1, 4096, "bf16", "bf16", "fp32", 1, 1, 1),
    (5, 264, "fp16", "fp32", "fp16", 1, 1, 5),
    (37, 512, "bf16", "fp32", "fp32", 0, 1, 1),
    (30, 520, "fp16", "fp16", "fp16", 1, 0, 6),
    (64, 1024, "bf16", "bf16", "bf16", 1, 1, 4),
    (33, 1032, "fp16", "fp32", "fp32", 1, 1, 33),
    (600, 2048, "bf16", "bf16", "fp32", 1, 1, 300),
    (20, 2056, "bf16", "bf16", "fp32", 1, 1, 2),
    (700, 4096, "bf16", "fp32", "bf16", 1, 1, 7),
    (9, 8192, "fp16", "fp32", "fp32", 1, 1, 3),
    (300, 12288, "fp16", "fp32", "fp32", 1, 1, 4),
    (11, 12296, "bf16", "bf16", "fp32", 1, 1, 1),
    (6, 16384, "bf16", "fp32", "bf16", 1, 1, 6),
    (3000, 64, "bf16", "bf16", "bf16", 1, 1, 1500),
    (9000, 8, "fp16", "fp16", "fp32", 1, 1, 4500),
    (2, 72, "bf16", "bf16", "bf16", 0, 1, 0),
    (50, 640, "bf16", "bf16", "none", 0, 1, 0),
]


def _inputs(M, N, dt, stream, block, post, pre, G, seed=1):
    rng = np.random.default_rng(seed)
    r = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    b = None if block == "none" else 1.5 * r(M, N)
    if b is not None and M > 2:
        b[1] = 0                               # a row of zeros: rms is sqrt(eps)
    return {"block": _dev(b, "fp32" if block == "none" else block), "resid": _dev(2 * r(M, N), stream),
            "w_post": _dev(1 + 0.3 * r(N), dt) if post else None,
            "w_pre": _dev(1 + 0.3 * r(N), dt) if pre else None,
            "gate": _dev(r(G, N), dt) if G else None}


@pytest.mark.parametrize("M,N,dt,stream,block,post,pre,G", CASES)
def test_norm_forward(M, N, dt, stream, block, post, pre, G):
    import torch
    say(f"norm M={M} N={N} {dt}/{stream}/{block} post={post} pre={pre} G={G}")
    v = _inputs(M, N, dt, stream, block, post, pre, G)
    out, out_end = _buf((M, N), stream)
    y, y_end = _buf((M, N), dt)
    rq, rq_end = _buf((M,), "fp32")
    rp, rp_end = _buf((M,), "fp32")
    fm.fm_norm_residual(out, y if pre else None, **v, scale=0.7, eps=EPS,
                        rstd_post=rq if post else None, rstd_pre=rp if pre else None)
    torch.cuda.synchronize()
    for e in (out_end, y_end, rq_end, rp_end):
        assert (e == -7).all()
    ro, ry, rrq, rrp, mag = ob.norm(*(_host(v[k]) for k in ("block", "resid", "w_post", "w_pre",
                                                            "gate")), np.float32(0.7), EPS)
    err = np.abs(_host(out) - ro)
    assert (err <= 32 * U * mag + HALF[stream] * np.abs(ro) + TINY[stream]).all()
    if post:
        np.testing.assert_allclose(_host(rq), rrq, rtol=24 * U)
    if pre:
        # the rms of out moves by at most the largest relative error of its rows' terms
        rel = 32 * U * np.linalg.norm(mag, axis=1) / np.maximum(np.linalg.norm(ro, axis=1), 1e-30)
        assert (np.abs(_host(rp) / rrp - 1) <= 24 * U + rel).all()
        w = np.abs(_host(v["w_pre"]))
        lim = (32 * U * mag + (28 * U + rel)[:, None] * np.abs(ro)) * rrp[:, None] * w
        assert (np.abs(_host(y) - ry) <= lim + HALF[dt] * np.abs(ry) + TINY[dt]).all()
    # in place, without what is not wanted, and the same bits
    r2 = v["resid"].clone()
    fm.fm_norm_residual(r2, None, **{**v, "resid": r2, "w_pre": None}, scale=0.7, eps=EPS)
    assert torch.equal(r2, out)
    if pre:
        y2 = torch.empty_like(y)
        fm.fm_norm_residual(None, y2, **v, scale=0.7, eps=EPS)
        assert torch.equal(y2, y)


@pytest.mark.parametrize("M,N,dt,stream,block,post,pre,G", CASES)
def test_norm_backward(M, N, dt, stream, block, post, pre, G):
    import torch
    say(f"norm bwd M={M} N={N} {dt}/{stream}/{block} post={post} pre={pre} G={G}")
    v = _inputs(M, N, dt, stream, block, post, pre, G, seed=2)
    has_block = v["block"] is not None
    rng = np.random.default_rng(3)
    d_y = _dev(rng.standard_normal((M, N)), dt) if pre else None
    d_out = _dev(rng.standard_normal((M, N)), stream)
    rq = _dev(1 / np.sqrt((_host(v["block"]) ** 2).mean(1) + EPS), "fp32") if post else None
    rp = _dev(1 / np.sqrt((_host(v["resid"]) ** 2).mean(1) + EPS), "fp32") if pre else None
    ends, got = [], {}

    def buf(name, shape, t, want=True):
        if want:
            got[name], e = _buf(shape, t)
            ends.append(e)
        return got.get(name)

    ws = torch.full((fm.fm_norm_residual_workspace_bytes(M, N, G) + 64,), 0xFF, dtype=torch.uint8,
                    device="cuda:0")
    kw = dict(out=v["resid"], block=v["block"], d_y=d_y, d_out=d_out, w_post=v["w_post"],
              w_pre=v["w_pre"], gate=v["gate"], scale=0.7, rstd_post=rq, rstd_pre=rp, ws=ws[:-64])
    fm.fm_norm_residual_bwd(buf("d_resid", (M, N), stream),
                            buf("d_block", (M, N), block, has_block),
                            d_w_post=buf("d_w_post", (N,), "fp32", post),
                            d_w_pre=buf("d_w_pre", (N,), "fp32", pre),
                            d_gate=buf("d_gate", (G, N), "fp32", G), **kw)
    torch.cuda.synchronize()
    for e in ends + [ws[-64:].float()]:
        assert (e == (255 if e is not ends[0] and e.numel() == 64 else -7)).all()
    ref, mag = ob.norm_bwd(*(_host(x) for x in (d_y, d_out, v["resid"], v["block"], v["w_post"],
                                                v["w_pre"], v["gate"])), float(np.float32(0.7)),
                           _host(rq), _host(rp))
    types = {"d_resid": stream, "d_block": block}
    for name, t in got.items():
        d = types.get(name, "fp32")
        more = 0 if name in types else M / 256 + 80
        err = np.abs(_host(t) - ref[name])
        lim = (128 + more) * U * mag[name] + HALF[d] * np.abs(ref[name]) + TINY[d]
        assert (err <= lim).all(), (name, float((err / lim).max()))
    # d_resid over d_out, one gradient at a time, and the same bits
    do = d_out.clone()
    fm.fm_norm_residual_bwd(do, None, **{**kw, "d_out": do})
    assert torch.equal(do, got["d_resid"])
    for name in got:
        if name == "d_resid":
            continue
        one = torch.full_like(got[name], -7.0)
        args = {"d_w_post": None, "d_w_pre": None, "d_gate": None, "d_block": None, name: one}
        fm.fm_norm_residual_bwd(None, args.pop("d_block"), **args, **kw)
        assert torch.equal(one, got[name]), name


def test_norm_backward_without_rows():
    """The column sums of no rows are zero."""
    import torch
    e = torch.empty(0, 64, device="cuda:0", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda:0", dtype=torch.bfloat16)
    d = torch.full((64,), 5.0, device="cuda:0")
    fm.fm_norm_residual_bwd(e, e, out=e, block=e, d_y=e, d_out=e, w_pre=w, w_post=w,
                            rstd_post=torch.empty(0, device="cuda:0"),
                            rstd_pre=torch.empty(0, device="cuda:0"), d_w_pre=d, d_w_post=d.clone(),
                            ws=fm.norm_residual_workspace(0, 64))
    assert (d == 0).all()


def test_norm_only_loss_gradient_of_out():
    """Without d_out the stream's gradient is the norm's alone."""
    import torch
    v = _inputs(40, 256, "bf16", "fp32", "fp32", 1, 1, 0)
    rp = _dev(1 / np.sqrt((_host(v["resid"]) ** 2).mean(1) + EPS), "fp32")
    d_y = _dev(np.random.default_rng(0).standard_normal((40, 256)), "bf16")
    d = torch.empty(40, 256, device="cuda:0")
    fm.fm_norm_residual_bwd(d, None, out=v["resid"], d_y=d_y, w_pre=v["w_pre"], rstd_pre=rp)
    ref, mag = ob.norm_bwd(_host(d_y), None, _host(v["resid"]), None, None, _host(v["w_pre"]), None,
                           1.0, None, _host(rp))
    assert (np.abs(_host(d) - ref["d_resid"]) <= 128 * U * mag["d_resid"] + 1e-38).all()


@pytest.mark.parametrize("M,N,stream,block,G", [(5, 264, "fp32", "fp32", 0), (37, 4096, "bf16", "bf16", 1),
                                                (6, 16384, "fp32", "bf16", 6), (300, 64, "bf16", "fp32", 100)])
def test_norm_backward_of_a_frozen_block(M, N, stream, block, G):
    """Where only d_resid and d_w_pre are wanted, w_post, gate and scale have no part: neither
    block nor rstd_post has to be there, and the gradients are those of the call with both."""
    import torch
    say(f"norm bwd, frozen block M={M} N={N} {stream}/{block} G={G}")
    v = _inputs(M, N, "bf16", stream, block, 1, 1, G, seed=4)
    rng = np.random.default_rng(5)
    d_y, d_out = _dev(rng.standard_normal((M, N)), "bf16"), _dev(rng.standard_normal((M, N)), stream)
    rq = _dev(1 / np.sqrt((_host(v["block"]) ** 2).mean(1) + EPS), "fp32")
    rp = _dev(1 / np.sqrt((_host(v["resid"]) ** 2).mean(1) + EPS), "fp32")
    kw = dict(out=v["resid"], d_y=d_y, d_out=d_out, w_post=v["w_post"], w_pre=v["w_pre"], gate=v["gate"],
              scale=0.7, rstd_pre=rp, ws=fm.norm_residual_workspace(M, N, G))
    grads = []
    for more, wanted in ((dict(block=v["block"], rstd_post=rq), "rp"), (dict(), "rp"), (dict(), "r"),
                         (dict(), "p"), (dict(block=v["block"]), "rp")):
        d = torch.full((M, N), -7.0, device="cuda:0", dtype=_dtype(stream)) if "r" in wanted else None
        dp = torch.full((N,), -7.0, device="cuda:0") if "p" in wanted else None
        fm.fm_norm_residual_bwd(d, None, **kw, **more, d_w_pre=dp)
        torch.cuda.synchronize()
        grads.append((d, dp))
    ref, mag = ob.norm_bwd(*(_host(x) for x in (d_y, d_out, v["resid"], v["block"], v["w_post"],
                                                v["w_pre"], v["gate"])), float(np.float32(0.7)),
                           _host(rq), _host(rp))
    for k, t, h, more in (("d_resid", grads[0][0], HALF[stream], 0), ("d_w_pre", grads[0][1], U, M / 256 + 80)):
        err = np.abs(_host(t) - ref[k])
        assert (err <= (128 + more) * U * mag[k] + h * np.abs(ref[k]) + TINY[stream]).all(), k
    for d, dp in grads[1:]:
        assert d is None or torch.equal(d, grads[0][0])
        assert dp is None or torch.equal(dp, grads[0][1])
    with pytest.raises(fm.FluxMIError):      # d_w_post is a sum over block / rms(block)
        fm.fm_norm_residual_bwd(None, None, **kw, block=v["block"], d_w_post=torch.empty(N, device="cuda:0"))


@pytest.mark.parametrize("G", [0, 1, "rows"])
def test_norm_without_rows(G):
    """A batch of no tokens goes through forward and backward."""
    import torch
    e, r = torch.empty(0, 64, device="cuda:0", dtype=torch.bfloat16), torch.empty(0, device="cuda:0")
    w = torch.ones(64, device="cuda:0", dtype=torch.bfloat16)
    gate = {0: None, 1: w.view(1, 64), "rows": e}[G]
    fm.fm_norm_residual(e, e, block=e, resid=e, w_post=w, w_pre=w, gate=gate, rstd_post=r, rstd_pre=r)
    fm.fm_norm_residual_bwd(e, e, out=e, block=e, d_y=e, d_out=e, w_post=w, w_pre=w, gate=gate,
                            rstd_post=r, rstd_pre=r)
    torch.cuda.synchronize()
