"""fm_layer_norm and fm_layer_norm_bwd against the float64 definitions.

Tolerances, in units u = 2^-24.  out: bias, scale (its own rounding too) and residual,
6 u of the magnitudes of its terms.  mean: chains of at most 4 + 2 additions in a lane, 6
in a wave, 16 over the waves, and two for 1 / N: 32 u of the mean magnitude, and out's
error.  The variance v moves by the centred elements' errors d (out's and the mean's):
at most (2 |z'| |d| + |d|^2) / N, and 32 u of itself; rstd by half of that over v + eps,
and 2 u for the root.  y: the errors of the centred element and of rstd, and three
roundings, times |w|; one rounding for b.  Gradients: two means over the row (36 u) and
eight roundings, 48 u of their terms' magnitudes, 3 u more for dropout's scale.  Column
sums add one rounding a row of the longest chain (a block's rows, 16-way and 64-way
joins): M / 256 + 100 u.  An output of 16 bits rounds by eps / 2, one of 8 bits by half
a step and may lie on the other side of a half."""
import numpy as np
import pytest

import tile_gemm_communication_amd as fm
from gpu_util import say
from oracle import dense as od

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": U}
TINY = {"bf16": 1e-38, "fp16": 2.0 ** -25, "fp32": 1e-38}
EPS = 1e-5
SEED, OFFSET, DRAW, ROW = 0x123456789ABCDEF, 2 ** 63 - 4, 9, 2 ** 32 - 40000


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
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0").to(_dtype(dt))


def _host(t):
    return None if t is None else t.double().cpu().numpy()


def _rng():
    import torch
    return torch.tensor([SEED, OFFSET], dtype=torch.int64, device="cuda:0")


def _buf(shape, dt):
    """A view of `shape` and the sentinels behind it."""
    import torch
    n = int(np.prod(shape))
    t = torch.int8 if dt == "int8" else _dtype(dt)
    flat = torch.full((n + 16,), -7, device="cuda:0", dtype=t)
    return flat[:n].view(shape), flat[n:]


CASES = [  # M, N, dt, stream, block ("none": no block), bias, norm, p
    (1, 8, "bf16", "bf16", "fp32", 1, 1, 0.3),
    (1, 4096, "bf16", "bf16", "bf16", 1, 1, 0.0),
    (5, 264, "fp16", "fp32", "fp16", 1, 1, 0.5),
    (37, 512, "bf16", "fp32", "fp32", 0, 1, 0.1),
    (30, 520, "fp16", "fp16", "fp16", 1, 0, 0.1),
    (64, 1024, "bf16", "bf16", "bf16", 1, 1, 0.9),
    (33, 1032, "fp16", "fp32", "fp32", 1, 1, 0.1),
    (601, 2048, "bf16", "bf16", "fp32", 1, 1, 0.1),
    (20, 2056, "bf16", "bf16", "fp32", 1, 1, 0.0),
    (700, 4096, "bf16", "fp32", "bf16", 1, 1, 0.25),
    (9, 8192, "fp16", "fp32", "fp32", 1, 1, 0.1),
    (300, 12288, "fp16", "fp32", "fp32", 1, 1, 0.1),
    (7, 12280, "bf16", "bf16", "bf16", 0, 1, 0.1),
    (11, 12296, "bf16", "bf16", "fp32", 1, 1, 0.1),
    (6, 16384, "bf16", "fp32", "bf16", 1, 1, 0.1),
    (3001, 64, "bf16", "bf16", "bf16", 1, 1, 0.1),
    (9000, 8, "fp16", "fp16", "fp32", 1, 1, 0.1),
    (2, 72, "bf16", "bf16", "bf16", 0, 1, 1.0),
    (50, 640, "bf16", "bf16", "none", 0, 1, 0.0),
    (50, 136, "fp16", "fp32", "fp32", 1, 0, 0.0),
    (1031, 256, "bf16", "bf16", "fp32", 1, 1, 0.1),
    (70, 128, "fp16", "fp32", "fp16", 1, 1, 0.1),
    (33, 120, "bf16", "bf16", "bf16", 1, 1, 0.1),
]


def _inputs(M, N, dt, stream, block, bias, norm, p, seed=1):
    rng = np.random.default_rng(seed)
    r = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    b = None if block == "none" else 1.5 * r(M, N)
    z = 2 * r(M, N) + 3
    if M > 2:
        z[1] = 1.0                             # a row of equals: the variance is 0
        if b is not None:
            b[1] = 0
    return {"block": _dev(b, "fp32" if block == "none" else block), "resid": _dev(z, stream),
            "bias": _dev(0.3 * r(N), dt) if bias else None,
            "w": _dev(1 + 0.3 * r(N), dt) if norm else None,
            "b": _dev(0.3 * r(N), dt) if norm and N % 16 else None}


def _bounds(v, ro, mag, mean, rstd, y):
    """Bounds of the errors of (mean, rstd, y before it is stored)."""
    err = 6 * U * mag
    e_mean = 32 * U * np.abs(ro).mean(axis=1) + err.mean(axis=1)
    away = ro - mean[:, None]
    d = err + (e_mean + U * np.abs(mean))[:, None]
    var = (away * away).mean(axis=1)
    e_var = (2 * np.linalg.norm(away, axis=1) * np.linalg.norm(d, axis=1)
             + (d * d).sum(axis=1)) / ro.shape[1] + 34 * U * var
    # rstd falls like the root: half the relative change, a little more for large ones
    rel = np.minimum(e_var / (var + EPS), 0.5)
    e_rstd = rstd * (0.5 * rel + rel * rel + 3 * U)
    w = np.abs(_host(v["w"]))
    e_y = w * (d * (rstd + e_rstd)[:, None] + np.abs(away) * (e_rstd + 3 * U * rstd)[:, None])
    return e_mean, e_rstd, e_y + 2 * U * (np.abs(y) + (0 if v["b"] is None else np.abs(_host(v["b"]))))


@pytest.mark.parametrize("M,N,dt,stream,block,bias,norm,p", CASES)
def test_forward(M, N, dt, stream, block, bias, norm, p):
    import torch
    say(f"layer norm M={M} N={N} {dt}/{stream}/{block} bias={bias} norm={norm} p={p}")
    v = _inputs(M, N, dt, stream, block, bias, norm, p)
    draws = dict(p=p, rng=_rng() if p else None, draw=DRAW, row_begin=ROW)
    out, out_end = _buf((M, N), stream)
    y, y_end = _buf((M, N), dt)
    mean, mean_end = _buf((M,), "fp32")
    rstd, rstd_end = _buf((M,), "fp32")
    fm.fm_layer_norm(out, y if norm else None, **v, **draws, eps=EPS, mean=mean if norm else None,
                     rstd=rstd if norm else None)
    torch.cuda.synchronize()
    for e in (out_end, y_end, mean_end, rstd_end):
        assert (e == -7).all()
    f = od.keep_factor(M, N, p, SEED, OFFSET, DRAW, ROW)
    ro, ry, rm, rr, mag = od.layer_norm(*(_host(v[k]) for k in ("block", "resid", "bias", "w", "b")), f, EPS)
    assert (np.abs(_host(out) - ro) <= 6 * U * mag + HALF[stream] * np.abs(ro) + TINY[stream]).all()
    if norm:
        e_mean, e_rstd, e_y = _bounds(v, ro, mag, rm, rr, ry)
        assert (np.abs(_host(mean) - rm) <= e_mean).all()
        assert (np.abs(_host(rstd) - rr) <= e_rstd).all()
        assert (np.abs(_host(y) - ry) <= e_y + HALF[dt] * np.abs(ry) + TINY[dt]).all()
    # in place, without what is not wanted, and the same bits
    r2 = v["resid"].clone()
    fm.fm_layer_norm(r2, None, **{**v, "resid": r2, "w": None, "b": None}, **draws, eps=EPS)
    assert torch.equal(r2, out)
    if norm:
        y2 = torch.empty_like(y)
        fm.fm_layer_norm(None, y2, **v, **draws, eps=EPS)
        assert torch.equal(y2, y)


@pytest.mark.parametrize("M,N,dt,stream,block,bias,norm,p", [c for c in CASES if c[6]])
def test_forward_to_8_bits(M, N, dt, stream, block, bias, norm, p):
    import torch
    say(f"layer norm to 8 bits M={M} N={N} {dt}/{stream}/{block} p={p}")
    v = _inputs(M, N, dt, stream, block, bias, norm, p, seed=5)
    draws = dict(p=p, rng=_rng() if p else None, draw=DRAW, row_begin=ROW)
    q, q_end = _buf((M, N), "int8")
    scale, scale_end = _buf((M,), "fp32")
    out = torch.empty(M, N, dtype=_dtype(stream), device="cuda:0")
    fm.fm_layer_norm(out, q, **v, **draws, eps=EPS, y_scale=scale)
    torch.cuda.synchronize()
    assert (q_end == -7).all() and (scale_end == -7).all()
    f = od.keep_factor(M, N, p, SEED, OFFSET, DRAW, ROW)
    ro, ry, rm, rr, mag = od.layer_norm(*(_host(v[k]) for k in ("block", "resid", "bias", "w", "b")), f, EPS)
    e_y = _bounds(v, ro, mag, rm, rr, ry)[2]
    top = np.abs(ry).max(axis=1)
    e_top = np.where(np.abs(ry) + e_y >= (top - e_y.max(axis=1))[:, None], e_y, 0).max(axis=1)
    s = _host(scale)
    assert (np.abs(s - top / 127) <= (e_top + 2 * U * top) / 127 + 2.0 ** -100).all()
    # a value is held to half a step
    lim = 0.5 * s[:, None] + e_y + 4 * U * np.abs(ry) + 2.0 ** -100
    assert (np.abs(_host(q) * s[:, None] - ry) <= lim).all()
    # the same rows as the quantisation of the fp32 values: those of the 16-bit y nearly
    y = torch.empty(M, N, dtype=_dtype(dt), device="cuda:0")
    fm.fm_layer_norm(None, y, **v, **draws, eps=EPS)
    q2, s2 = torch.empty_like(q), torch.empty_like(scale)
    fm.fm_quant_i8(y, q2, s2)
    assert (q2.int() - q.int()).abs().max() <= 2


@pytest.mark.parametrize("M,N,dt,stream,block,bias,norm,p", CASES)
def test_backward(M, N, dt, stream, block, bias, norm, p):
    import torch
    say(f"layer norm bwd M={M} N={N} {dt}/{stream}/{block} bias={bias} norm={norm} p={p}")
    v = _inputs(M, N, dt, stream, block, bias, norm, p, seed=2)
    has_block = block != "none"
    bt = block if has_block else stream
    rng = np.random.default_rng(3)
    d_y = _dev(rng.standard_normal((M, N)), dt) if norm else None
    d_out = _dev(rng.standard_normal((M, N)), stream)
    z = _host(v["resid"])
    mean = _dev(z.mean(1), "fp32") if norm else None
    rstd = _dev(1 / np.sqrt(z.var(1) + EPS), "fp32") if norm else None
    draws = dict(p=p, rng=_rng() if p else None, draw=DRAW, row_begin=ROW)
    got, ends = {}, []
    for name, shape, t, want in (("d_resid", (M, N), stream, True), ("d_block", (M, N), bt, has_block),
                                 ("d_bias", (N,), "fp32", bias), ("d_w", (N,), "fp32", norm),
                                 ("d_b", (N,), "fp32", norm)):
        if want:
            got[name], e = _buf(shape, t)
            ends.append(e)
    ws = torch.full((fm.fm_layer_norm_workspace_bytes(M, N) + 64,), 0xFF, dtype=torch.uint8, device="cuda:0")
    kw = dict(out=v["resid"] if norm else None, d_y=d_y, d_out=d_out, w=v["w"], **draws, mean=mean, rstd=rstd,
              ws=ws[:-64])
    fm.fm_layer_norm_bwd(got["d_resid"], got.get("d_block"), d_bias=got.get("d_bias"), d_w=got.get("d_w"),
                         d_b=got.get("d_b"), **kw)
    torch.cuda.synchronize()
    assert all((e == -7).all() for e in ends) and (ws[-64:] == 0xFF).all()
    f = od.keep_factor(M, N, p, SEED, OFFSET, DRAW, ROW)
    g, m = od.layer_norm_bwd(_host(d_y), _host(d_out), z, _host(mean), _host(rstd), _host(v["w"]), f)
    for name, x in got.items():
        t = {"d_resid": stream, "d_block": bt}.get(name, "fp32")
        u = {"d_resid": 48, "d_block": 51}.get(name, 48 + 3 + 100 + M / 256)
        lim = u * U * m[name] + HALF[t] * np.abs(g[name]) + TINY[t]
        assert (np.abs(_host(x) - g[name]) <= lim).all(), name
    # alone, and in place: the same bits
    for name in got:
        x = torch.empty_like(got[name])
        one = {k: x if k == name else None for k in ("d_resid", "d_block", "d_bias", "d_w", "d_b")}
        fm.fm_layer_norm_bwd(one.pop("d_resid"), one.pop("d_block"), **one, **kw)
        assert torch.equal(x, got[name]), name
    z2 = d_out.clone()
    fm.fm_layer_norm_bwd(z2, None, **{**kw, "d_out": z2, "ws": None})
    assert torch.equal(z2, got["d_resid"])


def test_gradient_against_differences():
    """The forward's own outputs, in fp32 but for y: a step h moves the sum of out * g by
    h times the gradient; out's fp32 rounding over h bounds the difference."""
    import torch
    M, N, p = 3, 64, 0.3
    rng = np.random.default_rng(8)
    block, resid, g = (rng.standard_normal((M, N)).astype(np.float32) for _ in range(3))
    draws = dict(p=p, rng=_rng(), draw=1)
    db = torch.empty(M, N, device="cuda:0")
    fm.fm_layer_norm_bwd(None, db, d_out=_dev(g, "fp32"), **draws)

    def f(b):
        out = torch.empty(M, N, device="cuda:0")
        fm.fm_layer_norm(out, None, block=_dev(b, "fp32"), resid=_dev(resid, "fp32"), **draws)
        return float((_host(out) * g.astype(np.float64)).sum())

    h = 0.25
    lim = 2 * (6 * U * 8 * np.abs(g).sum()) / h + 2 * U * 4
    for i, j in ((0, 0), (0, 9), (1, 33), (2, 63), (2, 17)):
        step = np.zeros_like(block)
        step[i, j] = h
        num = (f(block + step) - f(block)) / np.float64(np.float32(block[i, j] + h) - block[i, j])
        assert abs(num - float(db[i, j])) <= lim


def test_no_rows():
    import torch
    e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda:0")  # noqa: E731
    fm.fm_layer_norm(e(0, 64), e(0, 64), block=e(0, 64), resid=e(0, 64), w=e(64))
    d = [torch.full((64,), 3.0, device="cuda:0") for _ in range(3)]
    fm.fm_layer_norm_bwd(e(0, 64), e(0, 64), out=e(0, 64), d_y=e(0, 64), w=e(64), mean=e(0, t=torch.float32),
                         rstd=e(0, t=torch.float32), d_bias=d[0], d_w=d[1], d_b=d[2],
                         ws=fm.layer_norm_workspace(0, 64))
    assert all((x == 0).all() for x in d)


def test_what_is_dropped_has_no_part():
    """NaN and infinities in dropped places leave the rows as if they were not there."""
    import torch
    M, N, p = 4, 256, 0.5
    f = od.keep_factor(M, N, p, SEED, OFFSET, 0)
    x = np.random.default_rng(1).standard_normal((M, N)).astype(np.float32)
    bad = np.where(f == 0, np.where(np.arange(N) % 2, np.nan, np.inf), x).astype(np.float32)
    w = _dev(np.ones(N), "bf16")
    got = []
    for b in (x, bad):
        out, y = torch.empty(M, N, device="cuda:0"), torch.empty(M, N, dtype=torch.bfloat16, device="cuda:0")
        fm.fm_layer_norm(out, y, block=_dev(b, "fp32"), w=w, p=p, rng=_rng())
        g = torch.empty(M, N, device="cuda:0")
        fm.fm_layer_norm_bwd(None, g, d_out=_dev(b, "fp32"), p=p, rng=_rng())
        got.append((out, y, g))
    assert all(torch.equal(a, b) and torch.isfinite(a).all() for a, b in zip(*got))


@pytest.mark.parametrize("N", [128, 4096, 12288])
def test_rows_far_from_zero(N):
    """Mean 1000 and deviation 1: the variance is taken of the centred row, so it loses what
    the mean's own rounding (32 u of 1000) costs, not 10^6 times that."""
    import torch
    rng = np.random.default_rng(N)
    z = (1000 + rng.standard_normal((7, N))).astype(np.float32)
    w = _dev(np.ones(N), "bf16")
    mean, rstd = torch.empty(7, device="cuda:0"), torch.empty(7, device="cuda:0")
    y16 = torch.empty(7, N, dtype=torch.float16, device="cuda:0")
    fm.fm_layer_norm(None, y16, resid=_dev(z, "fp32"), w=w.half(), mean=mean, rstd=rstd)
    ref, m = z.astype(np.float64), z.astype(np.float64).mean(1)
    r = 1 / np.sqrt(ref.var(1) + EPS)
    off = 32 * U * 1005                      # of the mean
    assert (np.abs(_host(mean) - m) <= off).all()
    assert (np.abs(_host(rstd) / r - 1) <= off * off + 40 * U).all()
    yr = (ref - m[:, None]) * r[:, None]
    assert (np.abs(_host(y16) - yr) <= off * r[:, None] + 64 * U * np.abs(yr) + HALF["fp16"] * np.abs(yr) + 1e-7).all()


def test_rows_with_nan_are_their_own():
    import torch
    x = torch.randn(5, 512, device="cuda:0")
    x[1, 7], x[3, 500] = float("nan"), float("inf")
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda:0")
    y = torch.empty(5, 512, dtype=torch.bfloat16, device="cuda:0")
    q, s = torch.empty(5, 512, dtype=torch.int8, device="cuda:0"), torch.empty(5, device="cuda:0")
    fm.fm_layer_norm(None, y, resid=x, w=w)
    fm.fm_layer_norm(None, q, resid=x, w=w, y_scale=s)
    good = torch.tensor([0, 2, 4], device="cuda:0")
    assert torch.isfinite(y[good]).all() and torch.isfinite(s[good]).all()
    assert y[[1, 3]].isnan().all() and s[[1, 3]].isnan().all() and (q[[1, 3]] == 0).all()


def test_binding_refusals():
    import torch
    bf = torch.bfloat16
    e = lambda *s, t=bf: torch.empty(s, dtype=t, device="cuda:0")  # noqa: E731
    x, w, rng = e(4, 64), e(64), _rng()
    ok = dict(block=x, resid=x, w=w)
    fm.fm_layer_norm(e(4, 64), e(4, 64), **ok)
    f32 = torch.float32
    for bad in (dict(block=e(4, 72)), dict(block=x.cpu()), dict(block=e(64, 4).t()), dict(w=e(64, t=f32)),
                dict(b=e(32)), dict(bias=e(64, t=torch.float16)), dict(mean=e(4)), dict(rstd=e(3, t=f32)),
                dict(y_scale=e(4, t=f32)), dict(p=0.1, rng=rng.int()), dict(p=0.1, rng=rng.cpu()),
                dict(p=0.1, rng=e(3, t=torch.int64))):
        with pytest.raises((ValueError, TypeError)):
            fm.fm_layer_norm(e(4, 64), e(4, 64), **{**ok, **bad})
    with pytest.raises(OverflowError):
        fm.fm_layer_norm(e(4, 64), e(4, 64), **ok, p=0.1, rng=rng, draw=2 ** 63)
    for bad in (dict(p=0.1), dict(p=1.5, rng=rng), dict(p=0.5, rng=rng, row_begin=-1)):
        with pytest.raises(fm.FluxMIError):
            fm.fm_layer_norm(e(4, 64), e(4, 64), **ok, **bad)
    with pytest.raises(ValueError):
        fm.fm_layer_norm(e(4, 64), e(4, 64))
    with pytest.raises(ValueError):
        fm.fm_layer_norm_bwd(e(4, 64), None)
    with pytest.raises(fm.FluxMIError):
        fm.fm_layer_norm_bwd(e(4, 64), None, out=x, d_y=x, w=w, mean=e(4, t=f32), rstd=e(4, t=f32),
                             d_w=e(64, t=f32))
