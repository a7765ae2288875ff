"""fm_dropout: the mask is the definition's, bit for bit, and what is kept is one product
with a scale that is rounded once: 2 u of its magnitude (u = 2^-24), and half a step
(eps / 2) of a 16-bit output."""
import numpy as np
import pytest

import tile_gemm_communication_amd as fm
from gpu_util import say
from oracle import dense as od

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": U}
TINY = {"bf16": 1e-38, "fp16": 2.0 ** -25, "fp32": 1e-38}


@pytest.fixture(autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _rng(seed, offset):
    import torch
    wrap = lambda x: x - 2 ** 64 if x >= 2 ** 63 else x  # noqa: E731
    return torch.tensor([wrap(seed), wrap(offset)], dtype=torch.int64, device="cuda:0")


@pytest.mark.parametrize("M,N,dt,p,seed,offset,draw,row,col", [
    (1, 8, "bf16", 0.5, 1, 2, 0, 0, 0),
    (61, 2816, "fp16", 0.1, 7, 2 ** 32 - 1, 1, 0, 0),
    (3, 520, "fp32", 0.9, 2 ** 64 - 1, 2 ** 64 - 1, 5, 2 ** 32 - 3, 2 ** 34 - 520),
    (1000, 24, "bf16", 0.3, 2 ** 63, 9, -4, 100, 8),
    (257, 1032, "fp32", 0.01, 5, 6, 0, 0, 16),
    (4, 49152, "bf16", 0.1, 11, 0, 3, 77, 0),
    (5, 64, "fp16", 0.0, 1, 1, 0, 0, 0),
    (5, 64, "fp16", 2.0 ** -18, 1, 1, 0, 0, 0),
    (5, 64, "bf16", 1.0, 1, 1, 0, 0, 0),
    (70000, 8, "fp16", 0.2, 3, 3, 0, 0, 0),
])
def test_dropout(M, N, dt, p, seed, offset, draw, row, col):
    import torch
    say(f"dropout M={M} N={N} {dt} p={p}")
    x = torch.randn(M, N, device="cuda:0").to(_dtype(dt))
    x[x == 0] = 1
    flat = torch.full((M * N + 8,), -7.0, device="cuda:0", dtype=x.dtype)
    y = flat[:M * N].view(M, N)
    rng = _rng(seed, offset)
    kw = dict(draw=draw, row_begin=row, col_begin=col)
    fm.fm_dropout(x, y, p, rng, **kw)
    torch.cuda.synchronize()
    assert (flat[M * N:] == -7).all()
    f = od.keep_factor(M, N, p, seed, offset, draw, row, col)
    got, ref = y.double().cpu().numpy(), x.double().cpu().numpy() * f
    assert np.array_equal(got != 0, f != 0)
    assert (np.abs(got - ref) <= (2 * U + HALF[dt]) * np.abs(ref) + TINY[dt]).all()
    assert rng.tolist() == _rng(seed, offset).tolist()
    fm.fm_dropout(x, x, p, rng, **kw)           # in place
    assert torch.equal(x, y)


def test_what_is_dropped_is_zero_whatever_it_was():
    import torch
    f = od.keep_factor(8, 64, 0.5, 1, 1)
    x = torch.full((8, 64), float("nan"), device="cuda:0")
    x[:, ::2] = float("inf")
    y = torch.empty_like(x)
    fm.fm_dropout(x, y, 0.5, _rng(1, 1))
    got = y.cpu().numpy()
    assert (got[f == 0] == 0).all() and not np.isfinite(got[f != 0]).any()


def test_parts_draw_what_the_whole_draws():
    import torch
    x = torch.randn(96, 512, device="cuda:0")
    rng, whole = _rng(4, 5), torch.empty_like(x)
    fm.fm_dropout(x, whole, 0.4, rng, draw=3)
    for r0, r1, c0, c1 in ((0, 48, 0, 512), (48, 96, 0, 256), (30, 31, 8, 16), (0, 96, 504, 512)):
        part = x[r0:r1, c0:c1].clone(memory_format=torch.contiguous_format)   # not x itself
        fm.fm_dropout(part, part, 0.4, rng, draw=3, row_begin=r0, col_begin=c0)
        assert torch.equal(part, whole[r0:r1, c0:c1])
    # and the layer norm's dropout is the same
    out = torch.empty_like(x)
    fm.fm_layer_norm(out, None, block=x, p=0.4, rng=rng, draw=3)
    assert torch.equal(out, whole)


def test_another_stream_and_refusals():
    import torch
    x, rng = torch.randn(64, 256, device="cuda:0"), _rng(1, 2)
    a, b = torch.empty_like(x), torch.empty_like(x)
    fm.fm_dropout(x, a, 0.3, rng)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fm.fm_dropout(x, b, 0.3, rng, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b)
    for bad in (dict(x=x.cpu()), dict(x=x.t()), dict(x=x[0]), dict(x=x.double()), dict(y=a[:1]),
                dict(y=a.half()), dict(rng=rng.float()), dict(rng=rng[:1]), dict(rng=3)):
        kw = {**dict(x=x, y=a, p=0.3, rng=rng), **bad}
        with pytest.raises((ValueError, TypeError)):
            fm.fm_dropout(**kw)
    for bad in (dict(p=2.0), dict(rng=None), dict(col_begin=4), dict(row_begin=2 ** 32)):
        with pytest.raises(fm.FluxMIError):
            fm.fm_dropout(**{**dict(x=x, y=a, p=0.3, rng=rng), **bad})
