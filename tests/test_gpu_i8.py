"""fm_quant_i8, fm_gemm_i8 and fm_linear_i8 against the float64 definitions.

8-bit rows of 16-bit values are exact: 127 x has at most 18 bits, so the quotient is
rounded once, at a half to even, as the definition's is; of 32-bit values 127 x is
rounded too, which can only matter within 2^-22 of a half relative to 127.  Scales are one division.

Products, in units u = 2^-24: the sum is exact, its conversion, the scales' product, theirs
and the bias's sum are a rounding each: 4 u of the magnitudes.  Activations: slope at most
1.13, and for the exponential of an argument z an error of 2 |z| + 8 u of the result
(z = 2 * 0.798 (x + 0.0447 x^3) with 4 u of its own; z = x)."""
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


def _dev(a, dt="fp32"):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0").to(_dtype(dt))


def _host(t):
    return None if t is None else t.double().cpu().numpy()


def _sentinels(shape, t):
    import torch
    n = int(np.prod(shape))
    flat = torch.full((n + 64,), -7, device="cuda:0", dtype=t)
    return flat[:n].view(shape), flat[n:]


@pytest.mark.parametrize("M,N,dt", [(1, 8, "bf16"), (61, 2816, "fp16"), (7, 8184, "bf16"), (3, 8192, "fp16"),
                                    (5, 8200, "fp32"), (9, 49152, "bf16"), (2000, 64, "fp32"), (2, 100008, "fp16")])
def test_quant(M, N, dt):
    import torch
    say(f"quant M={M} N={N} {dt}")
    rng = np.random.default_rng(N)
    x = _dev(rng.standard_normal((M, N)).astype(np.float32) * np.exp(rng.standard_normal((M, 1)) * 4), dt)
    if M > 1:
        x[1, :3] = torch.tensor([4.0, 2.0, -2.0])     # halves of steps
        x[1] = x[1].clamp(-4, 4)
    q, q_end = _sentinels((M, N), torch.int8)
    s, s_end = _sentinels((M,), torch.float32)
    fm.fm_quant_i8(x, q, s)
    torch.cuda.synchronize()
    assert (q_end == -7).all() and (s_end == -7).all()
    rq, rs = od.quant(_host(x))
    rs = np.where(np.isnan(rs), np.nan, np.abs(_host(x)).max(1).astype(np.float32) / np.float32(127))
    assert np.array_equal(s.cpu().numpy(), rs.astype(np.float32), equal_nan=True)   # (fp16 rows may overflow)
    off = np.abs(q.cpu().numpy() - rq)
    if dt == "fp32":
        near = np.abs(np.abs(127 * _host(x) / np.abs(_host(x)).max(1)[:, None]) % 1 - 0.5) < 127 * 2.0 ** -22
        assert (off[~near] == 0).all() and off.max() <= 1
    else:
        assert (off == 0).all()


def test_quant_of_strange_rows():
    import torch
    x = torch.randn(9, 264, device="cuda:0")
    x[0] = 0
    x[1, 5], x[2, 263], x[3, 0] = float("nan"), float("inf"), float("-inf")
    x[4] *= 1e-32
    x[5, 7] = 2.0 ** 120
    x[6, 7] = -2.0 ** 119.9
    x[7] *= 2.0 ** -98
    q, s = torch.empty(9, 264, dtype=torch.int8, device="cuda:0"), torch.empty(9, device="cuda:0")
    fm.fm_quant_i8(x, q, s)
    rq, rs = od.quant(_host(x))
    # 32-bit values: 127 x is rounded, and a value next to a half may go the other way
    assert np.abs(q.cpu().numpy() - rq).max() <= 1
    for i in (0, 1, 2, 3, 4, 5):
        assert (q[i] == 0).all()
    assert s[[1, 2, 3, 5]].isnan().all() and (s[[0, 4]] == 0).all()
    assert np.allclose(_host(s)[6:], rs[6:], rtol=2 * U)
    none, at = torch.empty(3, 0, device="cuda:0"), torch.full((3,), 9.0, device="cuda:0")
    fm.fm_quant_i8(none, torch.empty(3, 0, dtype=torch.int8, device="cuda:0"), at)
    assert (at == 0).all()


# M: one token to several tiles, odd ones at every variant's edge; K: less than a step
# of the loop, its tails, and long; N: 8 columns, ragged tiles
SIZES = [(1, 8, 16), (1, 4096, 1024), (2, 264, 272), (3, 1000, 4112), (5, 40, 48), (8, 2816, 4096), (13, 136, 80),
         (16, 520, 144), (17, 264, 2064), (31, 72, 112), (32, 1024, 512), (33, 4104, 400), (45, 1536, 3104),
         (48, 256, 6160), (61, 2816, 1040), (64, 512, 1024), (65, 264, 96), (97, 1032, 656), (127, 8, 4096),
         (128, 128, 128), (129, 136, 1552), (200, 2824, 400), (255, 256, 272), (257, 520, 2064), (509, 2816, 1024),
         (700, 1304, 160), (1023, 2048, 144), (2049, 264, 80), (1, 16, 131056), (3, 8, 0), (300, 40, 0)]


def _case(M, N, K, dt, bias, seed):
    rng = np.random.default_rng(seed)
    A = rng.integers(-128, 128, (M, K)).astype(np.int8)
    W = rng.integers(-128, 128, (N, K)).astype(np.int8)
    sa = (0.5 + rng.random(M)).astype(np.float32)
    sw = ((0.5 + rng.random(N)) / (5461 * max(K, 1) ** 0.5)).astype(np.float32)
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    return A, sa, W, sw, b


def _limit(ref, v, mag, act, to):
    e = 4 * U * mag
    z = {0: 0 * v, 1: 0 * v, 2: 1.6 * (np.abs(v) + 0.0447 * np.abs(v) ** 3), 3: np.abs(v)}[act]
    rel = 0 if act < 2 else (10 * z + 8) * U if act == 2 else (2 * z + 8) * U
    return 1.13 * e + rel * np.abs(ref) + HALF[to] * np.abs(ref) + TINY[to]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_gemm(M, N, K):
    import torch
    for i, (dt, to, bias, act) in enumerate((("bf16", "bf16", 1, 2), ("fp16", "fp32", 0, 0), ("bf16", "fp32", 1, 3),
                                             ("fp16", "fp16", 1, 1))):
        say(f"gemm i8 M={M} N={N} K={K} {dt}->{to} bias={bias} act={act}")
        A, sa, W, sw, b = _case(M, N, K, dt, bias, seed=M + N + i)
        C, end = _sentinels((M, N), _dtype(to))
        bd = _dev(b, dt)
        fm.fm_gemm_i8(torch.from_numpy(A).cuda(), _dev(sa), torch.from_numpy(W).cuda(), _dev(sw), C, bias=bd,
                      act=act)
        torch.cuda.synchronize()
        assert (end == -7).all()
        ref, v, mag = od.gemm_i8(A, sa.astype(np.float64), W, sw.astype(np.float64), _host(bd), act)
        err = np.abs(_host(C) - ref)
        assert (err <= _limit(ref, v, mag, act, to)).all(), (dt, to, err.max())


# Sizes whose rounds choose each macro-tile, with one to nine K steps, whole and ragged
# ones, and edges in both directions.
TILED = {
    "64x64": [(301, 520, 128), (301, 520, 16), (301, 520, 256), (301, 520, 144), (301, 520, 384), (301, 520, 272),
              (301, 520, 400), (301, 520, 1040)],
    "64x128": [(3599, 520, 128), (3599, 520, 16), (3599, 520, 144), (3599, 520, 272), (3599, 520, 400), (1853, 520, 1040)],
    "128x128": [(3599, 520, 1024), (3599, 520, 1040)],
    "128x192": [(2920, 2056, 384), (2920, 2056, 272), (2920, 2056, 400), (7285, 520, 656), (7285, 520, 1024), (7285, 520, 1040)],
    "256x128": [(5442, 1032, 384), (5442, 1032, 272), (5442, 1032, 400), (398, 12296, 656), (398, 12296, 1024), (398, 12296, 1040)],
    "256x192": [(5830, 2056, 128), (5830, 2056, 16), (5830, 2056, 256), (5830, 2056, 144), (4860, 2056, 384), (4860, 2056, 272),
                (4860, 2056, 400), (7285, 1032, 656), (7285, 1032, 1024), (7285, 1032, 1040)],
    "256x256": [(6800, 2056, 128), (6800, 2056, 16), (980, 12296, 256), (980, 12296, 144), (980, 12296, 384), (980, 12296, 272),
                (883, 12296, 400), (883, 12296, 656), (786, 12296, 1024), (786, 12296, 1040)],
}


@pytest.mark.parametrize("M,N,K,tile", [(*s, t) for t, ss in TILED.items() for s in ss])
def test_gemm_of_every_tile(M, N, K, tile):
    """Against float64 sums on the GPU (exact: below 2^53), by plain matrix products."""
    import torch
    say(f"gemm i8 tile {tile}: M={M} N={N} K={K}")
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + K)
    A = torch.randint(-128, 128, (M, K), generator=g, device="cuda").to(torch.int8)
    W = torch.randint(-128, 128, (N, K), generator=g, device="cuda").to(torch.int8)
    sa = 0.5 + torch.rand(M, generator=g, device="cuda")
    sw = (0.5 + torch.rand(N, generator=g, device="cuda")) / (5461 * K ** 0.5)
    sums = A.double() @ W.double().t().contiguous()
    for dt, to, act in ((torch.bfloat16, torch.bfloat16, 2), (torch.float16, torch.float32, 0)):
        b = torch.randn(N, generator=g, device="cuda").to(dt) if act else None
        C, end = _sentinels((M, N), to)
        fm.fm_gemm_i8(A, sa, W, sw, C, bias=b, act=act)
        v = sums * (sa.double()[:, None] * sw.double())
        mag = v.abs()
        if act:
            v, mag = v + b.double(), mag + b.double().abs()
            u = 0.7978845608028654 * (v + 0.044715 * v ** 3)
            ref, z = 0.5 * v * (1 + torch.tanh(u)), 1.6 * (v.abs() + 0.0447 * v.abs() ** 3)
        else:
            ref, z = v, 0 * v
        name = {torch.bfloat16: "bf16", torch.float32: "fp32"}[to]
        lim = 1.13 * 4 * U * mag + (10 * z + 8) * U * ref.abs() + HALF[name] * ref.abs() + TINY[name]
        assert (end == -7).all()
        assert ((C.double() - ref).abs() <= lim).all(), (to, act)


@pytest.mark.parametrize("N", [2040, 2056, 4104, 6152, 8192, 12296])
@pytest.mark.parametrize("M", [1, 7, 8, 9, 16, 17, 32, 33, 48, 49, 64])
def test_few_rows(M, N):
    """Every number of rows at an edge, with one to six eights of columns a block, over k of less
    than a step, whole steps, tails, and more steps than a wave's ring holds: the product
    against float64 sums on the GPU, and the layer on 16-bit rows against the product."""
    import torch
    say(f"few rows M={M} N={N}")
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N)
    for K in (16, 128, 1040, 1536, 4112, 6144):
        x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
        q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        fm.fm_quant_i8(x, q, s)
        W = torch.randint(-128, 128, (N, K), generator=g, device="cuda").to(torch.int8)
        sw = (0.5 + torch.rand(N, generator=g, device="cuda")) / (70 * K ** 0.5)
        C, end = _sentinels((M, N), torch.float32)
        fm.fm_gemm_i8(q, s, W, sw, C)
        ref = (q.double() @ W.double().t().contiguous()) * (s.double()[:, None] * sw.double())
        assert (end == -7).all() and ((C.double() - ref).abs() <= 4 * U * ref.abs() + 1e-38).all(), K
        L, end = _sentinels((M, N), torch.float32)
        fm.fm_linear_i8(x, W, sw, L, ws=fm.linear_i8_workspace(M, K))
        assert (end == -7).all() and torch.equal(L, C), K


def test_gemm_of_the_largest_sums():
    """Every product 2^14: the sum of 131056 of them is 2^31 less 2^18."""
    import torch
    for M in (1, 40, 300):
        A = torch.full((M, 131056), -128, dtype=torch.int8, device="cuda:0")
        W = torch.full((16, 131056), -128, dtype=torch.int8, device="cuda:0")
        C = torch.empty(M, 16, device="cuda:0")
        fm.fm_gemm_i8(A, torch.ones(M, device="cuda:0"), W, torch.ones(16, device="cuda:0"), C)
        assert (C.double() == float(np.float32(131056 * 16384))).all()


@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear(M, N, K):
    import torch
    for i, (dt, to, bias, act) in enumerate((("bf16", "bf16", 1, 2), ("fp16", "fp32", 0, 0))):
        say(f"linear i8 M={M} N={N} K={K} {dt}->{to}")
        _, _, W, sw, b = _case(M, N, K, dt, bias, seed=M + N + i)
        x = _dev(np.random.default_rng(K).standard_normal((M, K)).astype(np.float32), dt)
        if M > 2 and K:
            x[1] = 0
            x[2, K - 1] = float("nan")
        Wd, swd, bd = torch.from_numpy(W).cuda(), _dev(sw), _dev(b, dt)
        n = fm.fm_linear_i8_workspace_bytes(M, K)
        ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda:0")
        C, end = _sentinels((M, N), _dtype(to))
        fm.fm_linear_i8(x, Wd, swd, C, bias=bd, act=act, ws=ws[:n])
        torch.cuda.synchronize()
        assert (end == -7).all() and (ws[n:] == 0xFF).all()
        rq, rs = od.quant(_host(x))
        ref, v, mag = od.gemm_i8(rq, rs, W, sw.astype(np.float64), _host(bd), act)
        got = _host(C)
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        fine = ~np.isnan(ref)
        # the row's scale is rounded once more
        lim = _limit(ref, v, mag, act, to) + 1.13 * U * mag
        assert (np.abs(got - ref)[fine] <= lim[fine]).all()
        # the same bits as the two calls
        q, s = torch.empty(M, K, dtype=torch.int8, device="cuda:0"), torch.empty(M, device="cuda:0")
        fm.fm_quant_i8(x, q, s)
        C2 = torch.empty_like(C)
        fm.fm_gemm_i8(q, s, Wd, swd, C2, bias=bd, act=act)
        assert torch.equal(C.nan_to_num(7.0), C2.nan_to_num(7.0))


def test_no_rows_and_refusals():
    import torch
    i8, f32, bf = torch.int8, torch.float32, torch.bfloat16
    e = lambda *s, t=bf: torch.empty(s, dtype=t, device="cuda:0")  # noqa: E731
    ws = fm.linear_i8_workspace(4, 64)
    fm.fm_quant_i8(e(0, 64), e(0, 64, t=i8), e(0, t=f32))
    fm.fm_gemm_i8(e(0, 64, t=i8), e(0, t=f32), e(32, 64, t=i8), e(32, t=f32), e(0, 32))
    fm.fm_linear_i8(e(0, 64), e(32, 64, t=i8), e(32, t=f32), e(0, 32), ws=ws)
    good = dict(A=e(4, 64, t=i8), a_scale=e(4, t=f32), W=e(32, 64, t=i8), w_scale=e(32, t=f32), C=e(4, 32))
    fm.fm_gemm_i8(**good)
    for bad in (dict(A=e(4, 64)), dict(A=e(4, 64, t=torch.uint8)), dict(a_scale=e(5, t=f32)), dict(a_scale=e(4)),
                dict(W=e(64, 32, t=i8).t()), dict(W=e(32, 48, t=i8)), dict(w_scale=e(31, t=f32)),
                dict(C=e(4, 40)), dict(bias=e(16)), dict(A=good["A"].cpu()),
                dict(C=e(4, 32, t=torch.float64))):
        with pytest.raises((ValueError, TypeError)):
            fm.fm_gemm_i8(**{**good, **bad})
    for bad in (dict(act=7), dict(bias=e(32, t=f32), C=e(4, 32, t=f32)), dict(bias=e(32, t=torch.float16))):
        with pytest.raises(fm.FluxMIError):
            fm.fm_gemm_i8(**{**good, **bad})
    lin = dict(X=e(4, 64), W=good["W"], w_scale=good["w_scale"], C=good["C"], ws=ws)
    fm.fm_linear_i8(**lin)
    for bad in (dict(ws=None), dict(ws=ws[:64]), dict(X=e(4, 64, t=f32))):
        with pytest.raises(fm.FluxMIError):
            fm.fm_linear_i8(**{**lin, **bad})
    for bad in (dict(X=e(4, 64).cpu()), dict(bias=e(32, t=f32)), dict(W=e(32, 64))):
        with pytest.raises((ValueError, TypeError)):
            fm.fm_linear_i8(**{**lin, **bad})
    with pytest.raises((ValueError, TypeError)):
        fm.fm_quant_i8(e(4, 64), e(4, 64), e(4, t=f32))


def test_extremes_of_scales():
    """NaN, infinite and zero scales stay in their rows and columns."""
    import torch
    for M in (3, 70, 300):
        A = torch.ones(M, 64, dtype=torch.int8, device="cuda:0")
        W = torch.ones(24, 64, dtype=torch.int8, device="cuda:0")
        sa, sw = torch.ones(M, device="cuda:0"), torch.ones(24, device="cuda:0")
        sa[1], sw[5], sw[6] = float("nan"), float("inf"), 0.0
        C = torch.empty(M, 24, device="cuda:0")
        fm.fm_gemm_i8(A, sa, W, sw, C)
        ref = 64.0 * sa[:, None] * sw
        assert torch.equal(C.nan_to_num(7, 8), ref.nan_to_num(7, 8))


@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("M,K", [(4, 512), (4, 16384), (40, 512), (70, 512), (300, 512)])
def test_nan_under_every_activation(M, K, act):
    """A row with a NaN, or too large for its scale, and a row or column with a NaN scale stay NaN
    whatever the activation: rows quantised in the product's blocks, before it, and on tiles."""
    import torch
    N = 72
    x = torch.randn(M, K, device="cuda:0").bfloat16()
    x[1, K - 1], x[2, 3] = float("nan"), 2.0 ** 120
    W = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda:0")
    sw, bias = 0.01 * torch.rand(N, device="cuda:0") + 1e-3, torch.randn(N, device="cuda:0").bfloat16()
    sw[5] = float("nan")
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda:0")
    bad[1:3], bad[:, 5] = True, True
    C = torch.empty(M, N, device="cuda:0")
    fm.fm_linear_i8(x, W, sw, C, bias=bias, act=act, ws=fm.linear_i8_workspace(M, K))
    assert torch.equal(C.isnan(), bad) and not C.isinf().any()
    q, s = torch.empty(M, K, dtype=torch.int8, device="cuda:0"), torch.empty(M, device="cuda:0")
    fm.fm_quant_i8(x, q, s)
    for to in (torch.float32, torch.bfloat16):
        C = torch.empty(M, N, dtype=to, device="cuda:0")
        fm.fm_gemm_i8(q, s, W, sw, C, bias=bias, act=act)
        assert torch.equal(C.isnan(), bad) and not C.isinf().any()


# Sizes with more tiles than blocks (two a unit of the two small ones) and an uneven last round,
# over whole and ragged steps of k.
ROUNDS = {
    "64x64": [(6529, 520, 384), (6529, 520, 1040), (6529, 520, 144)],
    "64x128": [(7233, 520, 384), (7233, 520, 400), (7169, 1032, 1024), (513, 12296, 656)],
    "128x128": [(513, 12296, 1024), (513, 12296, 1040)],
    "128x192": [(14529, 1032, 1024), (14529, 1032, 656)],
    "256x128": [(13057, 1032, 384), (13057, 1032, 272)],
    "256x192": [(1409, 12296, 1024), (11521, 2056, 400)],
    "256x256": [(1793, 12296, 1024), (1857, 12296, 400), (11777, 2056, 272), (7425, 4104, 128)],
}


@pytest.mark.parametrize("M,N,K,tile", [(*s, t) for t, ss in ROUNDS.items() for s in ss])
def test_blocks_that_take_several_tiles(M, N, K, tile):
    """The next tile's loads land where the last one's results were staged; every element."""
    test_gemm_of_every_tile(M, N, K, tile)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K", [(1, 16384), (1, 16368), (1, 15888), (2, 8192), (3, 5120), (4, 4096), (5, 3056), (6, 2560),
                                 (7, 2048), (8, 2048), (8, 2032), (8, 1552), (8, 16)])
def test_most_that_a_block_quantises(M, K, dt):
    """Up to 32 pieces of 512 values, the last one ragged too: codes and scales of the
    definition (exact for 16-bit rows), so the same bits as of the two calls, and the float64 product."""
    import torch
    N = 520
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K)
    x = (torch.randn(M, K, generator=g, device="cuda") * (1 + torch.arange(M, device="cuda")[:, None])).to(_dtype(dt))
    x[M - 1, K - 1] = 40.0                   # a row's largest in its last piece
    W = torch.randint(-128, 128, (N, K), generator=g, device="cuda").to(torch.int8)
    sw = (0.5 + torch.rand(N, generator=g, device="cuda")) / (70 * K ** 0.5)
    L, end = _sentinels((M, N), torch.float32)
    fm.fm_linear_i8(x, W, sw, L, ws=fm.linear_i8_workspace(M, K))
    assert (end == -7).all()
    rq, rs = od.quant(_host(x))
    ref = od.gemm_i8(rq, rs, W.cpu().numpy(), _host(sw), None, 0)[0]
    assert (np.abs(_host(L) - ref) <= 5 * U * np.abs(ref) + 1e-38).all()
    q, s, C = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"), torch.empty_like(L)
    fm.fm_quant_i8(x, q, s)
    fm.fm_gemm_i8(q, s, W, sw, C)
    assert torch.equal(L, C)
