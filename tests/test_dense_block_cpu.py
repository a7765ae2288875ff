"""The operators in a dense block, on the CPU side: the float64 definitions against
published values, hand-written ones and differences, and every refusal of the C
interface (these calls return during validation, so no GPU is touched)."""
import ctypes

import numpy as np
import pytest

import tile_gemm_communication_amd as fm
from oracle import dense as od

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(16)]
ODD = ctypes.c_void_p(0x10008)
ODD2 = ctypes.c_void_p(0x10002)
ODD4 = ctypes.c_void_p(0x10004)
BIG = 1 << 50
OK, INV, UNS = fm.FM_OK, fm.FM_ERR_INVALID_ARG, fm.FM_ERR_UNSUPPORTED


# -- definitions -----------------------------------------------------------------

@pytest.mark.parametrize("counter,key,want", [
    ((0,) * 4, (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_generator_against_published_values(counter, key, want):
    """The known answers that were published with Philox4x32-10."""
    assert tuple(int(x) for x in od.philox4x32(counter, key)) == want


def test_mask_is_a_function_of_the_place():
    whole = od.keep_factor(12, 64, 0.3, 5, 7, draw=2)
    assert np.array_equal(od.keep_factor(5, 24, 0.3, 5, 7, 2, row_begin=4, col_begin=16), whole[4:9, 16:40])
    assert np.array_equal(od.keep_factor(12, 64, 0.3, 5, 9), whole)
    assert not np.array_equal(od.keep_factor(12, 64, 0.3, 5, 10), whole)
    assert np.array_equal(od.keep_factor(12, 64, 0.3, 5, 2 ** 64 - 1, draw=10), whole)
    # 4 sigma of a binomial share, and the scale makes the mean 1
    big = od.keep_factor(400, 400, 0.3, 1, 1)
    assert abs((big > 0).mean() - 0.7) < 4 * np.sqrt(0.21 / 160000)
    assert np.isclose(big.max(), 65536 / od.threshold(0.3))


@pytest.mark.parametrize("p,t", [(0.0, 65536), (2 ** -18, 65536), (0.5, 32768), (1.0, 0), (0.1, 58982)])
def test_threshold(p, t):
    assert od.threshold(p) == t


@pytest.mark.parametrize("parts", ["all", "no norm", "no block", "no resid"])
def test_layer_norm_gradient_against_differences(parts):
    rng = np.random.default_rng(4)
    M, N, eps = 5, 16, 1e-3
    v = {"block": rng.standard_normal((M, N)), "resid": rng.standard_normal((M, N)) + 2,
         "bias": rng.standard_normal(N), "w": rng.standard_normal(N), "b": rng.standard_normal(N)}
    factor = od.keep_factor(M, N, 0.4, 3, 1)
    if parts == "no norm":
        v["w"] = v["b"] = None
    if parts == "no block":
        v["block"] = v["bias"] = factor = None
    if parts == "no resid":
        v["resid"] = None
    d_y, d_out = rng.standard_normal((M, N)), rng.standard_normal((M, N))

    def f(v):
        out, y, *_ = od.layer_norm(v["block"], v["resid"], v["bias"], v["w"], v["b"], factor, eps)
        return (out * d_out).sum() + (0.0 if y is None else (y * d_y).sum())

    out, _, mean, rstd, _ = od.layer_norm(v["block"], v["resid"], v["bias"], v["w"], v["b"], factor, eps)
    g, _ = od.layer_norm_bwd(d_y if v["w"] is not None else None, d_out, out, mean, rstd, v["w"], factor)
    for name, x in v.items():
        if x is None:
            continue
        for at in np.ndindex(x.shape):
            h = np.zeros_like(x)
            h[at] = 1e-5
            num = (f(dict(v, **{name: x + h})) - f(dict(v, **{name: x - h}))) / 2e-5
            assert abs(num - g["d_" + name][at]) < 1e-7, (name, at)


def test_rows_in_8_bits_by_hand():
    x = np.array([[2.0, 1.0, -0.5, 0.0], [0.0, 0.0, 0.0, 0.0], [1e-31, 0, 0, 0],
                  [np.inf, 1, 0, 0], [np.nan, 1, 0, 0], [-254.0, 3.0, 5.0, 1.0]])
    q, s = od.quant(x)
    assert q.tolist() == [[127, 64, -32, 0], [0] * 4, [0] * 4, [0] * 4, [0] * 4, [-127, 2, 2, 0]]
    assert np.allclose(s[[0, 1, 2, 5]], [2 / 127, 0, 0, 2]) and np.isnan(s[[3, 4]]).all()


def test_8_bit_product_by_hand():
    C, v, mag = od.gemm_i8(np.array([[1, -2]]), np.array([0.5]), np.array([[3, 4], [5, 6]]),
                           np.array([2.0, 1.0]), np.array([1.0, 8.0]), 1)
    assert C.tolist() == [[0.0, 4.5]] and v.tolist() == [[-4.0, 4.5]] and mag.tolist() == [[6.0, 11.5]]


# -- refusals ---------------------------------------------------------------------

pytestmark = pytest.mark.usefixtures("built_library")


def drop_call(dt=1, M=4, N=64, x=P[0], p=0.1, rng=P[1], draw=0, row=0, col=0, y=P[2]):
    return fm.lib().fm_dropout(dt, M, N, x, p, rng, draw, row, col, y, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=3), UNS), (dict(M=-1), INV), (dict(N=-8), INV), (dict(N=12), INV), (dict(M=1 << 31), UNS),
    (dict(N=1 << 31), UNS), (dict(p=-0.1), INV), (dict(p=1.1), INV), (dict(p=float("nan")), INV),
    (dict(rng=None), INV), (dict(rng=ODD4), INV), (dict(row=-1), INV), (dict(col=-8), INV),
    (dict(col=4), INV), (dict(row=(1 << 32) - 3), UNS), (dict(col=(1 << 34) - 56), UNS),
    (dict(x=None), INV), (dict(y=None), INV), (dict(x=ODD), INV), (dict(y=ODD), INV),
    (dict(M=0, x=None, y=None), OK), (dict(N=0, x=None, y=None), OK),
    (dict(M=0, p=0.0, rng=None), OK), (dict(M=0, p=0.5, rng=None), INV),
])
def test_dropout_refusals(kw, want):
    assert drop_call(**kw) == want


def ln_call(dt=1, sd=1, bd=2, M=4, N=64, block=P[0], resid=P[1], bias=P[2], w=P[3], b=P[4], p=0.1,
            rng=P[5], draw=0, row=0, eps=1e-5, out=P[6], y=P[7], y_scale=None, mean=P[8], rstd=P[9]):
    return fm.lib().fm_layer_norm(dt, sd, bd, M, N, block, resid, bias, w, b, p, rng, draw, row, eps,
                                  out, y, y_scale, mean, rstd, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), UNS), (dict(dt=3), UNS), (dict(sd=0), UNS), (dict(bd=0), UNS), (dict(sd=3), UNS),
    (dict(M=-1), INV), (dict(N=-8), INV), (dict(N=4), INV), (dict(N=16392), UNS), (dict(M=1 << 31), UNS),
    (dict(p=-1.0), INV), (dict(p=2.0), INV), (dict(rng=None), INV), (dict(rng=ODD4), INV),
    (dict(row=-1), INV), (dict(row=1 << 32), UNS), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(y=None), INV), (dict(w=None), INV), (dict(w=None, y=None), INV),       # b without w
    (dict(w=None, y=None, b=None), INV),                                       # mean without w
    (dict(w=None, y=None, b=None, mean=None), INV), (dict(w=None, y=None, b=None, rstd=None), INV),
    (dict(w=None, y=None, b=None, mean=None, rstd=None, y_scale=P[10]), INV),
    (dict(w=None, y=None, b=None, mean=None, rstd=None, out=None), INV),
    (dict(block=None), INV), (dict(block=None, bias=None), INV),                 # p without block
    (dict(block=None, bias=None, p=0.0, resid=None), INV), (dict(block=None, p=0.0), INV),
    (dict(block=ODD), INV), (dict(resid=ODD), INV), (dict(bias=ODD), INV), (dict(w=ODD), INV),
    (dict(b=ODD), INV), (dict(out=ODD), INV), (dict(y=ODD), INV), (dict(y_scale=ODD2), INV),
    (dict(mean=ODD2), INV), (dict(rstd=ODD2), INV),
    (dict(M=0, block=None, resid=None, out=None, y=None), OK), (dict(N=0), OK),
])
def test_layer_norm_refusals(kw, want):
    assert ln_call(**kw) == want


def ln_bwd_call(dt=1, sd=1, bd=2, M=4, N=64, d_y=P[0], d_out=P[1], out=P[2], mean=P[3], rstd=P[4],
                w=P[5], p=0.1, rng=P[6], draw=0, row=0, d_resid=P[7], d_block=P[8], d_bias=P[9],
                d_w=P[10], d_b=P[11], ws=P[12], n=BIG):
    return fm.lib().fm_layer_norm_bwd(dt, sd, bd, M, N, d_y, d_out, out, mean, rstd, w, p, rng, draw,
                                      row, d_resid, d_block, d_bias, d_w, d_b, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), UNS), (dict(sd=0), UNS), (dict(bd=0), UNS), (dict(M=-1), INV), (dict(N=20), INV),
    (dict(N=16392), UNS), (dict(M=1 << 31), UNS), (dict(p=-1.0), INV), (dict(rng=None), INV),
    (dict(row=-1), INV), (dict(row=1 << 32), UNS),
    (dict(d_y=None), INV), (dict(w=None), INV), (dict(out=None), INV), (dict(mean=None), INV),
    (dict(rstd=None), INV), (dict(w=None, d_y=None), INV),                     # d_w without w
    (dict(w=None, d_y=None, d_w=None), INV),                                   # d_b without w
    (dict(w=None, d_y=None, d_w=None, d_b=None, d_out=None), INV),
    (dict(d_resid=None, d_block=None, d_bias=None, d_w=None, d_b=None), INV),
    (dict(ws=None), INV), (dict(n=64), INV), (dict(ws=ODD), INV),
    (dict(d_y=ODD), INV), (dict(d_out=ODD), INV), (dict(out=ODD), INV), (dict(w=ODD), INV),
    (dict(mean=ODD2), INV), (dict(rstd=ODD2), INV), (dict(d_resid=ODD), INV), (dict(d_block=ODD), INV),
    (dict(d_bias=ODD), INV), (dict(d_w=ODD), INV), (dict(d_b=ODD), INV),
    (dict(N=0), OK),
    (dict(M=0, d_y=None, d_out=None, out=None, mean=None, rstd=None, d_bias=None, d_w=None, d_b=None,
          ws=None, n=0), OK),
])
def test_layer_norm_bwd_refusals(kw, want):
    assert ln_bwd_call(**kw) == want


@pytest.mark.parametrize("M,N", [(-1, 64), (4, -8), (4, 12), (4, 16392), (1 << 31, 64)])
def test_layer_norm_workspace_refusals(M, N):
    assert fm.fm_layer_norm_workspace_bytes(M, N) == 0


def test_layer_norm_workspace_holds_a_partial_row_a_block():
    assert fm.fm_layer_norm_workspace_bytes(0, 64) == 256
    assert fm.fm_layer_norm_workspace_bytes(10 ** 6, 16384) == 256 * 16384 * 12


def quant_call(dt=1, M=4, N=64, x=P[0], q=P[1], scale=P[2]):
    return fm.lib().fm_quant_i8(dt, M, N, x, q, scale, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=3), UNS), (dict(M=-1), INV), (dict(N=-8), INV), (dict(N=4), INV), (dict(M=1 << 31), UNS),
    (dict(N=1 << 31), UNS), (dict(x=None), INV), (dict(q=None), INV), (dict(scale=None), INV),
    (dict(x=ODD), INV), (dict(q=ODD), INV), (dict(scale=ODD2), INV), (dict(M=0, x=None, q=None), OK),
])
def test_quant_refusals(kw, want):
    assert quant_call(**kw) == want


def gemm_call(dt=1, c=1, M=4, N=64, K=64, A=P[0], a_scale=P[1], W=P[2], w_scale=P[3], bias=P[4], act=0,
              C=P[5]):
    return fm.lib().fm_gemm_i8(dt, c, M, N, K, A, a_scale, W, w_scale, bias, act, C, None)


LIMITS = [
    (dict(dt=2), UNS), (dict(dt=3), UNS), (dict(c=0), UNS), (dict(c=3), UNS), (dict(M=-1), INV),
    (dict(N=-8), INV), (dict(K=-16), INV), (dict(N=12), INV), (dict(K=24), INV), (dict(M=1 << 22), UNS),
    (dict(N=1 << 22), UNS), (dict(K=131072), UNS), (dict(act=-1), INV), (dict(act=4), INV),
    (dict(W=None), INV), (dict(w_scale=None), INV), (dict(C=None), INV), (dict(W=ODD), INV),
    (dict(w_scale=ODD), INV), (dict(bias=ODD), INV), (dict(C=ODD), INV), (dict(M=0, C=None), OK),
    (dict(N=0, C=None), OK),
]


@pytest.mark.parametrize("kw,want", LIMITS + [
    (dict(A=None), INV), (dict(a_scale=None), INV), (dict(A=ODD), INV), (dict(a_scale=ODD2), INV),
])
def test_gemm_i8_refusals(kw, want):
    assert gemm_call(**kw) == want


def linear_call(dt=1, c=1, M=4, N=64, K=64, X=P[0], W=P[2], w_scale=P[3], bias=P[4], act=0, C=P[5],
                ws=P[6], n=BIG):
    return fm.lib().fm_linear_i8(dt, c, M, N, K, X, W, w_scale, bias, act, C, ws, n, None)


@pytest.mark.parametrize("kw,want", LIMITS + [
    (dict(X=None), INV), (dict(X=ODD), INV), (dict(ws=None), INV), (dict(ws=ODD), INV), (dict(n=255), INV),
    (dict(M=100, n=100 * 64 + 399), INV),
])
def test_linear_i8_refusals(kw, want):
    assert linear_call(**kw) == want


@pytest.mark.parametrize("M,K", [(-1, 64), (4, -16), (4, 24), (1 << 22, 64), (4, 131072)])
def test_linear_i8_workspace_refusals(M, K):
    assert fm.fm_linear_i8_workspace_bytes(M, K) == 0


def test_linear_i8_workspace_holds_codes_and_scales():
    assert fm.fm_linear_i8_workspace_bytes(0, 64) == 256
    assert fm.fm_linear_i8_workspace_bytes(100, 64) >= 100 * 64 + 400
