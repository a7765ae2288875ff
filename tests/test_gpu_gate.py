"""fm_moe_gate and fm_moe_gate_bwd against the float64 definitions.

Tolerances, in units u = 2^-24 of fp32 arithmetic.  A share or weight is
exp(x - m) over a sum of E such terms.  With |x - m| <= R the rounded difference,
the product with log2(e) and that constant move the exponent by at most 3 R u; exp2
adds 2 u, 1 + exp and the quotient of a sigmoid 6 u, the sum (chains of 16 and 6) 22 u
and its own terms' 3 R u, the reciprocal and products 8 u: (6 R + 48) u, relative.
Sums over tokens add at most one rounding a term of the longest chain (passes of a
block, rows of a block, blocks): under 256 u up to the sizes here.  A gradient is a sum
of such terms: the same relative to the sum of their magnitudes, with one more factor
and 64 u for the sums over the slots and experts.  Each 16-bit output rounds by eps / 2."""
import numpy as np
import pytest

import tile_gemm_communication_amd as fm
from gpu_util import say
from oracle import block as ob

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _logits(T, E, dt, seed, closed=0, spread=1.5, ties=False):
    import torch
    rng = np.random.default_rng(seed)
    x = spread * rng.standard_normal((T, E))
    if ties:
        x = np.round(x)                       # many equal logits, -0.0 among them
        x[::3] = np.where(x[::3] == 0, -0.0, x[::3])
    if closed:
        x[:, rng.permutation(E)[:closed]] = -np.inf
    t = torch.from_numpy(x).to("cuda:0").to(_dtype(dt))
    return t, t.double().cpu().numpy()


def _range(x):
    f = np.where(np.isfinite(x), x, 0)
    return float(np.abs(f).max() * 2 + 1)


def _forward(x, topk, **kw):
    import torch
    T, E = x.shape
    pad = 3
    ids = torch.full((T * topk + pad,), -7, dtype=torch.int32, device="cuda:0")
    w = torch.full((T * topk + pad,), -7.0, device="cuda:0")
    c = torch.full((E + 1 + pad,), -7, dtype=torch.int32, device="cuda:0")
    s = torch.full((E + pad,), -7.0, device="cuda:0")
    loss = torch.full((1,), -7.0, device="cuda:0")
    ws = torch.full((fm.fm_moe_gate_workspace_bytes(T, E) + 64,), 0x5A, dtype=torch.uint8,
                    device="cuda:0")
    fm.fm_moe_gate(x, ids[:T * topk].view(T, topk), w[:T * topk].view(T, topk), counts=c[:E + 1],
                   prob_sums=s[:E], loss=loss, ws=ws[:-64], **kw)
    torch.cuda.synchronize()
    for t, n in ((ids, T * topk), (w, T * topk), (c, E + 1), (s, E)):
        assert (t[n:] == -7).all(), "written past the end"
    assert (ws[-64:] == 0x5A).all()
    return (ids[:T * topk].view(T, topk), w[:T * topk].view(T, topk), c[:E + 1], s[:E], loss)


CASES = [  # T, E, topk, dt, score, renorm, bias, mask, closed, ties
    (1, 64, 2, "bf16", 0, False, False, False, 0, False),
    (1, 1, 1, "fp32", 0, True, False, False, 0, False),
    (3, 5, 5, "fp16", 1, False, False, False, 2, False),
    (7, 8, 3, "bf16", 0, True, False, True, 0, True),
    (130, 61, 8, "fp32", 1, True, True, True, 3, False),
    (257, 64, 4, "bf16", 1, True, True, False, 0, True),
    (200, 100, 6, "fp16", 0, False, True, True, 0, True),
    (333, 256, 8, "fp32", 1, True, False, True, 0, False),
    (65, 130, 10, "bf16", 0, True, False, False, 120, True),
    (90, 384, 16, "fp32", 0, False, False, False, 0, False),
    (40, 511, 16, "fp16", 1, True, True, False, 0, False),
    (33, 1024, 16, "bf16", 0, True, False, True, 0, True),
    (21, 1023, 3, "fp32", 1, False, True, False, 1000, False),
    (5000, 16, 2, "bf16", 0, False, False, True, 0, True),
    (20000, 64, 2, "bf16", 0, False, False, False, 0, True),
]


@pytest.mark.parametrize("T,E,topk,dt,score,renorm,bias,mask,closed,ties", CASES)
def test_gate_forward(T, E, topk, dt, score, renorm, bias, mask, closed, ties):
    import torch
    say(f"gate T={T} E={E} topk={topk} {dt} score={score} renorm={renorm} bias={bias}")
    x, x64 = _logits(T, E, dt, T + E, closed, ties=ties)
    rng = np.random.default_rng(9)
    b = (0.1 * rng.standard_normal(E)).astype(np.float32) if bias else None
    m = (rng.random(T) < 0.8).astype(np.uint8) if mask else None
    if mask:
        x[torch.from_numpy(m == 0).to("cuda:0")] = float("nan")   # what padding holds is not used
    kw = dict(score=score, renormalize=renorm, scale=2.5)
    dev = dict(kw, bias=None if b is None else torch.from_numpy(b).to("cuda:0"),
               token_mask=None if m is None else torch.from_numpy(m).to("cuda:0"))
    ids, w, c, s, loss = _forward(x, topk, **dev)
    rid, rw, rc, rs, rl = ob.gate(x64, topk, score, renorm, 2.5,
                                  None if b is None else b.astype(np.float64), m)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert np.array_equal(c.cpu().numpy(), rc)
    tol = (6 * _range(x64) + 48) * U
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=tol, atol=1e-37)
    np.testing.assert_allclose(s.cpu().numpy(), rs, rtol=tol + 256 * U, atol=1e-36)
    np.testing.assert_allclose(loss.item(), rl, rtol=tol + 256 * U, atol=1e-37)
    # the same bits again, and without the statistics
    again = _forward(x, topk, **dev)
    for p, q in zip((ids, w, c, s, loss), again):
        assert torch.equal(p, q)
    i2, w2 = torch.empty_like(ids), torch.empty_like(w)
    fm.fm_moe_gate(x, i2, w2, **dev)
    assert torch.equal(i2, ids) and torch.equal(w2, w)


@pytest.mark.parametrize("T,E,topk,dt,score,renorm,bias,mask,closed,ties", CASES)
def test_gate_backward(T, E, topk, dt, score, renorm, bias, mask, closed, ties):
    import torch
    say(f"gate bwd T={T} E={E} topk={topk} {dt} score={score} renorm={renorm}")
    T = min(T, 700)
    x, x64 = _logits(T, E, dt, T + E, closed, ties=ties)
    rng = np.random.default_rng(11)
    m = (rng.random(T) < 0.8).astype(np.uint8) if mask else None
    ids, _, counts, _, _ = ob.gate(x64, topk, score, renorm, 2.5, mask=m)
    ids[0, 0] = E + 5                         # slots outside take no part
    if topk > 1 and T > 1:
        ids[1, 1] = ids[1, 0]                 # an expert named twice adds up
    d_w = rng.standard_normal((T, topk)).astype(np.float32)
    d_w[ids < 0] = np.nan
    d_l = np.float32(0.7 * T)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")  # noqa: E731
    mk = None if m is None else dev(m)
    if mask:
        x[mk == 0] = float("nan")
    tol = (6 * _range(x64) + 48 + 64 + 2 * topk) * U
    eps = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": U}[dt]
    tiny = {"bf16": 1e-36, "fp16": 2.0 ** -25, "fp32": 1e-36}[dt]   # half the smallest subnormal
    for has_w, has_l in ((1, 1), (1, 0), (0, 1), (0, 0)):
        dx = torch.full((T * E + 3,), -7.0, device="cuda:0", dtype=x.dtype)
        fm.fm_moe_gate_bwd(x, dev(ids.astype(np.int32)), dx[:T * E].view(T, E), score=score,
                           renormalize=renorm, scale=2.5, token_mask=mk,
                           d_weights=dev(d_w) if has_w else None,
                           counts=dev(counts.astype(np.int32)) if has_l else None,
                           d_loss=dev(np.array([d_l])) if has_l else None)
        torch.cuda.synchronize()
        assert (dx[T * E:] == -7).all()
        ref, mag = ob.gate_bwd(x64, ids, score, renorm, 2.5, m, d_w.astype(np.float64) if has_w else None,
                               counts if has_l else None, float(d_l))
        got = dx[:T * E].view(T, E).double().cpu().numpy()
        err = np.abs(got - ref)
        lim = tol * mag + eps * np.abs(ref) + tiny
        assert (err <= lim).all(), (has_w, has_l, float((err / lim).max()))


def test_gate_extremes():
    """Shares that would vanish in fp32, closed and infinite rows, NaN."""
    import torch
    inf = float("inf")
    x = torch.tensor([[-200.0, -201, -202, -inf], [300.0, 299, -300, 0], [-inf] * 4,
                      [88.0, -88, 0, 1]], device="cuda:0")
    x64 = x.double().cpu().numpy()
    for score in (0, 1):
        for renorm in (False, True):
            ids, w, c, s, loss = _forward(x, 3, score=score, renormalize=renorm)
            r = ob.gate(x64, 3, score, renorm, 1.0)
            assert np.array_equal(ids.cpu().numpy(), r[0]) and np.array_equal(c.cpu().numpy(), r[2])
            np.testing.assert_allclose(w.cpu().numpy(), r[1], rtol=4000 * U, atol=1e-37)
            np.testing.assert_allclose(s.cpu().numpy(), r[3], rtol=4000 * U, atol=1e-37)
    x[1, 2] = float("nan")
    ids, w, c, s, loss = _forward(x, 3, score=0)
    assert ids[1].tolist() == [0, 1, 3]       # a NaN is never chosen
    assert torch.isnan(s).all() and torch.isnan(loss).all()
    mask = torch.zeros(4, dtype=torch.bool, device="cuda:0")     # bool holds the same bytes
    ids, w, c, s, loss = _forward(x, 2, token_mask=mask)
    assert (ids == -1).all() and (w == 0).all() and (c == 0).all() and (s == 0).all()
    assert loss.item() == 0


def test_gate_no_tokens():
    import torch
    x = torch.empty(0, 8, device="cuda:0")
    ids, w, c, s, loss = _forward(x, 2)
    assert (c == 0).all() and (s == 0).all() and loss.item() == 0


def test_gate_feeds_the_route(oracle):
    """The router's ids go straight into fm_moe_route, unfilled slots included."""
    import torch
    x, x64 = _logits(500, 16, "bf16", 2, closed=13)
    ids, w, c, _, _ = _forward(x, 4)
    assert (ids[:, 3] == -1).all()
    sp = torch.full((2000,), -1, dtype=torch.int32, device="cuda:0")
    off = torch.zeros(9, dtype=torch.int32, device="cuda:0")
    fm.fm_moe_route(ids, 4, 8, sp, off, fm.moe_workspace(500, 4, 64, 8))
    torch.cuda.synchronize()
    roff, rsp = oracle.moe_route(ids.cpu().numpy(), 4, 8)
    assert np.array_equal(off.cpu().numpy(), roff)
    assert np.array_equal(sp[:roff[-1]].cpu().numpy(), rsp)
    assert np.array_equal(np.diff(roff), c.cpu().numpy()[4:12])


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_gate_bias_and_rows_that_are_not_finite(dt, bad):
    """Keys of a biased choice are made of scores: under a softmax one NaN (or +inf) makes all of
    its row's NaN and the row finds no expert; sigmoid scores stand each for itself."""
    import torch
    rng = np.random.default_rng(21)
    T, E, topk = 40, 24, 4
    t = torch.from_numpy(rng.standard_normal((T, E))).to("cuda:0").to(_dtype(dt))
    b = torch.from_numpy((0.1 * rng.standard_normal(E)).astype(np.float32)).to("cuda:0")
    clean, b64 = t.double().cpu().numpy(), b.double().cpu().numpy()
    t[7, 3] = bad
    t[33] = bad
    rest = [i for i in range(T) if i not in (7, 33)]
    ids, w, c, s, loss = _forward(t, topk, score=0, bias=b)
    want = ob.gate(clean, topk, 0, False, 1.0, b64)[0]
    got = ids.cpu().numpy()
    assert np.array_equal(got[rest], want[rest]) and (got[[7, 33]] == -1).all()
    assert (w[[7, 33]] == 0).all() and torch.isfinite(w).all()
    assert c[:E].sum().item() == topk * len(rest) and c[E].item() == T
    assert torch.isnan(s).all() and torch.isnan(loss).all()
    ids, w, c, s, loss = _forward(t, topk, score=1, bias=b)
    want = clean.copy()
    want[7, 3], want[33] = (-np.inf, -np.inf) if np.isnan(bad) else (bad, bad)   # chosen as +inf, never as NaN
    want = ob.gate(want, topk, 1, False, 1.0, b64)[0]
    assert np.array_equal(ids.cpu().numpy(), want) and torch.isfinite(w).all()


def test_gate_bias_that_closes_experts():
    """A bias of -inf or NaN keeps an expert from being chosen and leaves its share."""
    import torch
    x, x64 = _logits(50, 12, "fp32", 4)
    b = np.zeros(12, np.float32)
    b[[2, 5]] = -np.inf
    want = ob.gate(x64, 3, 0, False, 1.0, b.astype(np.float64))
    b[5] = np.nan
    ids, w, c, s, loss = _forward(x, 3, bias=torch.from_numpy(b).to("cuda:0"))
    assert np.array_equal(ids.cpu().numpy(), want[0]) and np.array_equal(c.cpu().numpy(), want[2])
    np.testing.assert_allclose(w.cpu().numpy(), want[1], rtol=(6 * _range(x64) + 48) * U)
    np.testing.assert_allclose(s.cpu().numpy(), want[3], rtol=(6 * _range(x64) + 304) * U)
