"""The products with 4-bit weights against the float64 definitions.

Tolerances, u = 2^-24.  A group's sums t = sum x (base + code) and S = sum x are
exact products added in fp32: at most 32 additions in an instruction (2 u each, if it
truncates) and 4 instructions, 72 u of sum |x| (base + 15).  scale, zero and the two
fused multiply-adds add 4 u of the same; groups and waves are added up in chains of
K / (32 * 8) and 8: (K / 256 + 8) u.  (Where the waves share several tiles the chains
are up to K / 32 long, of terms within 15 sum |x| scale: up to K = 2185 that is within
(K / 256 + 8) u of the magnitude below.)  With a base of at most 16 (bf16) or 64
(fp16; the kernels use 16 for both) and |code - zero| <= 15 this is, for each output,
  (K / 256 + 84) u * 2 (base + 15) * sum_k |x_k| scale_k.
Two roundings follow for a weight and the sum over k (topk u), each 16-bit output rounds
by eps / 2, activations have slopes up to 1.13 and add 16 u."""
import numpy as np
import pytest

import tile_gemm_communication_amd as fm
import workloads as wl
from gpu_util import say
from oracle import block as ob

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": U}
TINY = {"bf16": 1e-38, "fp16": 2.0 ** -25, "fp32": 1e-38}
BASE = {"bf16": 16, "fp16": 64}


@pytest.fixture(autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _dev(a, dt=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")
    return t if dt is None else t.to(_dtype(dt))


def _host(t):
    return t.double().cpu().numpy()


def _weights(lead, K, N, group, dt, zeros, rng):
    """(codes, scales, zeros) as device tensors."""
    G = -(-K // group)
    codes = rng.integers(0, 16, lead + (K, N)).astype(np.uint8)
    s = _dev((0.2 + rng.random(lead + (G, N))) / (4.6 * max(K, 1) ** 0.5), dt)
    z = rng.integers(0, 16, lead + (G, N)).astype(np.uint8) if zeros else None
    return codes, s, (None if z is None else _dev(z))


def _pack(codes):
    import torch
    K, N = codes.shape[-2:]
    out = torch.full(codes.shape[:-2] + (N, fm.fm_w4_row_bytes(K)), 0xEE, dtype=torch.uint8,
                     device="cuda:0")
    fm.fm_w4_pack(_dev(codes), out)
    return out


def _bound(x, scales, K, group, dt):
    """The tolerance of each output of x @ W (scales [G, N])."""
    s = scales[np.arange(K) // group]
    return (K / 256 + 84) * U * 2 * (BASE[dt] + 15) * (np.abs(x) @ np.abs(s))


@pytest.mark.parametrize("K,N,lead", [(8, 8, ()), (128, 24, (3,)), (136, 16, (2, 2)), (1000, 40, ())])
def test_pack(K, N, lead):
    codes = np.random.default_rng(K).integers(0, 16, lead + (K, N)).astype(np.uint8)
    got = _pack(codes + 16 * (codes % 3)).cpu().numpy()   # the high bits are dropped
    for at in np.ndindex(*lead):
        assert np.array_equal(got[at], ob.w4_pack(codes[at]))


@pytest.mark.parametrize("M,N,K,group,dt,out,zeros", [
    (1, 8, 8, 32, "bf16", "fp32", False),
    (1, 16, 128, 128, "fp16", "fp16", True),
    (1, 1000, 1000, 64, "bf16", "bf16", True),
    (2, 72, 4096, 128, "bf16", "fp32", False),
    (4, 24, 136, 32, "fp16", "fp32", True),
    (5, 40, 264, 64, "bf16", "fp32", True),
    (15, 136, 2816, 32, "bf16", "bf16", False),
    (16, 64, 1280, 128, "fp16", "fp32", True),
    (17, 48, 392, 32, "fp16", "fp16", False),
    (33, 56, 520, 64, "bf16", "fp32", True),
    (45, 520, 648, 32, "bf16", "fp32", True),
    (64, 16, 1024, 128, "fp16", "fp32", False),
    (131, 200, 328, 64, "bf16", "bf16", True),
    (300, 8, 3000, 128, "bf16", "fp32", False),
    (4, 72, 12288, 128, "bf16", "fp32", True),
    (7, 40, 6152, 32, "fp16", "fp32", False),
    (8, 24, 16384, 64, "bf16", "fp32", True),
    (3, 16, 65536, 128, "bf16", "fp32", False),
])
def test_gemm_w4(M, N, K, group, dt, out, zeros):
    import torch
    say(f"gemm_w4 M={M} N={N} K={K} group={group} {dt}->{out}")
    rng = np.random.default_rng(M + N + K)
    codes, s, z = _weights((), K, N, group, dt, zeros, rng)
    x = _dev(rng.standard_normal((M, K)), dt)
    c = torch.full((M * N + 8,), -7.0, device="cuda:0", dtype=_dtype(out))
    fm.fm_gemm_w4(x, _pack(codes), s, c[:M * N].view(M, N), group, zeros=z)
    torch.cuda.synchronize()
    assert (c[M * N:] == -7).all()
    W = ob.w4_matrix(codes, _host(s), None if z is None else z.cpu().numpy(), group)
    ref = _host(x) @ W
    err = np.abs(_host(c[:M * N].view(M, N)) - ref)
    lim = _bound(_host(x), _host(s), K, group, dt) + HALF[out] * np.abs(ref) + TINY[out]
    assert (err <= lim).all(), float((err / lim).max())
    if out == "fp32" and K >= 128:   # the bound is a worst case; roundings of random sign stay far below
        assert np.linalg.norm(err) <= 2e-6 * (BASE[dt] / 16) * np.linalg.norm(ref)


def test_gemm_w4_codes_past_k_and_scales_are_exact():
    """One-hot rows return each weight exactly, whatever the padding codes hold."""
    import torch
    K, N, group = 200, 24, 32
    rng = np.random.default_rng(0)
    codes, _, z = _weights((), K, N, group, "bf16", True, rng)
    s = _dev(2.0 ** rng.integers(-6, 6, (7, N)), "bf16")
    packed = _pack(np.concatenate([codes, np.zeros((56, N), np.uint8)]))
    other = _pack(np.concatenate([codes, np.full((56, N), 15, np.uint8)]))
    x = torch.eye(K, device="cuda:0").to(torch.bfloat16)
    c, d = torch.empty(K, N, device="cuda:0"), torch.empty(K, N, device="cuda:0")
    fm.fm_gemm_w4(x, packed, s, c, group, zeros=z)
    fm.fm_gemm_w4(x, other, s, d, group, zeros=z)
    assert np.array_equal(_host(c), ob.w4_matrix(codes, _host(s), z.cpu().numpy(), group))
    assert torch.equal(c, d)


def test_gemm_w4_without_k():
    import torch
    c = torch.full((3, 16), 5.0, device="cuda:0")
    e = torch.empty(3, 0, device="cuda:0", dtype=torch.bfloat16)
    fm.fm_gemm_w4(e, torch.empty(16, 0, dtype=torch.uint8, device="cuda:0"),
                  torch.empty(0, 16, device="cuda:0", dtype=torch.bfloat16), c, 32)
    assert (c == 0).all()


def _act64(x, act):
    if act == fm.FM_ACT_RELU:
        return np.maximum(x, 0)
    if act == fm.FM_ACT_GELU_TANH:
        return 0.5 * x * (1 + np.tanh(np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)))
    return x / (1 + np.exp(-x)) if act == fm.FM_ACT_SILU else x


MOE = [  # T, hidden, ffn, E, nl, e0, topk, group, dt, zeros, act, closed (no token there)
    (1, 256, 128, 8, 8, 0, 2, 128, "bf16", False, 3),
    (1, 256, 128, 16, 4, 8, 2, 64, "fp16", True, 0),
    (3, 136, 264, 4, 4, 0, 4, 32, "bf16", True, 2),
    (17, 520, 72, 8, 8, 0, 1, 64, "fp16", True, 1),
    (61, 384, 176, 64, 64, 0, 2, 128, "bf16", True, 3),
    (61, 384, 176, 64, 8, 8, 2, 32, "fp16", False, 2),
    (40, 256, 200, 2, 2, 0, 2, 128, "bf16", True, 0),      # every token in both experts
    (200, 128, 136, 4, 3, 1, 2, 64, "bf16", False, 3),
    (2100, 64, 72, 8, 4, 0, 4, 32, "fp16", True, 0),
    (4, 264, 4104, 4, 4, 0, 2, 128, "bf16", True, 3),      # eight pairs, long rows
    (13, 4104, 40, 16, 16, 0, 3, 64, "bf16", False, 1),
    (2, 16384, 72, 4, 2, 2, 2, 32, "fp16", True, 0),       # rows too long for LDS
    (9, 72, 20480, 8, 8, 0, 1, 128, "bf16", True, 2),
    (128, 136, 72, 64, 64, 0, 4, 64, "fp16", True, 3),     # 512 pairs: the most that one launch sorts
    (129, 136, 72, 64, 64, 0, 4, 64, "fp16", True, 3),
    (100, 1288, 264, 64, 64, 0, 4, 32, "bf16", True, 3),   # 2 and 8 tiles a block; 1 to 12 rows
    (61, 264, 520, 8, 8, 0, 2, 32, "bf16", False, 2),      # 8 to 22 rows
    (61, 1288, 264, 64, 64, 0, 2, 128, "fp16", True, 0),
    (6, 12288, 72, 4, 4, 0, 2, 128, "bf16", False, 0),     # four rows nearly fill LDS
    (6, 72, 12288, 4, 4, 0, 2, 64, "fp16", True, 0),
]


def _moe(T, hidden, ffn, E, nl, e0, topk, group, dt, zeros, seed=5):
    rng = np.random.default_rng(seed + T)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :topk].astype(np.int32)
    if T > 8:
        ids[3] = -1                                        # a token that goes nowhere
    return rng, ids


@pytest.mark.parametrize("T,hidden,ffn,E,nl,e0,topk,group,dt,zeros,act", MOE)
def test_gather_w4(oracle, T, hidden, ffn, E, nl, e0, topk, group, dt, zeros, act):
    import torch
    say(f"gather_w4 T={T} {hidden}x{ffn} E={E} nl={nl} e0={e0} topk={topk} group={group} {dt}")
    rng, ids = _moe(T, hidden, ffn, E, nl, e0, topk, group, dt, zeros)
    codes, s, z = _weights((nl,), hidden, ffn, group, dt, zeros, rng)
    x = _dev(rng.standard_normal((T, hidden)), dt)
    h = torch.full((T * topk + 1, ffn), -7.0, device="cuda:0", dtype=_dtype(dt))
    sp = torch.full((T * topk + 1,), -9, dtype=torch.int32, device="cuda:0")
    off = torch.full((nl + 1,), -9, dtype=torch.int32, device="cuda:0")
    ws = fm.moe_workspace(T, topk, hidden, nl)
    for _ in range(2):
        fm.fm_moe_gather_gemm_w4(x, _dev(ids), _pack(codes), s, h, sp, off, e0, group, ws, zeros=z,
                                 act=act)
    torch.cuda.synchronize()
    roff, rsp = oracle.moe_route(ids, e0, nl)
    rows = int(roff[-1])
    assert np.array_equal(off.cpu().numpy(), roff)
    assert np.array_equal(sp[:rows].cpu().numpy(), rsp) and (sp[rows:] == -9).all()
    assert (h[rows:] == -7).all()                          # rows behind the last are left
    for e in range(nl):
        a, b = roff[e], roff[e + 1]
        if a == b:
            continue
        xe = _host(x)[rsp[a:b] // topk]
        v = xe @ ob.w4_matrix(codes[e], _host(s)[e], None if z is None else z[e].cpu().numpy(), group)
        ref = _act64(v, act)
        lim = 1.13 * _bound(xe, _host(s)[e], hidden, group, dt) + 16 * U * np.abs(v) + \
            HALF[dt] * np.abs(ref) + TINY[dt]
        err = np.abs(_host(h[a:b]) - ref)
        assert (err <= lim).all(), (e, float((err / lim).max()))


@pytest.mark.parametrize("T,hidden,ffn,E,nl,e0,topk,group,dt,zeros,act", MOE)
def test_scatter_w4(oracle, T, hidden, ffn, E, nl, e0, topk, group, dt, zeros, act):
    import torch
    say(f"scatter_w4 T={T} {ffn}x{hidden} E={E} nl={nl} e0={e0} topk={topk} group={group} {dt}")
    rng, ids = _moe(T, hidden, ffn, E, nl, e0, topk, group, dt, zeros, seed=50)
    if T > 8:
        ids[5, -1] = ids[5, 0]                             # one expert twice
    roff, rsp = oracle.moe_route(ids, e0, nl)
    rows = int(roff[-1])
    codes, s, z = _weights((nl,), ffn, hidden, group, dt, zeros, rng)
    h = _dev(rng.standard_normal((T * topk, ffn)), dt)
    h[rows:] = float("nan")
    w = rng.random((T, topk)).astype(np.float32)
    w[(ids < e0) | (ids >= e0 + nl)] = np.nan              # weights of other ranks' pairs
    add = rng.standard_normal((T, hidden)).astype(np.float32)
    sp = np.full(T * topk, -9, np.int32)
    sp[:rows] = rsp
    args = (h, _pack(codes), s, _dev(ids), _dev(sp), _dev(roff.astype(np.int32)), _dev(w))
    ws = torch.full((fm.fm_moe_w4_workspace_bytes(T, topk, hidden) + 64,), 0xFF, dtype=torch.uint8,
                    device="cuda:0")
    outs = []
    for given in (None, _dev(add)):
        out = torch.full((T * hidden + 8,), -7.0, device="cuda:0")
        fm.fm_moe_gemm_scatter_w4(*args, out[:T * hidden].view(T, hidden), e0, group, ws[:-64],
                                  zeros=z, add=given)
        torch.cuda.synchronize()
        assert (out[T * hidden:] == -7).all() and (ws[-64:] == 0xFF).all()
        outs.append(out[:T * hidden].view(T, hidden))
    ref, lim = np.zeros((T, hidden)), np.zeros((T, hidden))
    for e in range(nl):
        a, b = roff[e], roff[e + 1]
        if a == b:
            continue
        p = rsp[a:b]
        v = _host(h[a:b]) @ ob.w4_matrix(codes[e], _host(s)[e], None if z is None else z[e].cpu().numpy(),
                                         group)
        wt = w.reshape(-1)[p].astype(np.float64)[:, None]
        np.add.at(ref, p // topk, wt * v)
        np.add.at(lim, p // topk, wt * (_bound(_host(h[a:b]), _host(s)[e], ffn, group, dt)
                                        + (topk + 2) * U * np.abs(v)))
    for out, plus in zip(outs, (0.0, add.astype(np.float64))):
        err = np.abs(_host(out) - (ref + plus))
        assert (err <= lim + 2 * U * (np.abs(plus) + np.abs(ref)) + 1e-38).all()
    # add may be out itself; the same bits on every call
    inplace = _dev(add)
    fm.fm_moe_gemm_scatter_w4(*args, inplace, e0, group, ws[:-64], zeros=z, add=inplace)
    assert torch.equal(inplace, outs[1])


@pytest.mark.parametrize("T", [1, 3, 40, 600])
def test_empty_contractions(T):
    """Sums over nothing: zeros in C and in the local rows of H, add (or zeros) in out."""
    import torch
    say(f"w4 K=0 T={T}")
    dev, bf = "cuda:0", torch.bfloat16
    nl, topk, n = 4, 2, 200
    x = torch.empty(T, 0, device=dev, dtype=bf)
    c = torch.full((T, n), -7.0, device=dev)
    fm.fm_gemm_w4(x, torch.empty(n, 0, dtype=torch.uint8, device=dev),
                  torch.empty(0, n, dtype=bf, device=dev), c, 64)
    assert (c == 0).all()
    ids = _dev(np.stack([np.arange(T) % 8, np.arange(T) % 8 + 1], 1).astype(np.int32))   # some not local
    local = int((ids < nl).sum())
    p = torch.empty(nl, n, 0, dtype=torch.uint8, device=dev)
    s = torch.empty(nl, 0, n, dtype=bf, device=dev)
    h = torch.full((T * topk, n), -7.0, device=dev, dtype=bf)
    sp = torch.full((T * topk,), -9, dtype=torch.int32, device=dev)
    off = torch.zeros(nl + 1, dtype=torch.int32, device=dev)
    fm.fm_moe_gather_gemm_w4(x, ids, p, s, h, sp, off, 0, 64, fm.moe_workspace(T, topk, n, nl))
    assert int(off[-1]) == local and (h[:local] == 0).all() and (h[local:] == -7).all()
    w = torch.ones(T, topk, device=dev)
    add = torch.randn(T, n, device=dev)
    ws = fm.moe_w4_workspace(T, topk, n)
    he = torch.empty(T * topk, 0, device=dev, dtype=bf)
    for given in (add, None):
        out = torch.full((T, n), -7.0, device=dev)
        fm.fm_moe_gemm_scatter_w4(he, p, s, ids, sp, off, w, out, 0, 64, ws, add=given)
        assert torch.equal(out, add if given is not None else torch.zeros_like(add))


def test_w4_agrees_with_the_16_bit_layer():
    """The same expert weights unpacked to 16 bits through the existing layer: codes and
    power-of-two scales are exact in bf16, so only the summation order differs."""
    import torch
    T, hidden, ffn, E, nl, topk, group = 48, 256, 128, 8, 8, 2, 64
    rng, ids = _moe(T, hidden, ffn, E, nl, 0, topk, group, "bf16", True, seed=1)
    ids[3] = [0, 1]
    mats = []
    for K, N in ((hidden, ffn), (ffn, hidden)):
        codes, _, z = _weights((nl,), K, N, group, "bf16", True, rng)
        s = _dev(2.0 ** -rng.integers(5, 8, (nl, K // group, N)), "bf16")
        W = np.stack([ob.w4_matrix(codes[e], _host(s)[e], z[e].cpu().numpy(), group) for e in range(nl)])
        mats.append((_pack(codes), s, z, _dev(W, "bf16")))
        assert np.array_equal(_host(mats[-1][3]), W)
    x = _dev(rng.standard_normal((T, hidden)), "bf16")
    w = _dev(rng.random((T, topk)).astype(np.float32))
    outs = []
    for four in (False, True):
        h = torch.zeros(T * topk, ffn, device="cuda:0", dtype=torch.bfloat16)
        sp = torch.zeros(T * topk, dtype=torch.int32, device="cuda:0")
        off = torch.zeros(nl + 1, dtype=torch.int32, device="cuda:0")
        out = torch.zeros(T, hidden, device="cuda:0")
        ws = fm.moe_workspace(T, topk, hidden, nl)
        (p1, s1, z1, W1), (p2, s2, z2, W2) = mats
        if four:
            fm.fm_moe_gather_gemm_w4(x, _dev(ids), p1, s1, h, sp, off, 0, group, ws, zeros=z1,
                                     act=fm.FM_ACT_RELU)
            h.copy_(outs[0][0])                            # the same 16-bit rows for the second layer
            fm.fm_moe_gemm_scatter_w4(h, p2, s2, _dev(ids), sp, off, w, out, 0, group,
                                      fm.moe_w4_workspace(T, topk, hidden), zeros=z2)
        else:
            fm.fm_moe_gather_gemm_act(x, _dev(ids), W1, h, sp, off, 0, fm.FM_ACT_RELU, ws)
            fm.fm_moe_gemm_scatter(h, W2, sp, off, w, out, ws)
        torch.cuda.synchronize()
        outs.append((h, out))
    d = (outs[0][1] - outs[1][1]).double()
    assert d.norm() <= 4e-6 * outs[0][1].double().norm()


def test_tensors_the_kernels_cannot_take_are_refused():
    import torch
    x = torch.zeros(2, 256, device="cuda:0", dtype=torch.bfloat16)
    p = torch.zeros(16, 128, device="cuda:0", dtype=torch.uint8)
    s, c = torch.zeros(8, 16, device="cuda:0", dtype=torch.bfloat16), torch.zeros(2, 16, device="cuda:0")
    good = dict(A=x, packed=p, scales=s, C=c, group=32)
    fm.fm_gemm_w4(**good)
    for name, bad in (("A", x.float()), ("A", x[:, ::2]), ("packed", p[:, :64]), ("packed", p.int()),
                      ("scales", s[:4]), ("scales", s.half()), ("scales", s.cpu()), ("C", c.double()),
                      ("C", torch.zeros(3, 16, device="cuda:0")), ("group", 64), ("group", 16)):
        with pytest.raises((ValueError, TypeError)):
            fm.fm_gemm_w4(**{**good, name: bad})
    with pytest.raises(fm.FluxMIError):      # 16-bit output of another type: refused by the library
        fm.fm_gemm_w4(x, p, s, c.half(), 32)
    with pytest.raises(fm.FluxMIError):      # a row that starts between 16-byte boundaries
        fm.fm_gemm_w4(x.view(-1)[4:260].view(1, 256), p, s, c[:1], 32)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("M", [1, 3, 20, 50])
def test_one_sided_integers_are_exact(M, dt):
    """Large positive integers, as far from a sum that cancels as an activation's output gets.  A
    group's sum of x (16 + code) is at most 128 * 2047 * 31 < 2^24, and so are its sum of x times
    (16 + zero) and what the groups add up to (asserted): every number on the way is an integer
    below 2^24, and the result exact, in whatever order it is summed."""
    import torch
    say(f"w4 one-sided M={M} {dt}")
    K, N, group = 1024, 40, 128
    rng = np.random.default_rng(M)
    top = {"bf16": 256, "fp16": 2048}[dt]
    x = rng.integers(top - top // 8, top, (M, K)).astype(np.float64)
    codes = rng.integers(0, 16, (K, N)).astype(np.uint8)
    zeros = rng.integers(5, 11, (K // group, N)).astype(np.uint8)
    W = ob.w4_matrix(codes, np.ones((K // group, N)), zeros, group)
    parts = np.einsum("mgk,gkn->gmn", x.reshape(M, -1, group), W.reshape(-1, group, N))
    assert np.abs(parts).sum(axis=0).max() < 2 ** 24
    one = torch.ones(K // group, N, device="cuda:0").to(_dtype(dt))
    c = torch.empty(M, N, device="cuda:0")
    fm.fm_gemm_w4(_dev(x, dt), _pack(codes), one, c, group, zeros=_dev(zeros))
    assert not (_host(c) != x @ W).any()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 12, 60])
def test_one_sided_integers_through_an_expert_are_exact(oracle, T, dt):
    """The same through the experts' forms: scaled to 16-bit outputs by nothing (the combine's out is
    fp32), with weights of 1 or 0.5 and sums that stay integers or halves below 2^23."""
    say(f"w4 one-sided experts T={T} {dt}")
    E, K, N, topk, group = 4, 512, 40, 2, 128
    rng = np.random.default_rng(T)
    top = {"bf16": 256, "fp16": 2048}[dt]
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :topk].astype(np.int32)
    roff, rsp = oracle.moe_route(ids, 0, E)
    h = rng.integers(top - top // 8, top, (T * topk, K)).astype(np.float64)
    codes = rng.integers(0, 16, (E, K, N)).astype(np.uint8)
    zeros = rng.integers(6, 10, (E, K // group, N)).astype(np.uint8)
    w = rng.choice([0.5, 1.0], (T, topk)).astype(np.float32)
    ref, total = np.zeros((T, N)), np.zeros((T, N))
    for e in range(E):
        p = rsp[roff[e]:roff[e + 1]]
        W = ob.w4_matrix(codes[e], np.ones((K // group, N)), zeros[e], group)
        hr = h[roff[e]:roff[e + 1]]
        np.add.at(ref, p // topk, w.reshape(-1)[p][:, None] * (hr @ W))
        parts = np.einsum("mgk,gkn->gmn", hr.reshape(len(p), K // group, group), W.reshape(-1, group, N))
        np.add.at(total, p // topk, np.abs(parts).sum(axis=0))
    assert total.max() < 2 ** 23
    import torch
    out = torch.empty(T, N, device="cuda:0")
    fm.fm_moe_gemm_scatter_w4(_dev(h, dt), _pack(codes), torch.ones(E, K // group, N, device="cuda:0").to(_dtype(dt)),
                              _dev(ids), _dev(rsp.astype(np.int32)), _dev(roff.astype(np.int32)), _dev(w), out, 0,
                              group, fm.moe_w4_workspace(T, topk, N), zeros=_dev(zeros))
    assert not (_host(out) != ref).any()


ONE_TOKEN = [  # T, hidden, ffn, E, nl, e0, topk, group, dt, zeros, act: at most three pairs
    (1, 264, 72, 8, 8, 0, 1, 32, "bf16", True, 3),         # one pair
    (1, 264, 72, 8, 8, 8, 1, 32, "bf16", True, 3),         # ... of another rank
    (1, 4096, 2816, 4, 4, 0, 1, 128, "fp16", False, 2),
    (1, 136, 16392, 2, 2, 0, 1, 64, "bf16", True, 0),      # two tiles a block, the last block's second past N
    (1, 24576, 40, 3, 3, 0, 1, 32, "fp16", True, 1),
    (1, 72, 2816, 8, 8, 0, 2, 128, "bf16", False, 3),      # three steps of a wave on each of two pairs
    (1, 72, 2816, 8, 4, 0, 2, 64, "fp16", True, 0),
    (1, 40, 1288, 4, 4, 0, 2, 32, "bf16", True, 2),        # a wave without steps, a short last block
    (1, 40, 2816, 8, 8, 0, 3, 64, "fp16", True, 3),
    (1, 56, 16384, 8, 8, 0, 3, 128, "bf16", False, 0),     # three rows nearly fill LDS
    (1, 24, 12296, 8, 4, 2, 3, 32, "fp16", True, 1),
    (3, 88, 1160, 4, 4, 0, 1, 32, "bf16", True, 0),
    (3, 88, 2824, 8, 4, 4, 1, 64, "fp16", True, 2),
    (2, 2056, 1416, 4, 4, 0, 1, 128, "bf16", False, 3),
    (2, 8, 136, 3, 1, 1, 1, 32, "fp16", True, 0),
]


@pytest.mark.parametrize("T,hidden,ffn,E,nl,e0,topk,group,dt,zeros,act", ONE_TOKEN)
def test_gather_w4_of_few_pairs(oracle, T, hidden, ffn, E, nl, e0, topk, group, dt, zeros, act):
    test_gather_w4(oracle, T, hidden, ffn, E, nl, e0, topk, group, dt, zeros, act)


@pytest.mark.parametrize("T,hidden,ffn,E,nl,e0,topk,group,dt,zeros,act", ONE_TOKEN)
def test_scatter_w4_of_few_pairs(oracle, T, hidden, ffn, E, nl, e0, topk, group, dt, zeros, act):
    test_scatter_w4(oracle, T, hidden, ffn, E, nl, e0, topk, group, dt, zeros, act)


def test_scatter_w4_of_an_expert_named_twice(oracle):
    """Both slots of one token name one expert: two rows, two weights."""
    import torch
    K, N, group = 1416, 40, 64
    rng = np.random.default_rng(8)
    codes, s, z = _weights((3,), K, N, group, "bf16", True, rng)
    h, w = _dev(rng.standard_normal((2, K)), "bf16"), rng.random((1, 2)).astype(np.float32)
    out = torch.empty(1, N, device="cuda:0")
    fm.fm_moe_gemm_scatter_w4(h, _pack(codes), s, _dev(np.array([[5, 5]], np.int32)),
                              _dev(np.array([0, 1], np.int32)), _dev(np.array([0, 2, 2, 2], np.int32)), _dev(w),
                              out, 5, group, fm.moe_w4_workspace(1, 2, N), zeros=z)
    v = _host(h) @ ob.w4_matrix(codes[0], _host(s)[0], z[0].cpu().numpy(), group)
    lim = w.astype(np.float64) @ (_bound(_host(h), _host(s)[0], K, group, "bf16") + 4 * U * np.abs(v))
    assert (np.abs(_host(out) - w.astype(np.float64) @ v) <= lim + 2 * U * np.abs(w @ v)).all()


@pytest.mark.parametrize("N,K,group,dt,out,zeros", [
    (16392, 520, 64, "bf16", "fp32", True),                # two tiles a block
    (32776, 136, 32, "fp16", "fp16", True),                # four
    (65544, 264, 128, "bf16", "bf16", False),              # eight
    (65560, 1032, 32, "fp16", "fp32", False),
])
def test_gemm_w4_of_one_long_row(N, K, group, dt, out, zeros):
    test_gemm_w4(1, N, K, group, dt, out, zeros)
