"""The operators around a sparse block, on the CPU side: the float64 definitions
against differences and hand-written values, and every refusal of the C
interface (these calls return during validation, so no GPU is touched)."""
import ctypes

import numpy as np
import pytest

import tile_gemm_communication_amd as fm
from oracle import block as ob

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(16)]
ODD = ctypes.c_void_p(0x10008)
ODD2 = ctypes.c_void_p(0x10002)
BIG = 1 << 40
OK, INV, UNS = fm.FM_OK, fm.FM_ERR_INVALID_ARG, fm.FM_ERR_UNSUPPORTED


# -- definitions -----------------------------------------------------------------

def test_gate_by_hand():
    """Two tokens, three experts; ln 2 makes the shares 1/2, 1/4, 1/4."""
    x = np.array([[np.log(2.0), 0.0, 0.0], [-np.inf, -np.inf, 1.0]])
    ids, w, counts, sums, loss = ob.gate(x, 2, ob.SOFTMAX, False, 2.0)
    assert ids.tolist() == [[0, 1], [2, -1]]           # equal keys: the lower expert
    assert np.allclose(w, [[1.0, 0.5], [2.0, 0.0]])
    assert counts.tolist() == [1, 1, 1, 2]
    assert np.allclose(sums, [0.5, 0.25, 1.25])
    assert np.isclose(loss, 3 / (2 * 4) * 2.0)
    ids, w, *_ = ob.gate(x, 2, ob.SOFTMAX, True, 1.0)
    assert np.allclose(w, [[2 / 3, 1 / 3], [1.0, 0.0]])
    ids, w, counts, _, loss = ob.gate(x, 1, ob.SIGMOID, False, 1.0, bias=np.array([0, 1.0, 0]),
                                      mask=np.array([1, 0]))
    assert ids.tolist() == [[1], [-1]] and np.allclose(w, [[0.5], [0.0]])
    assert counts.tolist() == [0, 1, 0, 1]
    assert ob.gate(x, 1, ob.SOFTMAX, False, 1.0, mask=np.zeros(2))[4] == 0.0


def test_balanced_experts_have_loss_one():
    x = np.log(np.full((8, 4), 0.25))
    x[np.arange(8), np.arange(8) % 4] += 1e-9     # each expert chosen twice
    assert np.isclose(ob.gate(x, 1, ob.SOFTMAX, False, 1.0)[4], 1.0)


@pytest.mark.parametrize("score", [ob.SOFTMAX, ob.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 7))
    mask = np.array([1, 1, 0, 1, 1])
    ids, w, counts, _, _ = ob.gate(x, 3, score, renorm, 1.7, mask=mask)
    ids[0, 2], ids[1, 1] = -1, ids[1, 0]          # a slot not taken, an expert named twice
    d_w, d_loss = rng.standard_normal((5, 3)), 11.0
    dx, _ = ob.gate_bwd(x, ids, score, renorm, 1.7, mask, d_w, counts, d_loss)
    for t in range(5):
        for e in range(7):
            h = np.zeros_like(x)
            h[t, e] = 1e-5
            f = [ob.gate_objective(v, ids, score, renorm, 1.7, mask, d_w, counts, d_loss)
                 for v in (x + h, x - h)]
            assert abs((f[0] - f[1]) / 2e-5 - dx[t, e]) < 1e-8


@pytest.mark.parametrize("post,pre,G", [(1, 1, 0), (1, 1, 1), (1, 1, 3), (1, 1, 6), (0, 1, 2),
                                        (1, 0, 6), (0, 1, 0)])
def test_norm_gradient_against_differences(post, pre, G):
    rng = np.random.default_rng(4)
    M, N, eps = 6, 8, 1e-3
    v = {"block": rng.standard_normal((M, N)), "resid": rng.standard_normal((M, N)),
         "w_post": rng.standard_normal(N) if post else None,
         "w_pre": rng.standard_normal(N) if pre else None,
         "gate": rng.standard_normal((G, N)) if G else None}
    d_y, d_out = rng.standard_normal((M, N)), rng.standard_normal((M, N))

    def f(v):
        out, y, *_ = ob.norm(v["block"], v["resid"], v["w_post"], v["w_pre"], v["gate"], 0.7, eps)
        return (out * d_out).sum() + ((y * d_y).sum() if pre else 0.0)

    out, y, rq, rp, _ = ob.norm(v["block"], v["resid"], v["w_post"], v["w_pre"], v["gate"], 0.7, eps)
    g, _ = ob.norm_bwd(d_y if pre else None, d_out, out, v["block"], v["w_post"], v["w_pre"],
                       v["gate"], 0.7, rq, rp)
    for name, x in v.items():
        if x is None:
            continue
        for at in np.ndindex(x.shape):
            h = np.zeros_like(x)
            h[at] = 1e-5
            num = (f(dict(v, **{name: x + h})) - f(dict(v, **{name: x - h}))) / 2e-5
            assert abs(num - g["d_" + name][at]) < 1e-7, (name, at)


def test_packed_bytes_by_hand():
    codes = np.zeros((136, 8), np.uint8)
    codes[0:8, 0] = range(1, 9)            # block 0, word 0
    codes[32, 1] = 5                       # j = 1 -> word 1
    codes[8, 2] = 6                        # q = 1 -> word 4
    codes[128 + 1, 3] = 7                  # second block, odd k -> nibble 4
    b = ob.w4_pack(codes)
    assert b.shape == (8, 128)
    assert b[0, :4].tolist() == [0x31, 0x75, 0x42, 0x86]
    assert b[1, 4] == 5 and b[2, 16] == 6 and b[3, 64 + 2] == 7
    assert b.sum() == 0x31 + 0x75 + 0x42 + 0x86 + 5 + 6 + 7


# -- refusals ---------------------------------------------------------------------

pytestmark = pytest.mark.usefixtures("built_library")


def gate_call(dt=1, T=16, E=64, topk=2, score=0, renorm=0, logits=P[0], bias=None, mask=None,
              ids=P[1], w=P[2], counts=P[3], sums=P[4], loss=P[5], ws=P[6], n=BIG):
    return fm.lib().fm_moe_gate(dt, T, E, topk, score, renorm, 1.0, logits, bias, mask, ids, w,
                                counts, sums, loss, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=3), UNS), (dict(T=-1), INV), (dict(E=0), INV), (dict(E=1025), INV),
    (dict(topk=0), INV), (dict(topk=17), INV), (dict(E=4, topk=5), INV), (dict(score=2), INV),
    (dict(renorm=2), INV), (dict(logits=None), INV), (dict(logits=ODD), INV),
    (dict(ids=None), INV), (dict(w=None), INV), (dict(ids=ODD2), INV), (dict(bias=ODD2), INV),
    (dict(counts=None), INV), (dict(sums=None), INV), (dict(loss=None), INV),
    (dict(ws=None), INV), (dict(ws=ODD), INV), (dict(n=16), INV), (dict(T=1 << 31), UNS),
    (dict(T=0, counts=None, sums=None, loss=None, logits=None, ids=None, w=None), OK),
])
def test_gate_refusals(kw, want):
    assert gate_call(**kw) == want


def gate_bwd_call(dt=1, T=16, E=64, topk=2, score=0, renorm=0, logits=P[0], mask=None, ids=P[1],
                  dw=P[2], counts=P[3], dl=P[4], dx=P[5]):
    return fm.lib().fm_moe_gate_bwd(dt, T, E, topk, score, renorm, 1.0, logits, mask, ids, dw,
                                    counts, dl, dx, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=-1), UNS), (dict(T=-1), INV), (dict(E=1025), INV), (dict(topk=17), INV),
    (dict(score=-1), INV), (dict(renorm=-1), INV), (dict(logits=None), INV), (dict(ids=None), INV),
    (dict(counts=None), INV), (dict(dl=None), INV), (dict(dx=None), INV), (dict(dx=ODD), INV),
    (dict(dx=P[0]), INV), (dict(T=0, dx=None, logits=None), OK),
])
def test_gate_bwd_refusals(kw, want):
    assert gate_bwd_call(**kw) == want


def norm_call(dt=1, sd=1, bd=2, M=16, N=64, block=P[0], resid=P[1], wq=P[2], wp=P[3], gate=P[4],
              G=4, eps=1e-6, out=P[5], y=P[6], rq=P[7], rp=P[8]):
    return fm.lib().fm_norm_residual(dt, sd, bd, M, N, block, resid, wq, wp, gate, G, 1.0, eps,
                                     out, y, rq, rp, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2, sd=2), UNS), (dict(sd=0), UNS), (dict(bd=0), UNS), (dict(M=-1), INV),
    (dict(N=60), INV), (dict(N=16392), UNS), (dict(M=1 << 31), UNS), (dict(G=3), INV),
    (dict(G=0), INV), (dict(G=32), INV), (dict(gate=None), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(y=None), INV), (dict(wp=None), INV),
    (dict(block=None), INV), (dict(block=None, wq=None, rq=None), INV), (dict(wq=None), INV),
    (dict(wp=None, y=None), INV), (dict(out=ODD), INV), (dict(resid=ODD), INV), (dict(rp=ODD2), INV),
    (dict(block=None, resid=None, wq=None, rq=None, gate=None, G=0), INV),
    (dict(out=None, y=None, wp=None, rp=None), INV), (dict(M=0), OK), (dict(N=0), OK),
])
def test_norm_refusals(kw, want):
    assert norm_call(**kw) == want


def norm_bwd_call(dt=1, sd=1, bd=2, M=16, N=64, dy=P[0], do=P[1], out=P[2], block=P[3], wq=P[4],
                  wp=P[5], gate=P[6], G=4, rq=P[7], rp=P[8], dr=P[9], db=P[10], dwq=P[11],
                  dwp=P[12], dg=P[13], ws=P[14], n=BIG):
    return fm.lib().fm_norm_residual_bwd(dt, sd, bd, M, N, dy, do, out, block, wq, wp, gate, G,
                                         1.0, rq, rp, dr, db, dwq, dwp, dg, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2, sd=2), UNS), (dict(N=12), INV), (dict(G=5), INV), (dict(dy=None), INV),
    (dict(wp=None, dwp=None), INV), (dict(out=None), INV), (dict(rp=None), INV),
    (dict(block=None), INV), (dict(rq=None), INV), (dict(wq=None), INV), (dict(gate=None, G=0), INV),
    (dict(ws=None), INV), (dict(n=1000), INV), (dict(ws=ODD), INV), (dict(dr=ODD), INV),
    (dict(dy=None, do=None, wp=None, dwp=None, rp=None), INV),
    (dict(dr=None, db=None, dwq=None, dwp=None, dg=None), INV), (dict(N=0), OK),
    (dict(M=0, dwq=None, dwp=None, dg=None), OK),
])
def test_norm_bwd_refusals(kw, want):
    assert norm_bwd_call(**kw) == want


def gemm_w4_call(ab=1, c=2, M=4, N=64, K=64, group=32, a=P[0], w=P[1], s=P[2], z=None, out=P[3]):
    return fm.lib().fm_gemm_w4(ab, c, M, N, K, group, a, w, s, z, out, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ab=2), UNS), (dict(ab=0, c=1), UNS), (dict(M=-1), INV), (dict(N=12), INV),
    (dict(K=12), INV), (dict(group=16), INV), (dict(a=None), INV), (dict(w=None), INV),
    (dict(s=None), INV), (dict(w=ODD), INV), (dict(out=None), INV), (dict(out=ODD), INV),
    (dict(K=1 << 22), UNS), (dict(M=1 << 31), UNS), (dict(M=0), OK), (dict(N=0), OK),
])
def test_gemm_w4_refusals(kw, want):
    assert gemm_w4_call(**kw) == want


def gather_w4_call(dt=1, T=16, hidden=64, ffn=64, topk=2, e0=0, nl=8, group=32, x=P[0], ids=P[1],
                   w=P[2], s=P[3], z=None, h=P[4], sp=P[5], off=P[6], act=0, ws=P[7], n=BIG):
    return fm.lib().fm_moe_gather_gemm_w4(dt, T, hidden, ffn, topk, e0, nl, group, x, ids, w, s, z,
                                          h, sp, off, act, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), UNS), (dict(T=-1), INV), (dict(hidden=60), INV), (dict(ffn=12), INV),
    (dict(topk=0), INV), (dict(nl=65), INV), (dict(nl=0), INV), (dict(group=48), INV),
    (dict(x=None), INV), (dict(ids=None), INV), (dict(w=None), INV), (dict(s=None), INV),
    (dict(h=None), INV), (dict(sp=None), INV), (dict(off=None), INV), (dict(act=4), INV),
    (dict(act=-1), INV), (dict(ws=None), INV), (dict(n=64), INV), (dict(T=1 << 30), UNS),
])
def test_gather_w4_refusals(kw, want):
    assert gather_w4_call(**kw) == want


def scatter_w4_call(dt=1, T=16, hidden=64, ffn=64, topk=2, e0=0, nl=8, group=32, h=P[0], w=P[1],
                    s=P[2], z=None, ids=P[3], sp=P[4], off=P[5], tw=P[6], add=None, out=P[7],
                    ws=P[8], n=BIG):
    return fm.lib().fm_moe_gemm_scatter_w4(dt, T, hidden, ffn, topk, e0, nl, group, h, w, s, z, ids,
                                           sp, off, tw, add, out, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), UNS), (dict(T=-1), INV), (dict(hidden=60), INV), (dict(ffn=12), INV),
    (dict(topk=0), INV), (dict(nl=65), INV), (dict(group=0), INV), (dict(h=None), INV),
    (dict(w=None), INV), (dict(s=None), INV), (dict(ids=None), INV), (dict(sp=None), INV),
    (dict(off=None), INV), (dict(tw=None), INV), (dict(out=None), INV), (dict(add=ODD), INV),
    (dict(ws=None), INV), (dict(n=64), INV), (dict(T=0), OK), (dict(hidden=0), OK),
])
def test_scatter_w4_refusals(kw, want):
    assert scatter_w4_call(**kw) == want


def test_pack_refusals_and_sizes():
    L = fm.lib()
    assert L.fm_w4_pack(-1, 64, 64, P[0], P[1], None) == INV
    assert L.fm_w4_pack(1, 60, 64, P[0], P[1], None) == INV
    assert L.fm_w4_pack(1, 64, 64, None, P[1], None) == INV
    assert L.fm_w4_pack(1, 64, 64, P[0], ODD, None) == INV
    assert L.fm_w4_pack(0, 64, 64, None, None, None) == OK
    assert [fm.fm_w4_row_bytes(k) for k in (0, 8, 128, 136, 2816)] == [0, 64, 64, 128, 1408]
    assert L.fm_w4_row_bytes(-8) == 0
    assert fm.fm_moe_w4_workspace_bytes(4, 2, 64) == 4 * 2 * 64 * 4
    assert fm.fm_moe_w4_workspace_bytes(-1, 2, 64) == 0
    assert fm.fm_moe_gate_workspace_bytes(16, 0) == 0 and fm.fm_moe_gate_workspace_bytes(0, 4) > 0
    assert fm.fm_norm_residual_workspace_bytes(16, 64, 5) == 0
    assert fm.fm_norm_residual_workspace_bytes(16, 64, 4) > 0


def test_token_counts_past_every_index():
    """Products of such a T wrap round; the counts themselves are refused."""
    T = 1 << 61
    assert gate_call(T=T, topk=16) == UNS and gate_bwd_call(T=T, topk=16) == UNS
    assert gather_w4_call(T=T) == UNS and scatter_w4_call(T=T, topk=8) == UNS
    assert fm.fm_moe_gate_workspace_bytes(T, 64) == 0
    assert fm.fm_moe_w4_workspace_bytes(T, 8, 64) == 0


def _native():
    pytest.importorskip("torch")
    fm.lib()
    from tile_gemm_communication_amd import _fluxmi
    return _fluxmi


def test_binding_refuses_tensors_it_cannot_pass():
    """The checks stand before any call of the library, so host tensors do."""
    import torch
    m = _native()
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)

    def refused(error, text, f, *args):
        with pytest.raises(error, match=text):
            f(0, 0, *args)

    refused(ValueError, "logits must live on the current GPU", m.moe_gate, x, i, torch.zeros(4, 2), 0,
            0, 1.0, None, None, None, None, None, None)
    refused(TypeError, "unsupported dtype", m.moe_gate, x.double(), i, x, 0, 0, 1.0, None, None, None,
            None, None, None)
    refused(TypeError, "logits must be a tensor", m.moe_gate, 3, i, x, 0, 0, 1.0, None, None, None,
            None, None, None)
    refused(ValueError, "topk_ids must be a matrix", m.moe_gate_bwd, x, None, x, 0, 0, 1.0, None, None,
            None, None)
    refused(ValueError, "must live", m.norm_residual, x, None, None, x, None, None, None, 1.0, 1e-6,
            None, None)
    refused(ValueError, "block or resid must be a matrix", m.norm_residual, None, None, None, None,
            None, None, None, 1.0, 1e-6, None, None)
    refused(ValueError, "group must be", m.gemm_w4, x, x, x, x, 48, None)
    refused(ValueError, "packed must have three dimensions", m.moe_gather_gemm_w4, x, i, x, x, x, i, i,
            0, 32, None, None, 0)
    refused(ValueError, "too short", m.moe_gather_gemm_w4, x, i, torch.zeros(2, 8, 64), x, x, i[:, 0],
            i, 0, 32, None, None, 0)
    with pytest.raises(TypeError, match="wrong number"):
        m.gemm_w4(0, 0)
    with pytest.raises(ValueError):
        fm.fm_norm_residual(None, None, resid=x)
    with pytest.raises(ValueError):
        fm.fm_norm_residual_bwd(x, None)
    with pytest.raises(ValueError):
        fm.fm_w4_pack(x, x)


NONE = dict(block=None, resid=None, out=None, y=None, rq=None, rp=None)


@pytest.mark.parametrize("kw", [dict(M=0), dict(M=0, gate=None, G=0), dict(M=0, wq=None, gate=None, G=0),
                                dict(M=0, wp=None), dict(M=0, G=1)])
def test_norm_of_no_rows(kw):
    """Tensors without rows have no address; weights have."""
    assert norm_call(**NONE, **kw) == OK
    grads = dict(dy=None, do=None, out=None, block=None, rq=None, rp=None, dr=None, db=None,
                 dwq=None, dwp=None, dg=None, ws=None, n=0)
    assert norm_bwd_call(**grads, **kw) == OK


def test_norm_of_no_rows_still_checks_the_rest():
    assert norm_call(**NONE, M=0, dt=2, sd=2) == UNS and norm_call(**NONE, M=0, N=60) == INV
    assert norm_call(**NONE, M=0, eps=-1.0) == INV


def test_binding_refuses_scalars_past_32_bits():
    """The C interface takes 32 bits: a larger number is refused, not cut to its low half."""
    import torch
    m = _native()
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    p, off, big = torch.zeros(2, 8, 64, dtype=torch.uint8), torch.zeros(3, dtype=torch.int32), 1 << 32
    s, sp = torch.zeros(2, 1, 8), torch.zeros(8, dtype=torch.int32)
    h = torch.zeros(8, 8)
    calls = [("score", m.moe_gate, (x, i, x, big, 0, 1.0, None, None, None, None, None, None)),
             ("renormalize", m.moe_gate, (x, i, x, 0, -big, 1.0, None, None, None, None, None, None)),
             ("score", m.moe_gate_bwd, (x, i, x, big + 1, 0, 1.0, None, None, None, None)),
             ("expert_begin", m.moe_gather_gemm_w4, (x, i, p, s, h, sp, off, big, 32, None, None, 0)),
             ("act", m.moe_gather_gemm_w4, (x, i, p, s, h, sp, off, 0, 32, None, None, big)),
             ("expert_begin", m.moe_gemm_scatter_w4, (h, p, s, i, sp, off, x[:, :2], x, -big, 32, None, None,
                                                      None))]
    for name, f, args in calls:
        with pytest.raises(ValueError, match=name + " does not fit"):
            f(0, 0, *args)
    with pytest.raises(TypeError):
        m.moe_gate(0, 0, x, i, x, "0", 0, 1.0, None, None, None, None, None, None)
    with pytest.raises(OverflowError):
        m.moe_gate(0, 0, x, i, x, 1 << 64, 0, 1.0, None, None, None, None, None, None)
