"""The operators around a sparse block on tensors whose offsets pass 32 bits: the last rows (or the
last expert) have the bits that a call on these alone gives."""
import pytest

import tile_gemm_communication_amd as fm
from gpu_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def test_router_rows_past_4_gib():
    import torch
    T, E, topk, n = (1 << 22) + 4321, 264, 4, 512          # 4.4 GB of logits
    say(f"router T={T} E={E}")
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.empty(T, E, device=DEV).normal_(generator=g)
    ids, w = torch.empty(T, topk, dtype=torch.int32, device=DEV), torch.empty(T, topk, device=DEV)
    fm.fm_moe_gate(x, ids, w)
    dx, d_w = torch.empty_like(x), torch.randn(T, topk, generator=g, device=DEV)
    fm.fm_moe_gate_bwd(x, ids, dx, d_weights=d_w)
    for rows in (slice(0, n), slice(T - n, T)):
        i2, w2, dx2 = torch.empty_like(ids[rows]), torch.empty_like(w[rows]), torch.empty_like(x[rows])
        fm.fm_moe_gate(x[rows], i2, w2)
        fm.fm_moe_gate_bwd(x[rows], i2, dx2, d_weights=d_w[rows])
        assert torch.equal(i2, ids[rows]) and torch.equal(w2, w[rows]) and torch.equal(dx2, dx[rows])


def test_norm_rows_past_4_gib():
    import torch
    M, N, n = 140000, 16384, 256                           # 4.6 GB a 16-bit tensor
    say(f"norm M={M} N={N}")
    bf = torch.bfloat16
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    block = torch.empty(M, N, device=DEV, dtype=bf).normal_(generator=g)
    resid = torch.empty(M, N, device=DEV, dtype=bf).normal_(generator=g)
    wq, wp = (1 + 0.1 * torch.randn(2, N, generator=g, device=DEV)).to(bf)
    gate = torch.randn(M // 4, N, generator=g, device=DEV).to(bf)
    out, y = torch.empty_like(resid), torch.empty_like(resid)
    rq, rp = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    fm.fm_norm_residual(out, y, block=block, resid=resid, w_post=wq, w_pre=wp, gate=gate, rstd_post=rq,
                        rstd_pre=rp)
    dz, db = torch.empty_like(out), torch.empty_like(block)
    fm.fm_norm_residual_bwd(dz, db, out=out, block=block, d_y=y, d_out=resid, w_post=wq, w_pre=wp, gate=gate,
                            rstd_post=rq, rstd_pre=rp)
    for r, q in ((slice(0, n), slice(0, n // 4)), (slice(M - n, M), slice((M - n) // 4, M // 4))):
        o2, y2 = torch.empty_like(out[r]), torch.empty_like(y[r])
        fm.fm_norm_residual(o2, y2, block=block[r], resid=resid[r], w_post=wq, w_pre=wp, gate=gate[q])
        assert torch.equal(o2, out[r]) and torch.equal(y2, y[r])
        z2, b2 = torch.empty_like(o2), torch.empty_like(o2)
        fm.fm_norm_residual_bwd(z2, b2, out=o2, block=block[r], d_y=y2, d_out=resid[r], w_post=wq, w_pre=wp,
                                gate=gate[q], rstd_post=rq[r], rstd_pre=rp[r])
        assert torch.equal(z2, dz[r]) and torch.equal(b2, db[r])


@pytest.mark.parametrize("T", [1, 3, 40])
def test_experts_past_4_gib(T):
    """36 matrices of 16384 x 16384 in 4 bits are 4.8 GB: the last expert alone, and among them."""
    import torch
    say(f"w4 experts past 4 GiB T={T}")
    nl, K, N, group, bf = 36, 16384, 16384, 128, torch.bfloat16
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    packed = torch.randint(0, 256, (nl, N, fm.fm_w4_row_bytes(K)), generator=g, device=DEV, dtype=torch.uint8)
    scales = (torch.rand(nl, K // group, N, generator=g, device=DEV) / 128).to(bf)
    zeros = torch.randint(0, 16, (nl, K // group, N), generator=g, device=DEV, dtype=torch.uint8)
    x = torch.randn(T, K, generator=g, device=DEV).to(bf)
    ids = torch.full((T, 1), nl - 1, dtype=torch.int32, device=DEV)
    wts = torch.rand(T, 1, generator=g, device=DEV)
    got = []
    for e0, part in ((0, slice(0, nl)), (nl - 1, slice(nl - 1, nl))):
        n = part.stop - part.start
        h = torch.full((T, N), -7.0, device=DEV, dtype=bf)
        sp = torch.full((T,), -1, dtype=torch.int32, device=DEV)
        off = torch.full((n + 1,), -1, dtype=torch.int32, device=DEV)
        out = torch.full((T, N), -7.0, device=DEV)
        fm.fm_moe_gather_gemm_w4(x, ids, packed[part], scales[part], h, sp, off, e0, group,
                                 fm.moe_workspace(T, 1, K, n), zeros=zeros[part])
        fm.fm_moe_gemm_scatter_w4(h, packed[part], scales[part], ids, sp, off, wts, out, e0, group,
                                  fm.moe_w4_workspace(T, 1, N), zeros=zeros[part])
        assert off[-1].item() == T and sorted(sp.tolist()) == list(range(T))
        got.append((h, out))
    # Each against the dense form on the last matrix.  Their sums run in other orders, each within
    # (K / 32 + 84) u * 62 sum |x| scale of the exact one (the waves' chains where they share tiles).
    rows = scales[nl - 1].float().repeat_interleave(group, 0)

    def dense(x):
        c = torch.empty(T, N, device=DEV)
        fm.fm_gemm_w4(x, packed[nl - 1], scales[nl - 1], c, group, zeros=zeros[nl - 1])
        return c, 2 * (K / 32 + 84) * 2.0 ** -24 * 62 * (x.float().abs() @ rows)

    for h, out in got:
        order = sp.long()                                  # topk 1: place -> token
        c, lim = dense(x[order].contiguous())
        assert ((h.float() - c).abs() <= lim + 2.0 ** -8 * c.abs()).all()
        c, lim = dense(h)
        assert ((out[order] - wts[order] * c).abs() <= wts[order] * (lim + 4 * 2.0 ** -24 * c.abs())).all()


def test_combine_rows_past_4_gib():
    """H of 4.9 GB: the last tokens' sums against a float32 product of their rows."""
    import torch
    T, topk, K, N, E, group, bf = 300000, 2, 4096, 8, 8, 64, torch.bfloat16
    say("combine H past 4 GiB")
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    codes = torch.randint(0, 16, (E, K, N), generator=g, device=DEV, dtype=torch.uint8)
    packed = torch.empty(E, N, fm.fm_w4_row_bytes(K), dtype=torch.uint8, device=DEV)
    fm.fm_w4_pack(codes, packed)
    scales = (torch.rand(E, K // group, N, generator=g, device=DEV) / 300).to(bf)
    ids = torch.rand(T, E, generator=g, device=DEV).topk(topk).indices.int().contiguous()
    h = torch.empty(T * topk, K, device=DEV, dtype=bf).normal_(generator=g)
    sp, off = torch.empty(T * topk, dtype=torch.int32, device=DEV), torch.empty(E + 1, dtype=torch.int32, device=DEV)
    fm.fm_moe_route(ids, 0, E, sp, off, fm.moe_workspace(T, topk, K, E))
    w, out = torch.rand(T, topk, generator=g, device=DEV), torch.empty(T, N, device=DEV)
    fm.fm_moe_gemm_scatter_w4(h, packed, scales, ids, sp, off, w, out, 0, group, fm.moe_w4_workspace(T, topk, N))
    W = (codes.double() - 8) * scales.double().repeat_interleave(group, 1)
    place = torch.empty(T * topk, dtype=torch.long, device=DEV)
    place[sp.long()] = torch.arange(T * topk, device=DEV)
    for t in list(range(0, 40)) + list(range(T - 40, T)):
        ref = sum(w[t, k].double() * (h[place[t * topk + k]].double() @ W[ids[t, k].long()]) for k in range(topk))
        # (K / 256 + 84) u * 62 sum |x| scale, as for every 4-bit product with base 16
        lim = sum(w[t, k].double() * (100 * 2.0 ** -24 * 62 * (h[place[t * topk + k]].double().abs()
                  @ scales[ids[t, k].long()].double().repeat_interleave(group, 0))) for k in range(topk))
        assert ((out[t].double() - ref).abs() <= lim + 4 * 2.0 ** -24 * ref.abs()).all(), t
