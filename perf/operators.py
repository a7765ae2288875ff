"""Cases of the operators around a sparse block, for timing and comparison.

  gate        router: logits -> experts and weights of each token, expert counts, balance loss
  gate_bwd    gradient of the weights and of the balance loss with respect to the logits
  norm        norm after a block, gate, scale, residual add, norm before the next block
  norm_bwd    its gradients: residual stream, block output, both norm weights, gate
  gemm_w4     few rows times one matrix of 4-bit weights with group scales
  gather_w4   few tokens through their experts' first 4-bit matrices (route and gather included)
  scatter_w4  the second 4-bit matrices and the weighted sum into the token rows

`run` computes them from elementary torch operations, or, where `own` is true, through the
library's entry points.

Packed 4-bit weights: a [K, N] matrix of codes 0..15 is held as N rows of ceil(K / 128) * 64
bytes.  Each 64-byte block holds 128 k of one column as 16 little-endian words; word 4 q + j holds
k = 32 j + 8 q + 0..7, its nibble p (from the low end) the k offset 2 p for p < 4 and 2 (p - 4) + 1
for p >= 4.  Codes past K are never used.  W[k, n] = (code - zero) * scale, with scale (and zero, 8
if there are none) of group k / group.
"""
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda:0"


def _case(op, **more):
    return dict(op=op, **more)


def listed():
    return [
        # One token of a decode step through the router of 64 experts: pure latency.
        dict(name="gate decode 1", op="gate", T=1, E=64, topk=2, score="softmax", renorm=False, scale=1.0, bias=False, mask=False,
             closed=0, stats=False, type="bf16"),
        # The router of the 16384-token expert-parallel layer in training: 64 experts, top 2, with counts and loss.
        dict(name="gate train 16384x64", op="gate", T=16384, E=64, topk=2, score="softmax", renorm=False, scale=1.0, bias=False,
             mask=False, closed=0, stats=True, type="bf16"),
        # A wide router's backward pass over a padded batch of odd size: sigmoid scores, renormalised top 8.
        dict(name="gate bwd 65521x256", op="gate_bwd", T=65521, E=256, topk=8, score="sigmoid", renorm=True, scale=2.5, bias=False,
             mask=True, closed=0, stats=True, type="fp32"),
        # Three sequences decoding: the norms between two blocks, the fp32 block output as the combine leaves it.
        dict(name="norm decode 3x4096", op="norm", M=3, N=4096, type="bf16", stream="bf16", block="fp32", post=True, pre=True,
             gate=0, scale=1.0),
        # A training step's tokens behind the expert layer, with one gate for every token.
        dict(name="norm train 16384x4096", op="norm", M=16384, N=4096, type="bf16", stream="bf16", block="fp32", post=True, pre=True,
             gate=16384, scale=0.5),
        # The dense layer's width, 8 sequences of 511 tokens, each with its own gate: backward.
        dict(name="norm bwd 4088x12288", op="norm_bwd", M=4088, N=12288, type="fp16", stream="fp32", block="fp32", post=True, pre=True,
             gate=511, scale=1.0),
        # One token through the dense layer's shard, held in 4 bits.
        dict(name="w4 1x6144x12288", op="gemm_w4", M=1, N=6144, K=12288, group=128, zeros=False, type="fp16", out="fp16"),
        # A ragged batch of decoding sequences through the second shard, small groups with zero points, fp32 out.
        dict(name="w4 45x12288x6144", op="gemm_w4", M=45, N=12288, K=6144, group=32, zeros=True, type="bf16", out="fp32"),
        # One token, its two experts of 64 on this rank.
        dict(name="gather w4 1 of 64", op="gather_w4", T=1, hidden=4096, ffn=2816, E=64, topk=2, e0=0, nl=64, group=128, zeros=False,
             act=3, type="bf16"),
        # 61 tokens on one of eight expert-parallel ranks.
        dict(name="gather w4 61 of 8", op="gather_w4", T=61, hidden=4096, ffn=2816, E=64, topk=2, e0=8, nl=8, group=64, zeros=True,
             act=2, type="fp16"),
        # The same single token's second matrices and weighted sum.
        dict(name="scatter w4 1 of 64", op="scatter_w4", T=1, hidden=4096, ffn=2816, E=64, topk=2, e0=0, nl=64, group=128, zeros=False,
             add=False, type="bf16"),
        # 61 tokens, every expert on this rank, added to what the other layers left.
        dict(name="scatter w4 61 of 64", op="scatter_w4", T=61, hidden=4096, ffn=2816, E=64, topk=2, e0=0, nl=64, group=128, zeros=True,
             add=True, type="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _log_8(rng, lo, hi):
    return max(8, 8 * _log_int(rng, max(1, lo // 8), hi // 8))


def draw(rng):
    op = rng.choice(["gate", "gate_bwd", "norm", "norm_bwd", "gemm_w4", "gather_w4", "scatter_w4"])
    t16 = rng.choice(["bf16", "fp16"])
    if op in ("gate", "gate_bwd"):
        E = _log_int(rng, 4, 384)
        topk = rng.randint(1, min(E, 10))
        T = _log_int(rng, 1, max(1, min(65521, 65521 * 256 // E)))
        closed = rng.choice([0, 0, rng.randint(0, E - topk)])
        return _case(op, T=T, E=E, topk=topk, score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5,
                     scale=rng.choice([1.0, 2.5]), bias=op == "gate" and rng.random() < 0.4, mask=rng.random() < 0.5, closed=closed,
                     stats=op == "gate_bwd" or rng.random() < 0.7, type=rng.choice(["bf16", "fp16", "fp32"]))
    if op in ("norm", "norm_bwd"):
        N = _log_8(rng, 64, 16384)
        rows = _log_int(rng, 1, max(1, min(32768, 4088 * 12288 // N)))
        post = rng.random() < 0.7
        pre = rng.random() < 0.8 or not post
        gates = rng.choice([0, 1, 2, 3])  # none, one for all, one per row, one per sequence
        seq = _log_int(rng, 1, rows)
        M = rows // seq * seq
        return _case(op, M=M, N=N, type=t16, stream=rng.choice([t16, "fp32"]), block=rng.choice([t16, "fp32"]), post=post, pre=pre,
                     gate=(0, M, 1, seq)[gates], scale=rng.choice([1.0, 0.5, 0.22]))
    group = rng.choice([32, 64, 128])
    zeros = rng.random() < 0.5
    if op == "gemm_w4":
        K, N = _log_8(rng, 64, 12288), _log_8(rng, 64, 12288)
        if K * N > 12288 * 6144:
            N = max(8, 12288 * 6144 // K // 8 * 8)
        return _case(op, M=_log_int(rng, 1, 45), N=N, K=K, group=group, zeros=zeros, type=t16, out=rng.choice([t16, "fp32"]))
    nl = _log_int(rng, 1, 64)
    E = nl * rng.choice([1, 1, 2, 8])
    hidden, ffn = _log_8(rng, 128, 4096), _log_8(rng, 128, 2816)
    topk = rng.randint(1, min(E, 4))
    T = _log_int(rng, 1, 61 if topk <= 2 else 30)
    e0 = nl * rng.randint(0, E // nl - 1)
    more = {"act": rng.randint(0, 3)} if op == "gather_w4" else {"add": rng.random() < 0.5}
    return _case(op, T=T, hidden=hidden, ffn=ffn, E=E, topk=topk, e0=e0, nl=nl, group=group, zeros=zeros, type=t16, **more)


def _bytes(name):
    return 4 if name == "fp32" else 2


def work(case):
    c = case
    if c["op"] in ("gate", "gate_bwd"):
        n, p = c["T"] * c["E"], c["T"] * c["topk"]
        logits = n * _bytes(c["type"]) * (2 if c["op"] == "gate_bwd" else 1)
        small = c["T"] * c["mask"] + c["E"] * (8 if c["stats"] else 0) + c["E"] * 4 * c["bias"]
        return {"bytes": logits + p * 8 + small, "flops": 8.0 * n}
    if c["op"] in ("norm", "norm_bwd"):
        n, t, s, b = c["M"] * c["N"], _bytes(c["type"]), _bytes(c["stream"]), _bytes(c["block"])
        gates = c["M"] // c["gate"] * c["N"] if c["gate"] else 0
        weights = c["N"] * (c["post"] + c["pre"])
        if c["op"] == "norm":  # block and residual in, residual and normed out
            return {"bytes": n * (b + 2 * s + t * c["pre"]) + t * (gates + weights) + 4 * c["M"] * (c["post"] + c["pre"]), "flops": 12.0 * n}
        # gradients of the normed and of the residual in, residual and block in, both gradients out
        moved = n * (t * c["pre"] + 2 * s + (s if c["pre"] else 0) + b + (b if c["post"] or c["gate"] else 0))
        return {"bytes": moved + (t + 4) * (gates + weights) + 4 * c["M"] * (c["post"] + c["pre"]), "flops": 24.0 * n}
    def matrix(K, N):
        groups = -(-K // c["group"]) * N
        return K * N // 2 + groups * (3 if c["zeros"] else 2)
    if c["op"] == "gemm_w4":
        return {"bytes": matrix(c["K"], c["N"]) + 2 * c["M"] * c["K"] + _bytes(c["out"]) * c["M"] * c["N"],
                "flops": 2.0 * c["M"] * c["N"] * c["K"]}
    hit = c["nl"] * (1 - (1 - c["topk"] / c["E"]) ** c["T"])  # experts that get a token
    pairs = c["T"] * c["topk"] * c["nl"] / c["E"]
    K, N = (c["hidden"], c["ffn"]) if c["op"] == "gather_w4" else (c["ffn"], c["hidden"])
    if c["op"] == "gather_w4":
        rest = 2 * c["T"] * K + pairs * (2 * N + 4) + c["T"] * c["topk"] * 4
    else:
        rest = pairs * 2 * K + c["T"] * N * 4 * (1 + c["add"]) + c["T"] * c["topk"] * 8
    return {"bytes": hit * matrix(K, N) + rest, "flops": 2.0 * pairs * K * N}


# -- inputs ----------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    dt = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    if case["op"] in ("gate", "gate_bwd"):
        T, E, topk = case["T"], case["E"], case["topk"]
        popular = -0.6 * torch.log(torch.arange(E, device=DEV) + 1.0)  # some experts are preferred
        x = 1.5 * normal(T, E) + popular[torch.randperm(E, generator=g, device=DEV)]
        if case["closed"]:  # experts that take no tokens
            x[:, torch.randperm(E, generator=g, device=DEV)[: case["closed"]]] = float("-inf")
        s["logits"] = x.to(dt)
        s["bias"] = 0.1 * normal(E) if case["bias"] else None
        s["mask"] = (uniform(T) < 0.9).to(torch.uint8) if case["mask"] else None
        if case["op"] == "gate":
            s["ids"] = torch.empty(T, topk, dtype=torch.int32, device=DEV)
            s["weights"] = torch.empty(T, topk, device=DEV)
            s["counts"] = torch.empty(E + 1, dtype=torch.int32, device=DEV) if case["stats"] else None
            s["sums"] = torch.empty(E, device=DEV) if case["stats"] else None
            s["loss"] = torch.empty(1, device=DEV) if case["stats"] else None
        else:
            s["ids"], _ = _choose(s["logits"].float(), topk, s["mask"])
            s["counts"] = _counts(s["ids"], T, E, s["mask"])
            s["d_weights"] = normal(T, topk)
            s["d_loss"] = T * (0.5 + uniform(1))  # a scaled loss
            s["d_logits"] = torch.empty_like(s["logits"])
    elif case["op"] in ("norm", "norm_bwd"):
        M, N, G = case["M"], case["N"], (case["M"] // case["gate"] if case["gate"] else 0)
        st, bt = TYPES[case["stream"]], TYPES[case["block"]]
        s["block"] = (1.3 * normal(M, N)).to(bt)
        s["w_post"] = (1 + 0.2 * normal(N)).to(dt) if case["post"] else None
        s["w_pre"] = (1 + 0.2 * normal(N)).to(dt) if case["pre"] else None
        s["gates"] = (0.5 + 0.5 * normal(G, N)).to(dt) if G else None
        s["resid"] = (2.0 * normal(M, N)).to(st)  # forward: the stream before; backward: the stream after
        if case["op"] == "norm":
            s["out"] = torch.empty(M, N, dtype=st, device=DEV)
            s["y"] = torch.empty(M, N, dtype=dt, device=DEV) if case["pre"] else None
            s["rstd_post"] = torch.empty(M, device=DEV) if case["post"] else None
            s["rstd_pre"] = torch.empty(M, device=DEV) if case["pre"] else None
        else:
            s["rstd_post"] = _rstd(s["block"].double()).float().reshape(M) if case["post"] else None
            s["rstd_pre"] = _rstd(s["resid"].double()).float().reshape(M) if case["pre"] else None
            s["d_y"] = normal(M, N).to(dt) if case["pre"] else None
            s["d_out"] = normal(M, N).to(st)
            s["d_resid"] = torch.empty(M, N, dtype=st, device=DEV)
            s["d_block"] = torch.empty(M, N, dtype=bt, device=DEV)
            s["d_w_post"] = torch.empty(N, device=DEV) if case["post"] else None
            s["d_w_pre"] = torch.empty(N, device=DEV) if case["pre"] else None
            s["d_gates"] = torch.empty(G, N, device=DEV) if G else None
    else:
        if case["op"] == "gemm_w4":
            lead, K, N = (), case["K"], case["N"]
        else:
            lead = (case["nl"],)
            K, N = (case["hidden"], case["ffn"]) if case["op"] == "gather_w4" else (case["ffn"], case["hidden"])
        groups = -(-K // case["group"])
        s["packed"] = torch.randint(0, 256, lead + (N, -(-K // 128) * 64), generator=g, device=DEV, dtype=torch.uint8)
        s["scales"] = ((0.6 + 0.8 * uniform(*lead, groups, N)) / (4.6 * K ** 0.5)).to(dt)
        s["zeros"] = torch.randint(5, 11, lead + (groups, N), generator=g, device=DEV, dtype=torch.uint8) if case["zeros"] else None
        if case["op"] == "gemm_w4":
            s["x"] = normal(case["M"], K).to(dt)
            s["out"] = torch.empty(case["M"], N, dtype=TYPES[case["out"]], device=DEV)
        else:
            T, topk, E = case["T"], case["topk"], case["E"]
            s["ids"] = torch.argsort(uniform(T, E), dim=1)[:, :topk].to(torch.int32).contiguous()
            if case["op"] == "gather_w4":
                s["x"] = normal(T, K).to(dt)
                s["h"] = torch.zeros(T * topk, N, dtype=dt, device=DEV)
                s["pairs"] = torch.full((T * topk,), -1, dtype=torch.int32, device=DEV)
                s["offsets"] = torch.empty(case["nl"] + 1, dtype=torch.int32, device=DEV)
            else:
                s["pairs"], s["offsets"], _ = _route(s["ids"], case["e0"], case["nl"])
                s["h"] = (0.7 * normal(T * topk, K)).to(dt)
                s["weights"] = torch.softmax(normal(T, topk), dim=1)
                s["add"] = normal(T, N) if case["add"] else None
                s["out"] = torch.empty(T, N, device=DEV)
    return s


# -- the operators from elementary operations ----------------------------------------


def _choose(keys, topk, mask):
    """Experts of the largest keys, ties to the lowest index; -1 where a key is -inf or the token is masked."""
    top, ids = torch.sort(keys, dim=1, descending=True, stable=True)
    top, ids = top[:, :topk], ids[:, :topk]
    open_ = top > float("-inf")
    if mask is not None:
        open_ = open_ & (mask != 0).unsqueeze(1)
    return torch.where(open_, ids, -1).to(torch.int32).contiguous(), open_


def _counts(ids, T, E, mask):
    """Tokens of each expert, and behind them the number of tokens that are not masked."""
    flat = ids.reshape(-1).long()
    per = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    per.scatter_add_(0, torch.where(flat < 0, E, flat), torch.ones_like(flat, dtype=torch.int32))
    per[E] = T if mask is None else (mask != 0).sum()
    return per


def _scores(x, score):
    """Scores and shares of all experts."""
    if score == "softmax":
        e = torch.exp(x - x.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
        return p, p
    s = 1 / (1 + torch.exp(-x))
    return s, s / s.sum(dim=1, keepdim=True)


def _gate(s):
    x = s["logits"].float()
    score, share = _scores(x, s["score"])
    if s["bias"] is None:
        keys = x
    else:  # the choice is made in 64 bits, next to a border too
        keys = _scores(s["logits"].double(), s["score"])[0] + s["bias"].double()
        keys = torch.where(x == float("-inf"), float("-inf"), keys)
    ids, open_ = _choose(keys, s["topk"], s["mask"])
    w = torch.where(open_, score.gather(1, ids.clamp(min=0).long()), 0)
    if s["renorm"]:
        w = torch.where(open_, w / w.sum(dim=1, keepdim=True), 0)
    out = {"ids": ids, "weights": w * s["scale"]}
    if s["stats"]:
        if s["mask"] is not None:
            share = torch.where((s["mask"] != 0).unsqueeze(1), share, 0)
        counts = _counts(ids, s["T"], s["E"], s["mask"])
        sums = share.sum(dim=0, dtype=torch.float64)
        n = counts[-1].double().clamp(min=1)
        loss = s["E"] / (s["topk"] * n * n) * (counts[:-1].double() * sums).sum()
        out.update(counts=counts, sums=sums.float(), loss=loss.float().reshape(1))
    return out


def _gate_bwd(s):
    x = s["logits"].float()
    score, share = _scores(x, s["score"])
    open_ = s["ids"] >= 0
    at = s["ids"].clamp(min=0).long()
    n = s["counts"][-1].double().clamp(min=1)
    d_share = (s["d_loss"] * s["E"] / (s["topk"] * n * n) * s["counts"][:-1]).float()
    # share = softmax of u, with u = x or log(sigmoid(x)); d u first
    d_u = share * (d_share - (share * d_share).sum(dim=1, keepdim=True))
    d_w = torch.where(open_, s["d_weights"] * s["scale"], 0)
    w = torch.where(open_, score.gather(1, at), 0)
    if s["renorm"]:
        q = w / w.sum(dim=1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny)
        d_u = d_u.scatter_add(1, at, q * (d_w - (q * d_w).sum(dim=1, keepdim=True)))
    elif s["score"] == "softmax":
        d_u = d_u.scatter_add(1, at, w * d_w) - score * (w * d_w).sum(dim=1, keepdim=True)
    else:
        d_u = d_u.scatter_add(1, at, w * d_w)
    d_x = d_u if s["score"] == "softmax" else d_u * (1 / (1 + torch.exp(x)))
    if s["mask"] is not None:
        d_x = torch.where((s["mask"] != 0).unsqueeze(1), d_x, 0)
    return {"d_logits": d_x.to(s["logits"].dtype)}


EPS = 1e-6


def _rstd(x):
    return 1 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS)


def _rows(gates, M):
    """Gates [G, N] as one for each row."""
    G, N = gates.shape
    return gates.float().unsqueeze(1).expand(G, M // G, N).reshape(M, N)


def _norm(s):
    b = s["block"].float()
    out = {}
    if s["post"]:
        r = _rstd(b)
        b = b * r * s["w_post"].float()
        out["rstd_post"] = r.reshape(-1)
    if s["gates"] is not None:
        b = b * _rows(s["gates"], s["M"])
    z = s["resid"].float() + s["scale"] * b
    out["out"] = z.to(TYPES[s["stream"]])
    if s["pre"]:
        r = _rstd(z)
        out["y"] = (z * r * s["w_pre"].float()).to(TYPES[s["type"]])
        out["rstd_pre"] = r.reshape(-1)
    return out


def _norm_bwd(s):
    M, N = s["M"], s["N"]
    out = {}
    dz = s["d_out"].float()
    if s["pre"]:
        dy, hat = s["d_y"].float(), s["resid"].float() * s["rstd_pre"].reshape(M, 1)
        t = dy * s["w_pre"].float()
        dz = dz + s["rstd_pre"].reshape(M, 1) * (t - hat * (t * hat).mean(dim=1, keepdim=True))
        out["d_w_pre"] = (dy * hat).sum(dim=0, dtype=torch.float64).float()
    out["d_resid"] = dz.to(TYPES[s["stream"]])
    b = s["block"].float()
    hat = b * s["rstd_post"].reshape(M, 1) if s["post"] else b
    normed = hat * s["w_post"].float() if s["post"] else b
    d = dz * s["scale"]
    if s["gates"] is not None:
        G = s["gates"].shape[0]
        out["d_gates"] = (d * normed).reshape(G, M // G, N).sum(dim=1, dtype=torch.float64).float()
        d = d * _rows(s["gates"], M)
    if s["post"]:
        out["d_w_post"] = (d * hat).sum(dim=0, dtype=torch.float64).float()
        t = d * s["w_post"].float()
        d = s["rstd_post"].reshape(M, 1) * (t - hat * (t * hat).mean(dim=1, keepdim=True))
    out["d_block"] = d.to(s["block"].dtype)
    return out


def _codes(packed, K):
    """Codes [..., N, K] of packed weights [..., N, bytes]."""
    lead = packed.shape[:-1]
    v = packed.reshape(*lead, -1, 4, 4, 4)  # block, q, j, byte
    v = torch.stack((v & 15, v >> 4), dim=-1).flatten(-2)  # nibbles of a word, from the low end
    v = torch.stack((v[..., :4], v[..., 4:]), dim=-1).flatten(-2)  # in the order of k
    return v.transpose(-3, -2).reshape(*lead, -1)[..., :K]


def _weights(s, K, at=None):
    """W [..., K, N] in 32 bits, of the matrices `at` where that is given."""

    def pick(v):
        return v if at is None else v[at]

    def each_k(v):
        return pick(v).repeat_interleave(s["group"], dim=-2)[..., :K, :].float()

    q = _codes(pick(s["packed"]), K).transpose(-2, -1).float()
    q = q - (each_k(s["zeros"]) if s["zeros"] is not None else 8.0)
    return (q * each_k(s["scales"])).contiguous()


def _products(s, x, at, K):
    """x [places, K], each row times its expert's matrix; the rows behind the last expert's hold anything."""
    at = at.clamp(max=s["nl"] - 1)
    if len(at) < s["nl"]:  # fewer places than experts: only the places' matrices are unpacked
        return torch.matmul(x.unsqueeze(1), _weights(s, K, at)).squeeze(1)
    return torch.matmul(x, _weights(s, K))[at, torch.arange(len(at), device=DEV)]


def _route(ids, e0, nl):
    """(sorted pairs, -1 behind the last; offsets; local expert of each sorted place, nl behind the last)."""
    e = ids.reshape(-1).long() - e0
    e = torch.where((e >= 0) & (e < nl), e, nl)
    at, order = torch.sort(e, stable=True)
    edges = torch.arange(nl + 1, device=ids.device)
    offsets = (e.unsqueeze(0) < edges.unsqueeze(1)).sum(dim=1).to(torch.int32)
    return torch.where(at < nl, order, -1).to(torch.int32), offsets, at


def _act(x, act):
    if act == 1:
        return torch.where(x > 0, x, 0)
    if act == 2:
        return 0.5 * x * (1 + torch.tanh(0.7978845608028654 * (x + 0.044715 * x * x * x)))
    return x / (1 + torch.exp(-x)) if act == 3 else x


def _gather_w4(s):
    pairs, offsets, at = _route(s["ids"], s["e0"], s["nl"])
    h = _products(s, s["x"].float()[pairs.clamp(min=0).long() // s["topk"]], at, s["hidden"])
    mine = at < s["nl"]
    h = torch.where(mine.unsqueeze(1), _act(h, s["act"]), 0)
    return {"h": h.to(TYPES[s["type"]]), "pairs": pairs, "offsets": offsets}


def _scatter_w4(s):
    T, topk = s["T"], s["topk"]
    at = _route(s["ids"], s["e0"], s["nl"])[2]
    mine = at < s["nl"]
    y = _products(s, s["h"].float(), at, s["ffn"])
    w = s["weights"].reshape(-1)[s["pairs"].clamp(min=0).long()]
    y = torch.where(mine.unsqueeze(1), y * w.unsqueeze(1), 0)
    token = torch.where(mine, s["pairs"].long() // topk, T)
    pick = (token.unsqueeze(0) == torch.arange(T, device=DEV).unsqueeze(1)).float()
    out = torch.matmul(pick, y)
    return {"out": out if s["add"] is None else s["add"] + out}


def _gemm_w4(s):
    return {"out": torch.matmul(s["x"].float(), _weights(s, s["K"])).to(s["out"].dtype)}


def run(state):
    if own:
        return _own(state)
    return {"gate": _gate, "gate_bwd": _gate_bwd, "norm": _norm, "norm_bwd": _norm_bwd, "gemm_w4": _gemm_w4, "gather_w4": _gather_w4,
            "scatter_w4": _scatter_w4}[state["op"]](state)


# -- the library's entry points ---------------------------------------------------------


def _own(s):
    import tile_gemm_communication_amd as fm

    op = s["op"]
    if op == "gate":
        if s["stats"] and "ws" not in s:
            s["ws"] = fm.moe_gate_workspace(s["T"], s["E"], device=DEV)
        fm.fm_moe_gate(s["logits"], s["ids"], s["weights"], score=fm.FM_GATE_SIGMOID if s["score"] == "sigmoid" else fm.FM_GATE_SOFTMAX,
                       renormalize=s["renorm"], scale=s["scale"], bias=s["bias"], token_mask=s["mask"], counts=s["counts"],
                       prob_sums=s["sums"], loss=s["loss"], ws=s.get("ws"))
        out = {"ids": s["ids"], "weights": s["weights"]}
        return dict(out, counts=s["counts"], sums=s["sums"], loss=s["loss"]) if s["stats"] else out
    if op == "gate_bwd":
        fm.fm_moe_gate_bwd(s["logits"], s["ids"], s["d_logits"], score=fm.FM_GATE_SIGMOID if s["score"] == "sigmoid" else fm.FM_GATE_SOFTMAX,
                           renormalize=s["renorm"], scale=s["scale"], token_mask=s["mask"], d_weights=s["d_weights"], counts=s["counts"],
                           d_loss=s["d_loss"])
        return {"d_logits": s["d_logits"]}
    if op == "norm":
        fm.fm_norm_residual(s["out"], s["y"], block=s["block"], resid=s["resid"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gates"],
                            scale=s["scale"], eps=EPS, rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"])
        got = {"out": s["out"], "y": s["y"], "rstd_post": s["rstd_post"], "rstd_pre": s["rstd_pre"]}
        return {k: v for k, v in got.items() if v is not None}
    if op == "norm_bwd":
        if "ws" not in s:
            s["ws"] = fm.norm_residual_workspace(s["M"], s["N"], s["M"] // s["gate"] if s["gate"] else 0, device=DEV)
        fm.fm_norm_residual_bwd(s["d_resid"], s["d_block"], out=s["resid"], block=s["block"], d_y=s["d_y"], d_out=s["d_out"],
                                w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gates"], scale=s["scale"], rstd_post=s["rstd_post"],
                                rstd_pre=s["rstd_pre"], d_w_post=s["d_w_post"], d_w_pre=s["d_w_pre"], d_gate=s["d_gates"], ws=s["ws"])
        got = {k: s[k] for k in ("d_resid", "d_block", "d_w_post", "d_w_pre", "d_gates")}
        return {k: v for k, v in got.items() if v is not None}
    if op == "gemm_w4":
        fm.fm_gemm_w4(s["x"], s["packed"], s["scales"], s["out"], s["group"], zeros=s["zeros"])
        return {"out": s["out"]}
    if op == "gather_w4":
        if "ws" not in s:
            s["ws"] = fm.moe_workspace(s["T"], s["topk"], s["hidden"], s["nl"], device=DEV)
        fm.fm_moe_gather_gemm_w4(s["x"], s["ids"], s["packed"], s["scales"], s["h"], s["pairs"], s["offsets"], s["e0"], s["group"], s["ws"],
                                 zeros=s["zeros"], act=s["act"])
        return {"h": s["h"], "pairs": s["pairs"], "offsets": s["offsets"]}
    if "ws" not in s:
        s["ws"] = fm.moe_w4_workspace(s["T"], s["topk"], s["hidden"], device=DEV)
    fm.fm_moe_gemm_scatter_w4(s["h"], s["packed"], s["scales"], s["ids"], s["pairs"], s["offsets"], s["weights"], s["out"], s["e0"], s["group"],
                              s["ws"], zeros=s["zeros"], add=s["add"])
    return {"out": s["out"]}


# -- the definitions, in 64 bits --------------------------------------------------------


def _exact_gate(s):
    x = s["logits"].double()
    T, E, topk = s["T"], s["E"], s["topk"]
    valid = torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"] > 0
    score = torch.softmax(x, dim=1) if s["score"] == "softmax" else torch.sigmoid(x)
    share = score / score.sum(dim=1, keepdim=True)
    left = (x if s["bias"] is None else score + s["bias"].double()).masked_fill(x.isinf(), -torch.inf)
    index = torch.arange(E, device=DEV)
    ids, w = [], []
    for _ in range(topk):  # the largest that is left, the first of equals
        best = left.amax(dim=1, keepdim=True)
        at = torch.where(left == best, index, E).amin(dim=1, keepdim=True)
        fine = (best > -torch.inf) & valid.unsqueeze(1)
        ids.append(torch.where(fine, at, -1))
        w.append(torch.where(fine, torch.gather(score, 1, at), 0))
        left = left.scatter(1, at, -torch.inf)
    ids, w = torch.cat(ids, 1), torch.cat(w, 1)
    if s["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total > 0, total, 1)
    out = {"ids": ids.int(), "weights": w * s["scale"]}
    if s["stats"]:
        counts = torch.stack([(ids == e).sum() for e in range(E)] + [valid.sum()])
        sums = (share * valid.unsqueeze(1)).sum(dim=0)
        n = max(int(counts[-1]), 1)
        out.update(counts=counts.int(), sums=sums, loss=(E * (counts[:-1] / (topk * n)) * (sums / n)).sum().reshape(1))
    return out


def _exact_gate_bwd(s):
    x = s["logits"].double().requires_grad_(True)
    score = torch.softmax(x, dim=1) if s["score"] == "softmax" else torch.sigmoid(x)
    share = score / score.sum(dim=1, keepdim=True)
    used = s["ids"] >= 0
    w = torch.gather(score, 1, torch.where(used, s["ids"], 0).long()) * used
    if s["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total > 0, total, 1)
    valid = torch.ones(s["T"], dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"] > 0
    n = max(int(s["counts"][-1]), 1)
    loss = s["E"] / (s["topk"] * n * n) * (s["counts"][:-1].double() * (share * valid.unsqueeze(1)).sum(dim=0)).sum()
    total = (w * s["scale"] * s["d_weights"].double() * valid.unsqueeze(1)).sum() + loss * s["d_loss"].double().squeeze()
    total.backward()
    return {"d_logits": x.grad}


def _exact_norm(s):
    b, out = s["block"].double(), {}
    if s["post"]:
        rms = (b.square().sum(dim=1) / s["N"] + EPS).sqrt()
        out["rstd_post"] = 1 / rms
        b = b / rms.unsqueeze(1) * s["w_post"].double()
    if s["gates"] is not None:
        b = (b.reshape(-1, s["gate"], s["N"]) * s["gates"].double().unsqueeze(1)).reshape(s["M"], s["N"])
    z = s["resid"].double() + s["scale"] * b
    out["out"] = z
    if s["pre"]:
        rms = (z.square().sum(dim=1) / s["N"] + EPS).sqrt()
        out["rstd_pre"] = 1 / rms
        out["y"] = z / rms.unsqueeze(1) * s["w_pre"].double()
    return out


def _exact_norm_bwd(s):
    def leaf(v):
        return v.double().requires_grad_(True) if v is not None else None

    def normed(v, w):
        return v / (v.square().sum(dim=1, keepdim=True) / s["N"] + EPS).sqrt() * w

    out = {}
    dz = s["d_out"].double()
    if s["pre"]:
        z, w = leaf(s["resid"]), leaf(s["w_pre"])
        normed(z, w).backward(s["d_y"].double())
        dz = dz + z.grad
        out["d_w_pre"] = w.grad
    out["d_resid"] = dz
    b, w, gates = leaf(s["block"]), leaf(s["w_post"]), leaf(s["gates"])
    v = normed(b, w) if s["post"] else b
    if gates is not None:
        v = (v.reshape(-1, s["gate"], s["N"]) * gates.unsqueeze(1)).reshape(s["M"], s["N"])
    (v * s["scale"]).backward(dz)
    out["d_block"] = b.grad
    if s["post"]:
        out["d_w_post"] = w.grad
    if gates is not None:
        out["d_gates"] = gates.grad
    return out


def _exact_matrix(s, e, K):
    """One expert's W [K, N] in 64 bits, word by word."""
    packed = s["packed"] if e is None else s["packed"][e]
    scales = s["scales"] if e is None else s["scales"][e]
    zeros = s["zeros"] if e is None or s["zeros"] is None else s["zeros"][e]
    N = packed.shape[0]
    words = packed.view(torch.int32).reshape(N, -1, 16)
    q = torch.empty(N, words.shape[1], 128, device=DEV, dtype=torch.float64)
    for w in range(16):
        for p in range(8):
            k = 32 * (w % 4) + 8 * (w // 4) + (2 * p if p < 4 else 2 * p - 7)
            q[:, :, k] = ((words[:, :, w] >> (4 * p)) & 15).double()
    q = q.reshape(N, -1)[:, :K]
    group = torch.arange(K, device=DEV) // s["group"]
    zero = zeros.double().t()[:, group] if zeros is not None else 8.0
    return ((q - zero) * scales.double().t()[:, group]).t()


def _exact_w4(s):
    if s["op"] == "gemm_w4":
        return {"out": s["x"].double() @ _exact_matrix(s, None, s["K"])}
    ids = s["ids"].reshape(-1).tolist()
    places = [(e, p) for e in range(s["nl"]) for p in range(len(ids)) if ids[p] == s["e0"] + e]
    first = [sum(x[0] < e for x in places) for e in range(s["nl"] + 1)]
    first[s["nl"]] = len(places)
    gather = s["op"] == "gather_w4"
    K, N = (s["hidden"], s["ffn"]) if gather else (s["ffn"], s["hidden"])
    out = torch.zeros(len(ids) if gather else s["T"], N, device=DEV, dtype=torch.float64)
    if not gather and s["add"] is not None:
        out += s["add"].double()
    weights = None if gather else s["weights"].double().reshape(-1)
    for e in range(s["nl"]):
        a, b = first[e], first[e + 1]
        if a == b:
            continue
        W = _exact_matrix(s, e, K)
        if gather:
            tokens = torch.tensor([p // s["topk"] for _, p in places[a:b]], device=DEV)
            v = s["x"][tokens].double() @ W
            out[a:b] = {0: v, 1: v.clamp(min=0), 2: torch.nn.functional.gelu(v, approximate="tanh"), 3: v * torch.sigmoid(v)}[s["act"]]
        else:
            p = torch.tensor([p for _, p in places[a:b]], device=DEV)
            out.index_add_(0, p // s["topk"], weights[p].unsqueeze(1) * (s["h"][a:b].double() @ W))
    if not gather:
        return {"out": out}
    pairs = [p for _, p in places] + [-1] * (len(ids) - len(places))
    return {"h": out, "pairs": torch.tensor(pairs, dtype=torch.int32, device=DEV), "offsets": torch.tensor(first, dtype=torch.int32, device=DEV)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"gate": _exact_gate, "gate_bwd": _exact_gate_bwd, "norm": _exact_norm, "norm_bwd": _exact_norm_bwd}.get(case["op"], _exact_w4)(s)
