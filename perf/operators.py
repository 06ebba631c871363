"""What is measured of the routing and dense 4-bit operators: cases, their
inputs, their plain forms in elementary torch operations, and the calls of
this package.

Three operators:

* ``select``: router logits to expert ids and weights (softmax or sigmoid
  scores, a bias that steers the choice, expert groups, top-k, renormalized
  and scaled weights);
* ``backward``: the gradient of those weights with respect to the logits;
* ``linear``: a dense product with 4-bit weights in affine groups, with the
  epilogues of a shared expert (SiLU(gate) * up; scaled rows added to another
  output).
"""

from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _select(name, M, E, k, score, renorm=True, bias=True, groups=1, kept=1, group_top=1, scale=1.0,
            op="select"):
    return dict(name=name, op=op, M=M, E=E, top_k=k, score=score, renormalize=renorm, bias=bias,
                n_group=groups, topk_group=kept, group_top=group_top, scale=scale)


def _linear(name, M, N, K, group, gated=False, row_scale=False, addend=False):
    return dict(name=name, op="linear", M=M, N=N, K=K, group=group, gated=gated,
                row_scale=row_scale, addend=addend)


def listed():
    return [
        # one decoded token of a layer with 256 experts in 8 groups: pure latency
        _select("select_M1_E256_grouped", 1, 256, 8, "sigmoid", True, True, 8, 4, 2, 2.5),
        # a decode batch of the 128-expert layer: softmax, no bias, no groups
        _select("select_M64_E128", 64, 128, 8, "softmax", True, False),
        # a prefill batch of the 60-expert layer, probabilities kept as they are
        _select("select_M2048_E60", 2048, 60, 4, "softmax", False, True),
        # a prefill batch of the 256-expert layer with groups
        _select("select_M8192_E256_grouped", 8192, 256, 8, "sigmoid", True, True, 8, 4, 2, 2.5),
        # the most tokens and experts that the package takes at once
        _select("select_M65536_E512", 65536, 512, 10, "sigmoid", True, True),
        # a training micro-batch of the 60-expert layer: every logit has a gradient
        _select("backward_M2048_E60", 2048, 60, 4, "softmax", False, op="backward"),
        # training batches of the sigmoid-scored layers: a gradient for the chosen experts alone
        _select("backward_M8192_E256", 8192, 256, 8, "sigmoid", True, scale=2.5, op="backward"),
        _select("backward_M65536_E512", 65536, 512, 10, "sigmoid", True, op="backward"),
        # one decoded token through a square projection: the smallest product
        _linear("linear_M1_2048x2048", 1, 2048, 2048, 64),
        # one decoded token through an output head of 128 Ki rows
        _linear("linear_M1_131072x2048", 1, 131072, 2048, 64),
        # a decode batch through a shared expert's gate and up rows (4 experts of 1408 wide)
        _linear("linear_M16_gated_11264x2048", 16, 11264, 2048, 32, gated=True),
        # a prefill batch through its down rows, scaled and added to the routed output
        _linear("linear_M2048_2048x5632_add", 2048, 2048, 5632, 128, row_scale=True, addend=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "backward", "linear", "linear"])
    if op == "linear":
        group = rng.choice([32, 64, 128])
        K = group * max(1, _log_int(rng, 128, 16384) // group)
        gated = rng.random() < 0.3
        N = _log_int(rng, 64, 32768)
        N += N & 1 if gated else 0
        M = _log_int(rng, 1, 2048)
        most = 2048 * 2048 * 5632
        if M * N * K > most:
            M = max(1, most // (N * K))
        return dict(op=op, M=M, N=N, K=K, group=group, gated=gated, row_scale=rng.random() < 0.3,
                    addend=rng.random() < 0.3)
    M = _log_int(rng, 1, 65536)
    score = rng.choice(["softmax", "sigmoid"])
    c = dict(op=op, M=M, score=score, renormalize=rng.random() < 0.6,
             scale=rng.choice([1.0, 1.0, 2.5]))
    groups = rng.choice([1, 1, 2, 4, 8, 16]) if op == "select" else 1
    size = _log_int(rng, 8 if groups == 1 else 2, 512 // groups)
    kept = rng.randint(1, groups)
    # one renormalized weight is constant: its gradient is zero
    least = 2 if op == "backward" and c["renormalize"] else 1
    c.update(E=groups * size, n_group=groups, topk_group=kept,
             group_top=rng.randint(1, 2) if groups > 1 else 1,
             top_k=rng.randint(least, min(kept * size, 16)),
             bias=op == "select" and rng.random() < 0.6)
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32)

    st = dict(case)
    M = case["M"]
    if case["op"] == "linear":
        N, K, group = case["N"], case["K"], case["group"]
        n_out = N // 2 if case["gated"] else N
        # codes uniform; scales and biases that spread the weights about
        # +-sqrt(3 / K), as the package's synthetic quantized layers do
        a = math.sqrt(3.0 / K)
        st["x"] = normal(M, K).to(torch.bfloat16)
        st["weight"] = dict(
            bits=4, group_size=group,
            q=torch.randint(-2 ** 31, 2 ** 31 - 1, (N, K // 8), generator=g, device=DEVICE,
                            dtype=torch.int32),
            scales=(2.0 * a / 15 * (1.0 + 0.1 * normal(N, K // group))).to(torch.bfloat16),
            biases=(-a * (1.0 + 0.1 * normal(N, K // group))).to(torch.bfloat16))
        st["row_scale"] = torch.sigmoid(normal(M)) if case["row_scale"] else None
        st["addend"] = normal(M, n_out).to(torch.bfloat16) if case["addend"] else None
        st["out"] = torch.empty((M, n_out), device=DEVICE, dtype=torch.bfloat16)
        return st
    E, k = case["E"], case["top_k"]
    # router logits of unit-variance tokens and weights of std 0.02 at 2048 features
    st["logits"] = normal(M, E) * 0.9
    # a balance bias is a sum of small steps up and down
    st["select_bias"] = torch.round(normal(E) * 30.0) * 1e-3 if case["bias"] else None
    if case["op"] == "select":
        st["topk_ids"] = torch.empty((M, k), device=DEVICE, dtype=torch.int32)
        st["topk_weights"] = torch.empty((M, k), device=DEVICE, dtype=torch.float32)
    else:
        st["topk_ids"] = torch.sort(st["logits"], dim=1, descending=True, stable=True)[1][
            :, :k].to(torch.int32).contiguous()
        st["grad_weights"] = normal(M, k)
        st["grad_logits"] = torch.empty((M, E), device=DEVICE, dtype=torch.float32)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _scores(logits, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _plain_select(st):
    # in 64 bits: two choice scores may lie next to each other
    M, E = st["logits"].shape
    s = _scores(st["logits"].double(), st["score"])
    if st["select_bias"] is not None:
        c = s + st["select_bias"].double()
    else:
        c = s
    G = st["n_group"]
    if G > 1:
        best = torch.sort(c.view(M, G, E // G), dim=2, descending=True)[0]
        group_score = best[:, :, :st["group_top"]].sum(dim=2)
        order = torch.sort(group_score, dim=1, descending=True, stable=True)[1]
        keep = torch.zeros((M, G), dtype=torch.bool, device=c.device)
        keep.scatter_(1, order[:, :st["topk_group"]], True)
        c = c.masked_fill(~keep.repeat_interleave(E // G, dim=1), -math.inf)
    ids = torch.sort(c, dim=1, descending=True, stable=True)[1][:, :st["top_k"]]
    w = torch.gather(s, 1, ids)
    if st["renormalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    return dict(topk_ids=ids.to(torch.int32), topk_weights=(w * st["scale"]).float())


def _plain_backward(st):
    ids = st["topk_ids"].long()
    s = _scores(st["logits"], st["score"])
    kept = torch.gather(s, 1, ids)
    d = st["grad_weights"] * st["scale"]
    if st["renormalize"]:
        # times each score, the softmax denominator is gone
        kept = kept / kept.sum(dim=1, keepdim=True)
        d = d - (d * kept).sum(dim=1, keepdim=True)
    d = d * kept
    if st["score"] == "sigmoid":
        d = d * (1.0 - torch.gather(s, 1, ids))
    grad = torch.zeros_like(s).scatter_(1, ids, d)
    if st["score"] == "softmax" and not st["renormalize"]:
        grad = grad - s * d.sum(dim=1, keepdim=True)
    return dict(grad_logits=grad)


def _dense_weight(weight, dtype):
    q, group = weight["q"], weight["group_size"]
    N, words = q.shape
    shifts = torch.arange(0, 32, 4, device=q.device, dtype=torch.int32)
    codes = ((q.unsqueeze(2) >> shifts) & 15).to(dtype).view(N, -1, group)
    w = codes * weight["scales"].to(dtype).unsqueeze(2) + weight["biases"].to(dtype).unsqueeze(2)
    return w.view(N, words * 8)


def _plain_linear(st):
    y = st["x"].float() @ _dense_weight(st["weight"], torch.float32).t()
    if st["gated"]:
        gate, up = y.chunk(2, dim=1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    if st["row_scale"] is not None:
        y = y * st["row_scale"].unsqueeze(1)
    if st["addend"] is not None:
        y = y + st["addend"].float()
    return dict(out=y.to(torch.bfloat16))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _routing(st):
    # a program builds its routing rule once, when it loads the model
    if "routing" not in st:
        import mixture_experts_ffn_renorm_amd as moe
        st["routing"] = moe.Routing(
            st["top_k"], score=st["score"], renormalize=st["renormalize"],
            select_bias=st["select_bias"], n_group=st["n_group"], topk_group=st["topk_group"],
            group_top=st["group_top"], scale=st["scale"])
    return st["routing"]


def run(st):
    if own:
        import mixture_experts_ffn_renorm_amd as moe
        if st["op"] == "select":
            ids, w = moe.moe_select(st["logits"], _routing(st), topk_ids=st["topk_ids"],
                                    topk_weights=st["topk_weights"])
            return dict(topk_ids=ids, topk_weights=w)
        if st["op"] == "backward":
            return dict(grad_logits=moe.moe_select_backward(
                st["logits"], st["topk_ids"], st["grad_weights"], _routing(st),
                grad_logits=st["grad_logits"]))
        return dict(out=moe.moe_linear_quantized(
            st["x"], st["weight"], gated=st["gated"], row_scale=st["row_scale"],
            addend=st["addend"], out=st["out"]))
    return {"select": _plain_select, "backward": _plain_backward,
            "linear": _plain_linear}[st["op"]](st)


def work(case):
    M = case["M"]
    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        n_out = N // 2 if case["gated"] else N
        rows = 1 + int(case["addend"])
        return {"bytes": N * K // 2 + 4 * N * (K // case["group"]) + 2 * M * K +
                2 * M * n_out * rows + 4 * M * int(case["row_scale"]),
                "flops": 2 * M * N * K}
    E, k = case["E"], case["top_k"]
    if case["op"] == "select":
        # an exponential, a quotient and a comparison for each logit
        return {"bytes": 4 * M * E + 4 * E * int(case["bias"]) + 8 * M * k, "flops": 4 * M * E}
    dense = case["score"] == "softmax" and not case["renormalize"]
    read = 4 * M * E if dense else 4 * M * k
    return {"bytes": read + 8 * M * k + 4 * M * E, "flops": 8 * M * k + (4 * M * E if dense else 0)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_choice(st):
    """ids by repeated maximum, scores through logarithms."""
    l = st["logits"].double()
    M, E = l.shape
    if st["score"] == "sigmoid":
        s = torch.sigmoid(l)
    else:
        s = torch.exp(l - torch.logsumexp(l, dim=1, keepdim=True))
    c = s.clone() if st["select_bias"] is None else s + st["select_bias"].double()
    low = torch.finfo(torch.float64).min
    rows = torch.arange(M, device=l.device)
    G = st["n_group"]
    if G > 1:
        size = E // G
        score = torch.zeros((M, G), dtype=torch.float64, device=l.device)
        for g in range(G):
            part = c[:, g * size:(g + 1) * size].clone()
            for _ in range(st["group_top"]):
                v, at = part.max(dim=1)
                score[:, g] += v
                part[rows, at] = low
        dropped = torch.ones((M, G), dtype=torch.bool, device=l.device)
        for _ in range(st["topk_group"]):
            top = score.amax(dim=1, keepdim=True)
            first = (score == top).int().argmax(dim=1)
            dropped[rows, first] = False
            score[rows, first] = low
        for g in range(G):
            c[:, g * size:(g + 1) * size][dropped[:, g]] = low
    ids = torch.empty((M, st["top_k"]), dtype=torch.int64, device=l.device)
    for j in range(st["top_k"]):
        top = c.amax(dim=1, keepdim=True)
        ids[:, j] = (c == top).int().argmax(dim=1)
        c[rows, ids[:, j]] = low
    return ids, s


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "select":
        ids, s = _exact_choice(st)
        w = s[torch.arange(ids.shape[0], device=ids.device).unsqueeze(1), ids]
        if case["renormalize"]:
            w = w / w.sum(dim=1, keepdim=True)
        return dict(topk_ids=ids.to(torch.int32), topk_weights=w * case["scale"])
    if case["op"] == "backward":
        # the Jacobian of each score row, contracted: d w_j / d s_i first
        ids = st["topk_ids"].long()
        l = st["logits"].double()
        gw = st["grad_weights"].double()
        if case["score"] == "sigmoid":
            s = torch.sigmoid(l)
        else:
            s = torch.softmax(l, dim=1)
        sk = s.gather(1, ids)
        gs = case["scale"] * gw
        if case["renormalize"]:
            S = sk.sum(dim=1, keepdim=True)
            gs = gs / S - (gs * sk).sum(dim=1, keepdim=True) / S ** 2
        out = torch.zeros_like(s)
        if case["score"] == "sigmoid":
            out.scatter_(1, ids, gs * torch.sigmoid(l.gather(1, ids)) *
                         torch.sigmoid(-l.gather(1, ids)))
        else:
            out.scatter_(1, ids, gs * sk)
            out -= s * (gs * sk).sum(dim=1, keepdim=True)
        return dict(grad_logits=out)
    # x W^T = sum over groups of s * (q . x) + b * (1 . x)
    wt, group = st["weight"], case["group"]
    M, N, K = case["M"], case["N"], case["K"]
    x = st["x"].double()
    sums = x.view(M, K // group, group).sum(dim=2)
    y = torch.empty((M, N), dtype=torch.float64, device=x.device)
    step = max(1, (1 << 26) // K)
    for r in range(0, N, step):
        q = wt["q"][r:r + step].long()
        part = torch.stack([(q >> (4 * i)) & 15 for i in range(8)], dim=2).double()
        part = part.view(-1, K // group, group) * wt["scales"][r:r + step].double().unsqueeze(2)
        y[:, r:r + step] = x @ part.reshape(-1, K).t() + \
            sums @ wt["biases"][r:r + step].double().t()
    if case["gated"]:
        gate, up = y[:, :N // 2], y[:, N // 2:]
        y = gate * torch.sigmoid(gate) * up
    if case["row_scale"]:
        y = y * st["row_scale"].double().unsqueeze(1)
    if case["addend"]:
        y = y + st["addend"].double()
    return dict(out=y)
