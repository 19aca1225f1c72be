"""The operators around the routed experts, as a serving program calls them: the choice of experts from
router logits, the experts' importances over a batch, and the dense product with its epilogue (the router's
projection, shared experts, projections added to the layer's output).

With ``own`` false, run() computes the plain form in elementary torch operations; with ``own`` true it calls
the library. exact() is the definition in 64 bits, written apart from both.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one token of the fine-grained layer (128 experts, top-8): pure latency
        dict(name="select_token", op="select", T=1, E=128, k=8, dtype="f32", score="softmax", bias=False,
             groups=1, keep=1, renorm=True, scale=1.0),
        # a decode batch of the repaging layer (256 experts, 128 tokens), balanced by a bias, in groups
        dict(name="select_decode_groups", op="select", T=128, E=256, k=8, dtype="f32", score="sigmoid",
             bias=True, groups=8, keep=4, renorm=True, scale=2.5),
        # the fine-grained layer's prefill batch, logits in bf16 (many exact ties)
        dict(name="select_prefill_bf16", op="select", T=8192, E=128, k=8, dtype="bf16", score="softmax",
             bias=False, groups=1, keep=1, renorm=True, scale=1.0),
        # a long prefill of the repaging layer, an odd number of tokens
        dict(name="select_prefill_groups", op="select", T=32767, E=256, k=8, dtype="f32", score="sigmoid",
             bias=True, groups=8, keep=4, renorm=True, scale=2.5),
        # importances from one decode batch
        dict(name="importance_batch", op="importance", T=64, E=128, dtype="f32", score="softmax"),
        # importances over a calibration set, before widths are allocated
        dict(name="importance_calibration", op="importance", T=65536, E=256, dtype="f32", score="softmax"),
        # the router's projection of a decode batch, logits in f32
        dict(name="router_decode", op="linear", M=64, N=128, K=2048, dtype="bf16", out="f32", bias=False,
             act="none", gated=False, residual=False),
        # a single token through a shared expert's down projection, added to the layer's output
        dict(name="down_token", op="linear", M=1, N=7168, K=2048, dtype="bf16", out="bf16", bias=False,
             act="none", gated=False, residual=True),
        # a decode batch through a shared expert's gate and up projections
        dict(name="gated_decode", op="linear", M=128, N=2048, K=7168, dtype="bf16", out="bf16", bias=False,
             act="silu", gated=True, residual=False),
        # odd sizes in fp16 with every part of the epilogue
        dict(name="ragged_f16", op="linear", M=333, N=4097, K=2040, dtype="f16", out="f16", bias=True,
             act="gelu", gated=False, residual=True),
        # a prefill batch through a shared expert's gate and up projections
        dict(name="gated_prefill", op="linear", M=8192, N=2048, K=7168, dtype="bf16", out="bf16", bias=False,
             act="silu", gated=True, residual=False),
        # a dense down projection of the large-expert layer at prefill, with bias and residual
        dict(name="down_prefill", op="linear", M=8192, N=4096, K=14336, dtype="bf16", out="bf16", bias=True,
             act="none", gated=False, residual=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["select", "select", "importance", "linear", "linear", "linear"])
    if op == "select":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log_int(rng, 8, 512 // groups)
        keep = rng.randint(max(1, groups // 2), groups)
        return dict(op=op, T=_log_int(rng, 1, 32768), E=E, k=rng.randint(1, min(16, keep * (E // groups))),
                    dtype=rng.choice(["f32", "bf16", "f16"]), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, keep=keep, renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]))
    if op == "importance":
        return dict(op=op, T=_log_int(rng, 1, 65536), E=_log_int(rng, 8, 512),
                    dtype=rng.choice(["f32", "bf16", "f16"]), score=rng.choice(["softmax", "sigmoid"]))
    dtype, gated = rng.choice(["bf16", "bf16", "f16"]), rng.random() < 0.3
    while True:
        M, N, K = _log_int(rng, 1, 8192), _log_int(rng, 8, 14336), _log_int(rng, 16, 14336)
        if M * N * K * (2 if gated else 1) <= 8192 * 4096 * 14336 and (M + N) * K <= 14336 * 14336:
            break
    if rng.random() < 0.7:  # most widths are multiples of 8; the others are ragged
        N, K = (N + 7) // 8 * 8, (K + 7) // 8 * 8
    return dict(op=op, M=M, N=N, K=K, dtype=dtype, out=rng.choice([dtype, dtype, "f32"]),
                bias=rng.random() < 0.5, act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                gated=gated, residual=rng.random() < 0.5)


def _rows(shape, sigma, dtype, gen):
    """A random matrix whose rows start at multiples of 8 elements (16 bytes of 16-bit values)."""
    pitch = (shape[1] + 7) // 8 * 8
    full = torch.empty((shape[0], pitch), dtype=torch.float32, device="cuda").normal_(0.0, sigma, generator=gen)
    return full.to(dtype)[:, :shape[1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    c, dt = case, DTYPES[case["dtype"]]
    s = {"case": c}
    if c["op"] in ("select", "importance"):
        # experts differ in popularity, tokens in what they ask for
        popular = torch.empty(c["E"], device="cuda").normal_(0.0, 0.7, generator=gen)
        logits = torch.empty((c["T"], c["E"]), device="cuda").normal_(0.0, 1.5, generator=gen)
        s["logits"] = (logits + popular).to(dt)
        s["score"] = "SCORE_" + c["score"].upper()
        if c["op"] == "select":
            s["bias"] = torch.empty(c["E"], device="cuda").normal_(0.0, 0.1, generator=gen) if c["bias"] else None
            s["ids"] = torch.empty((c["T"], c["k"]), dtype=torch.int32, device="cuda")
            s["w"] = torch.empty((c["T"], c["k"]), dtype=torch.float32, device="cuda")
        else:
            s["out"] = torch.empty(c["E"], dtype=torch.float32, device="cuda")
    else:
        out_dt, rows = DTYPES[c["out"]], c["N"] * (2 if c["gated"] else 1)
        s["act"] = "ACT_" + c["act"].upper()
        s["x"] = _rows((c["M"], c["K"]), 1.0, dt, gen)
        s["weight"] = _rows((rows, c["K"]), c["K"] ** -0.5, dt, gen)
        s["bias"] = torch.empty(rows, device="cuda").normal_(0.0, 0.5, generator=gen).to(dt) if c["bias"] else None
        s["residual"] = (torch.empty((c["M"], c["N"]), device="cuda").normal_(generator=gen).to(out_dt)
                         if c["residual"] else None)
        s["out"] = torch.empty((c["M"], c["N"]), dtype=out_dt, device="cuda")
    return s


def _plain_scores(l, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _plain_select(s, c):
    # 64 bits: which experts a token gets is decided between neighbouring values
    scores = _plain_scores(s["logits"].double(), c["score"])
    key = scores if s["bias"] is None else scores + s["bias"].double()
    if c["groups"] > 1:
        T, E, G = c["T"], c["E"], c["groups"]
        best = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values[:, :, :2].sum(dim=2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=key.device).scatter_(1, order, True)
        key = torch.where(kept[:, :, None], key.view(T, G, E // G), -math.inf).view(T, E)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = scores.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return {"ids": ids.to(torch.int32), "w": (c["scale"] * w).float()}


def _plain_act(v, act):
    if act == "relu":
        return torch.clamp(v, min=0.0)
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_linear(s, c):
    v = s["x"].float() @ s["weight"].float().t()
    if s["bias"] is not None:
        v = v + s["bias"].float()
    v = _plain_act(v[:, :c["N"]], c["act"]) * v[:, c["N"]:] if c["gated"] else _plain_act(v, c["act"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(s["out"].dtype)


def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "select":
            return _plain_select(s, c)
        if c["op"] == "importance":
            return _plain_scores(s["logits"].float(), c["score"]).mean(dim=0, dtype=torch.float64).float()
        return _plain_linear(s, c)
    import mixed_precision_expert_b200 as mpe
    if c["op"] == "linear":
        return mpe.linear(s["x"], s["weight"], bias=s["bias"], act=getattr(mpe, s["act"]), gated=c["gated"],
                          residual=s["residual"], out=s["out"])
    score = getattr(mpe, s["score"])
    if c["op"] == "importance":
        return mpe.expert_importance(s["logits"], score=score, out=s["out"])
    mpe.select_experts(s["logits"], c["k"], bias=s["bias"], score=score, n_groups=c["groups"],
                       keep_groups=c["keep"], renormalize=c["renorm"], scale=c["scale"], ids=s["ids"], w=s["w"])
    return {"ids": s["ids"], "w": s["w"]}


def work(case):
    c, size = case, {"f32": 4, "bf16": 2, "f16": 2}
    if c["op"] == "linear":
        rows = c["N"] * (2 if c["gated"] else 1)
        moved = size[c["dtype"]] * (c["M"] * c["K"] + rows * c["K"] + (rows if c["bias"] else 0))
        moved += size[c["out"]] * c["M"] * c["N"] * (2 if c["residual"] else 1)
        return {"bytes": moved, "flops": 2 * c["M"] * rows * c["K"]}
    read = size[c["dtype"]] * c["T"] * c["E"]
    # a score: an exponential, a subtraction or addition and a division
    if c["op"] == "importance":
        return {"bytes": read + 4 * c["E"], "flops": 4 * c["T"] * c["E"]}
    return {"bytes": read + (4 * c["E"] if c["bias"] else 0) + 8 * c["T"] * c["k"], "flops": 3 * c["T"] * c["E"]}


# ---- the definition in 64 bits ---------------------------------------------------------------------------
def _exact_select(s, c):
    l = s["logits"].double().cpu().numpy()
    if c["score"] == "softmax":
        p = np.exp(l - l.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
    else:
        p = np.reciprocal(1.0 + np.exp(-l))
    key = p + (0.0 if s["bias"] is None else s["bias"].double().cpu().numpy())
    T, E = l.shape
    if c["groups"] > 1:
        grouped = key.reshape(T, c["groups"], -1)
        top = np.partition(grouped, grouped.shape[2] - 2, axis=2)[:, :, -2:] if grouped.shape[2] > 1 else grouped
        order = np.argsort(-top.sum(axis=2), axis=1, kind="stable")
        dropped = np.zeros((T, c["groups"]), dtype=bool)
        np.put_along_axis(dropped, order[:, c["keep"]:], True, axis=1)
        key = np.where(np.repeat(dropped, E // c["groups"], axis=1), -np.inf, key)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :c["k"]]
    w = np.take_along_axis(p, ids, axis=1)
    if c["renorm"]:
        w = w / w.sum(axis=1, keepdims=True)
    return {"ids": ids.astype(np.int32), "w": c["scale"] * w}


def _exact_importance(s, c):
    l = s["logits"].double().cpu().numpy()
    if c["score"] == "softmax":
        l = np.exp(l - l.max(axis=1, keepdims=True))
        return (l / l.sum(axis=1, keepdims=True)).sum(axis=0) / len(l)
    return (1.0 / (1.0 + np.exp(-l))).sum(axis=0) / len(l)


def _exact_linear(s, c):
    x, w = s["x"].double(), s["weight"].double()
    b = None if s["bias"] is None else s["bias"].double()

    def product(first):
        v = torch.matmul(x, w[first:first + c["N"]].transpose(0, 1))
        return v if b is None else v.add_(b[first:first + c["N"]])

    v = product(0)
    if c["act"] == "relu":
        v = torch.where(v > 0, v, torch.zeros_like(v))
    elif c["act"] == "silu":
        v = v * torch.reciprocal(1.0 + torch.exp(-v))
    elif c["act"] == "gelu":
        v = v * torch.special.erfc(-v / math.sqrt(2.0)) / 2.0
    elif c["act"] == "gelu_tanh":
        z = math.sqrt(8.0 / math.pi) * (v + 0.044715 * v ** 3)
        v = v * torch.reciprocal(1.0 + torch.exp(-z))  # (1 + tanh(z / 2)) / 2
    if c["gated"]:
        v = v * product(c["N"])
    return v if s["residual"] is None else v.add_(s["residual"].double())


def exact(case, seed):
    s = prepare(case, seed)
    return {"select": _exact_select, "importance": _exact_importance, "linear": _exact_linear}[case["op"]](s, case)
