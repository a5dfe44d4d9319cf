"""The operators that read compressed weights where a model uses them, as calls
to be timed and compared: the linear product with its epilogue, the embedding
lookup and the embedding table's gradient.

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU,
``run`` makes one pass: with ``own`` false in plain torch operations in 32
bits on the uncompressed weights, with ``own`` true through the package, on
the weights in compressed form.  ``exact`` gives the same outputs from the
definition in 64 bits.
"""
import math

import torch

own = False

# Bytes a compressed Gaussian weight takes: 8 bits of sign and mantissa and a
# Huffman-coded exponent of 2.6 bits on average, chunk positions included.
WEIGHT_BYTES = 1.345
SLAB = 1 << 26  # weights widened at a time in exact()


def listed():
    return [
        # one token's query, key and value projections, with biases, one call
        dict(name="linear_qkv_token", op="linear", rows="4096+1024+1024", cols=4096, tokens=1,
             activation="none", bias=True, multiplier=False, residual=False, out="bf16",
             extras="bf16"),
        # the attention output of six drafted tokens, added to the residual stream
        dict(name="linear_out_drafts", op="linear", rows="4096", cols=4096, tokens=6,
             activation="none", bias=False, multiplier=False, residual=True, out="bf16",
             extras="bf16"),
        # the gate of a gated MLP for a decode batch of 24: silu(gate) * up
        dict(name="linear_gate_batch", op="linear", rows="12288", cols=4096, tokens=24,
             activation="silu", bias=False, multiplier=True, residual=False, out="bf16",
             extras="bf16"),
        # the LM head for a decode batch of eight, fp32 logits for a sampler
        dict(name="linear_head_batch", op="linear", rows="151936", cols=4096, tokens=8,
             activation="none", bias=False, multiplier=False, residual=False, out="fp32",
             extras="fp32"),
        # the down projection of a 2048-token prompt, added to the residual stream
        dict(name="linear_down_prefill", op="linear", rows="4096", cols=12288, tokens=2048,
             activation="none", bias=False, multiplier=False, residual=True, out="bf16",
             extras="bf16"),
        # an odd matrix with every part of the epilogue, a short ragged prompt
        dict(name="linear_ragged", op="linear", rows="1013", cols=1411, tokens=77,
             activation="gelu", bias=True, multiplier=True, residual=True, out="fp32",
             extras="fp32"),
        # one decode step of a batch of four: four rows of the table
        dict(name="embed_step", op="embed", vocab=151936, dim=4096, tokens=4, scale=False,
             out="bf16", ids="int64"),
        # a batch of prompts, scaled by the root of the width
        dict(name="embed_prompts", op="embed", vocab=151936, dim=4096, tokens=8192, scale=True,
             out="bf16", ids="int64"),
        # an odd table and a ragged number of tokens, fp32 out
        dict(name="embed_ragged", op="embed", vocab=50021, dim=1003, tokens=777, scale=True,
             out="fp32", ids="int32"),
        # the gradient of a small tuning step on a smaller table, odd sizes
        dict(name="grad_ragged", op="grad", vocab=5003, dim=333, tokens=300, scale=True,
             out="fp32", grads="fp32", ids="int32"),
        # one training step on a middling table, fp32 gradient for the optimiser
        dict(name="grad_step", op="grad", vocab=32768, dim=1024, tokens=8192, scale=False,
             out="fp32", grads="bf16", ids="int64"),
        # a full table and a large batch of tokens, gradient in BF16
        dict(name="grad_large", op="grad", vocab=151936, dim=4096, tokens=32768, scale=True,
             out="bf16", grads="bf16", ids="int64"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "embed", "grad"])
    if op == "linear":
        cols = _log(rng, 48, 12288)
        rows = _log(rng, 33, min(151936, 620_000_000 // cols))
        tokens = _log(rng, 1, min(2048, max(1, 8 * 10 ** 10 // (rows * cols))))
        if rng.random() < 0.5:  # whole tiles as often as odd sizes
            cols, rows = -(-cols // 64) * 64, -(-rows // 64) * 64
        text = str(rows)
        if rng.random() < 0.25 and rows <= 16384:  # several weights in one call
            text += "+%d" % max(1, rows // 4)
        return dict(op=op, rows=text, cols=cols, tokens=tokens,
                    activation=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                    bias=rng.random() < 0.5, multiplier=rng.random() < 0.3,
                    residual=rng.random() < 0.5, out=rng.choice(["bf16", "fp32"]),
                    extras=rng.choice(["bf16", "fp32"]))
    if op == "embed":
        dim = _log(rng, 40, 8192)
        vocab = _log(rng, 1000, min(151936, 620_000_000 // dim))
        if rng.random() < 0.5:
            dim = -(-dim // 64) * 64
        return dict(op=op, vocab=vocab, dim=dim, tokens=_log(rng, 1, 32_000_000 // dim),
                    scale=rng.random() < 0.5, out=rng.choice(["bf16", "fp32"]),
                    ids=rng.choice(["int32", "int64"]))
    dim = _log(rng, 40, 8192)
    vocab = _log(rng, 1000, min(151936, 300_000_000 // dim))
    if rng.random() < 0.5:
        dim = -(-dim // 64) * 64
    return dict(op=op, vocab=vocab, dim=dim, tokens=_log(rng, 1, min(32768, 100_000_000 // dim)),
                scale=rng.random() < 0.5, out=rng.choice(["bf16", "fp32"]),
                grads=rng.choice(["bf16", "fp32"]), ids=rng.choice(["int32", "int64"]))


TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "int32": torch.int32,
         "int64": torch.int64}


def _scale(case):
    """The root of the width as a 32-bit value, or one."""
    if not case["scale"]:
        return 1.0
    return float(torch.tensor(math.sqrt(case["dim"]), dtype=torch.float32))


def _normal(gen, shape, std, dtype):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)


def _token_ids(gen, case):
    """Tokens as text has them: few common ones, many rare ones (rank r with
    a probability near 1/r)."""
    u = torch.rand(case["tokens"], generator=gen, device="cuda", dtype=torch.float64)
    ids = torch.exp(u * math.log(case["vocab"] + 1.0)).long() - 1
    return ids.clamp_(0, case["vocab"] - 1).to(TYPES[case["ids"]])


def _rows(case):
    return [int(r) for r in case["rows"].split("+")]


def _inputs(case, seed):
    """The inputs of a case, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {}
    if case["op"] == "linear":
        rows, cols, tokens = _rows(case), case["cols"], case["tokens"]
        extras = TYPES[case["extras"]]
        s["x"] = _normal(gen, (tokens, cols), 1.0, torch.bfloat16)
        s["w"] = [_normal(gen, (r, cols), cols ** -0.5, torch.bfloat16) for r in rows]
        s["bias"] = [_normal(gen, (r,), 0.1, extras) if case["bias"] else None for r in rows]
        s["multiplier"] = [_normal(gen, (tokens, r), 1.0, extras) if case["multiplier"] else None
                           for r in rows]
        s["residual"] = [_normal(gen, (tokens, r), 1.0, extras) if case["residual"] else None
                         for r in rows]
    elif case["op"] == "embed":
        s["ids"] = _token_ids(gen, case)
        s["w"] = _normal(gen, (case["vocab"], case["dim"]), 0.02, torch.bfloat16)
    else:
        s["ids"] = _token_ids(gen, case)
        s["grad"] = _normal(gen, (case["tokens"], case["dim"]), 1e-2, TYPES[case["grads"]])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"], s["own"], s["scale"] = case, own, _scale(case) if "scale" in case else 1.0
    if not own:
        return s
    import huffman_decode_df11_b200 as df11
    s["df11"] = df11
    if case["op"] == "linear":
        # the weights once into compressed form, and the call's plan on its buffers
        ds = [df11.compress_linear(w) for w in s.pop("w")]
        ys = [torch.empty(case["tokens"], r, dtype=TYPES[case["out"]], device="cuda")
              for r in _rows(case)]
        s["plan"] = df11.LinearPlan(ds, [s["x"]] * len(ds), ys, biases=s["bias"],
                                    activations=[case["activation"]] * len(ds),
                                    multipliers=s["multiplier"], residuals=s["residual"])
    elif case["op"] == "embed":
        d = df11.compress_on_device(s.pop("w"))
        out = torch.empty(case["tokens"], case["dim"], dtype=TYPES[case["out"]], device="cuda")
        s["plan"] = df11.EmbeddingPlan(d, s["ids"], out, scale=s["scale"])
    return s


def _activate(name, v):
    if name == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _linear_plain(s):
    case, out = s["case"], []
    x = s["x"].float()
    for w, b, m, r in zip(s["w"], s["bias"], s["multiplier"], s["residual"]):
        y = x @ w.float().t()
        if b is not None:
            y = y + b.float()
        y = _activate(case["activation"], y)
        if m is not None:
            y = y * m.float()
        if r is not None:
            y = y + r.float()
        out.append(y.to(TYPES[case["out"]]))
    return out


def _embed_plain(s):
    y = s["w"][s["ids"].long()].float() * s["scale"]
    return [y.to(TYPES[s["case"]["out"]])]


def _grad_plain(s):
    case = s["case"]
    dw = torch.zeros(case["vocab"], case["dim"], dtype=torch.float32, device="cuda")
    dw.index_add_(0, s["ids"].long(), s["grad"].float() * s["scale"])
    return [dw.to(TYPES[case["out"]])]


def run(state):
    op = state["case"]["op"]
    if not state["own"]:
        return {"linear": _linear_plain, "embed": _embed_plain, "grad": _grad_plain}[op](state)
    if op == "grad":
        case = state["case"]
        return [state["df11"].embedding_gradient(state["ids"], state["grad"], case["vocab"],
                                                 scale=state["scale"],
                                                 out_dtype=TYPES[case["out"]])]
    return list(state["plan"].run())


def _distinct(case):
    """Rows of the table that the case's tokens touch, on average."""
    edges = torch.log(torch.arange(1, case["vocab"] + 2, dtype=torch.float64))
    p = (edges[1:] - edges[:-1]) / edges[-1]
    return float((1.0 - torch.pow(1.0 - p, case["tokens"])).sum())


def work(case):
    size = {"bf16": 2, "fp32": 4, "int32": 4, "int64": 8}
    if case["op"] == "linear":
        n, outs = sum(_rows(case)) * case["cols"], sum(_rows(case)) * case["tokens"]
        each = size[case["out"]] + size[case["extras"]] * (case["multiplier"] + case["residual"])
        return {"bytes": n * WEIGHT_BYTES + 2 * case["tokens"] * case["cols"] + outs * each
                + (sum(_rows(case)) * size[case["extras"]] if case["bias"] else 0),
                "flops": 2 * n * case["tokens"]}
    tokens, dim = case["tokens"], case["dim"]
    if case["op"] == "embed":
        return {"bytes": _distinct(case) * dim * WEIGHT_BYTES + tokens * dim * size[case["out"]]
                + tokens * size[case["ids"]],
                "flops": tokens * dim if case["scale"] else 0}
    return {"bytes": tokens * dim * size[case["grads"]] + tokens * size[case["ids"]]
            + case["vocab"] * dim * size[case["out"]],
            "flops": tokens * dim}


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "linear":
        x, outs = s["x"].double(), []
        for i, w in enumerate(s["w"]):
            step = max(1, SLAB // case["cols"])
            z = torch.cat([torch.matmul(x, w[j:j + step].double().transpose(0, 1))
                           for j in range(0, w.shape[0], step)], dim=1)
            if case["bias"]:
                z += s["bias"][i].double()[None, :]
            name = case["activation"]
            if name == "relu":
                z = z.clamp(min=0)
            elif name == "gelu":  # z times the normal distribution's value at z
                z = z * torch.special.ndtr(z)
            elif name == "gelu_tanh":  # (1 + tanh u) / 2 = sigmoid(2 u)
                z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
            elif name == "silu":
                z = z * torch.sigmoid(z)
            if case["multiplier"]:
                z *= s["multiplier"][i].double()
            if case["residual"]:
                z += s["residual"][i].double()
            outs.append(z)
        return outs
    ids = s["ids"].long()
    if case["op"] == "embed":
        return [torch.index_select(s["w"], 0, ids).double().mul_(_scale(case))]
    # tokens in sorted order, each added to its row of a 64-bit table
    order = torch.argsort(ids, stable=True)
    dw = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device=ids.device)
    step = max(1, SLAB // case["dim"])
    for j in range(0, len(order), step):
        part = order[j:j + step]
        dw.index_put_((ids[part],), s["grad"][part].double(), accumulate=True)
    return [dw.mul_(_scale(case))]
