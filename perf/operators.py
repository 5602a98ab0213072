"""The operators around the quantized layer, as they are measured: the INT8
W8A16 linear layer with bias, activation and residual in its epilogue (the
hyper-connection mixers, lm_head), and the rules on the logits that lm_head
answers with (penalties for repeated tokens, biases, grammar masks,
temperature).

`run` computes an operator in its plain form (torch in 32 bits), or, with
`own` set, through the package's entry points."""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "none": 0}

MIXER = {"op": "linear", "group": 64, "strided": False}
HEAD = {"op": "rules", "vocab": 248320}


def listed():
    return [
        # one decode step's hyper-connection pair: the down projection with
        # its SiLU, the up projection added to the residual stream
        {**MIXER, "name": "mixer down, 1 token", "tokens": 1, "n": 320, "k": 10240, "bias": "none",
         "activation": "silu", "residual": "none", "out": "bf16"},
        {**MIXER, "name": "mixer up, 4 tokens", "tokens": 4, "n": 10240, "k": 320, "bias": "none",
         "activation": "none", "residual": "bf16", "out": "bf16"},
        # a prefill chunk through the same pair
        {**MIXER, "name": "mixer down, 512 tokens", "tokens": 512, "n": 320, "k": 10240, "bias": "bf16",
         "activation": "silu", "residual": "none", "out": "bf16"},
        {**MIXER, "name": "mixer up, 512 tokens", "tokens": 512, "n": 10240, "k": 320, "bias": "none",
         "activation": "none", "residual": "bf16", "out": "bf16"},
        # a long prompt in one pass, the residual stream kept in fp32
        {**MIXER, "name": "mixer up, 8192 tokens", "tokens": 8192, "n": 10240, "k": 320, "bias": "bf16",
         "activation": "none", "residual": "fp32", "out": "fp32"},
        # lm_head for a batch of eight sequences, logits in fp32
        {"op": "linear", "name": "lm_head, 8 tokens", "tokens": 8, "n": 248320, "k": 2560, "group": 128,
         "strided": False, "bias": "none", "activation": "none", "residual": "none", "out": "fp32"},
        # an adapter of odd width inside wider rows
        {"op": "linear", "name": "odd adapter, 77 tokens", "tokens": 77, "n": 1003, "k": 1152, "group": 128,
         "strided": True, "bias": "fp32", "activation": "gelu", "residual": "fp16", "out": "fp16"},
        # one chat stream: a short history, every penalty, a few biased tokens
        {**HEAD, "name": "rules, 1 row", "rows": 1, "history": 512, "biases": 16, "mask": False,
         "logits": "bf16", "out": "fp32", "strided": False},
        # one agent stream deep in its context, its answer held to a grammar
        {**HEAD, "name": "rules, 1 row, long history", "rows": 1, "history": 131072, "biases": 0, "mask": True,
         "logits": "bf16", "out": "fp32", "strided": False},
        # a serving batch with everything on
        {**HEAD, "name": "rules, 64 rows", "rows": 64, "history": 4096, "biases": 300, "mask": True,
         "logits": "bf16", "out": "fp32", "strided": False},
        # the largest batch: short answers so far, bf16 in and out
        {**HEAD, "name": "rules, 256 rows", "rows": 256, "history": 1024, "biases": 0, "mask": True,
         "logits": "bf16", "out": "bf16", "strided": False},
        # a small odd vocabulary in padded rows
        {"op": "rules", "name": "odd rules, 33 rows", "rows": 33, "vocab": 32003, "history": 700, "biases": 40,
         "mask": True, "logits": "fp16", "out": "fp16", "strided": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        group = rng.choice([64, 128])
        tokens = _log(rng, 1, 8192)
        k = group * _log(rng, 1, 10240 // group)
        n = _log(rng, 33, 65536)
        # no more products, outputs or weights than the largest listed case
        n = max(1, min(n, 8192 * 10240 * 320 // (tokens * k), 8192 * 10240 // tokens))
        return {"op": "linear", "tokens": tokens, "n": n, "k": k, "group": group,
                "strided": rng.random() < 0.3, "bias": rng.choice(["none", "bf16", "fp32"]),
                "activation": rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu", "sigmoid"]),
                "residual": rng.choice(["none", "bf16", "fp16", "fp32"]),
                "out": rng.choice(["bf16", "fp16", "fp32"])}
    rows = _log(rng, 1, 256)
    vocab = _log(rng, 1000, 248320)
    history = rng.choice([0, _log(rng, 1, 131072), _log(rng, 1, 131072)])
    return {"op": "rules", "rows": rows, "vocab": vocab, "history": min(history, 262144 // rows),
            "biases": rng.choice([0, _log(rng, 1, 300)]), "mask": rng.random() < 0.6,
            "logits": rng.choice(["bf16", "fp16", "fp32"]), "out": rng.choice(["bf16", "fp16", "fp32"]),
            "strided": rng.random() < 0.3}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _wide(t, extra):
    """The same values inside rows that are `extra` elements longer."""
    wide = torch.zeros(t.shape[0], t.shape[1] + extra, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _prepare_linear(case, g):
    tokens, n, k, group = case["tokens"], case["n"], case["k"], case["group"]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    s = {"group": group, "activation": case["activation"]}
    s["x"] = normal(tokens, k).to(torch.bfloat16)
    s["packed"] = torch.randint(-2**31, 2**31 - 1, (n, k // 4), dtype=torch.int32, device="cuda", generator=g)
    # outputs of about unit size: what the activations bend and the residual meets
    s["scales"] = (normal(n, k // group).abs() * (0.0135 / math.sqrt(k))).to(torch.bfloat16)
    s["bias"] = None if case["bias"] == "none" else (normal(n) * 0.5).to(TYPES[case["bias"]])
    s["residual"] = None if case["residual"] == "none" else normal(tokens, n).to(TYPES[case["residual"]])
    s["out"] = torch.empty(tokens, n, dtype=TYPES[case["out"]], device="cuda")
    if case["strided"]:
        s["x"] = _wide(s["x"], 24)
        s["out"] = _wide(s["out"], 5)
        s["residual"] = None if s["residual"] is None else _wide(s["residual"], 11)
    if own:  # the layer that a program holds: its weights as they are
        from quantized_moe_router_amd.layer import Int8Linear
        s["layer"] = Int8Linear(s["packed"], s["scales"], group, bias=s["bias"], activation=s["activation"])
    return s


def _prepare_rules(case, g):
    rows, vocab, width, nb = case["rows"], case["vocab"], case["history"], case["biases"]

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    s = {"vocab": vocab, "logits": (torch.randn(rows, vocab, device="cuda", generator=g) * 3).to(TYPES[case["logits"]])}
    s["out"] = torch.empty(rows, vocab, dtype=TYPES[case["out"]], device="cuda")
    if case["strided"]:
        s["logits"], s["out"] = _wide(s["logits"], 29), _wide(s["out"], 7)
    s["temperature"] = 0.5 + uniform(rows)
    s["temperature"][1::4] = 0.0   # greedy rows are left unscaled
    if width:
        # text repeats few tokens often; behind a row's length stand stale ids
        ids = (vocab * uniform(rows, width) ** 3).long().clamp_(max=vocab - 1)
        s["history"] = ((ids * 7919) % vocab).to(torch.int32)
        s["lengths"] = (width * (0.5 + 0.5 * uniform(rows))).to(torch.int32)
        s["lengths"][0] = width
        s["lengths"][3::8] = 0     # a request without any token yet
        s["prompts"] = (s["lengths"] * uniform(rows)).to(torch.int32)
        s["repetition"] = 1 + 0.3 * uniform(rows)
        s["repetition"][2::4] = 1.0
        s["frequency"] = uniform(rows) - 0.2
        s["presence"] = uniform(rows)
    if nb:
        s["bias_ids"] = torch.randint(0, vocab, (rows, nb), dtype=torch.int32, device="cuda", generator=g)
        s["bias_values"] = torch.randn(rows, nb, device="cuda", generator=g) * 4
        s["bias_values"][:, ::5] = -math.inf   # banned tokens
        s["bias_lengths"] = (nb * (0.5 + 0.5 * uniform(rows))).to(torch.int32)
    if case["mask"]:
        words = (vocab + 31) // 32
        mask = torch.randint(-2**31, 2**31 - 1, (rows, words), dtype=torch.int32, device="cuda", generator=g)
        mask[uniform(rows, words) < 0.9] = 0       # a grammar allows few tokens,
        mask[1::2] = -1                            # a row without one all,
        mask[7::16] = 0                            # one in a dead end none
        s["mask"] = mask
    if own:  # the rules that a program holds: its tables as they are
        from quantized_moe_router_amd.layer import LogitsRules
        s["rules"] = LogitsRules(vocab, history=s.get("history"), history_lengths=s.get("lengths"),
                                 prompt_lengths=s.get("prompts"), repetition=s.get("repetition"),
                                 frequency=s.get("frequency"), presence=s.get("presence"),
                                 bias_ids=s.get("bias_ids"), bias_values=s.get("bias_values"),
                                 bias_lengths=s.get("bias_lengths"), mask=s.get("mask"),
                                 temperature=s["temperature"])
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = _prepare_linear(case, g) if case["op"] == "linear" else _prepare_rules(case, g)
    s["op"] = case["op"]
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _activate(y, kind):
    if kind == "silu":
        return y / (1 + torch.exp(-y))
    if kind == "gelu":
        return 0.5 * y * torch.special.erfc(y * -math.sqrt(0.5))
    if kind == "gelu_tanh":
        return y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-y))
    return torch.clamp(y, min=0) if kind == "relu" else y


def _linear(s):
    n, words = s["packed"].shape
    codes = s["packed"].view(torch.uint8).view(n, -1, s["group"]).float() - 128
    w = (codes * s["scales"].float().unsqueeze(2)).view(n, 4 * words)
    y = s["x"].float() @ w.T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _activate(y, s["activation"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["out"].dtype)


def _rules(s):
    y = s["logits"].float()
    rows, vocab = y.shape
    row = torch.arange(rows, device=y.device).unsqueeze(1)
    if "history" in s:
        at = torch.arange(s["history"].shape[1], device=y.device).unsqueeze(0)
        live = at < s["lengths"].unsqueeze(1)
        answer = live & (at >= s["prompts"].unsqueeze(1))
        place = (row * vocab + s["history"]).view(-1)
        seen = torch.zeros(rows * vocab, dtype=torch.int32, device=y.device)
        seen.scatter_add_(0, place, live.view(-1).int())
        count = torch.zeros(rows * vocab, dtype=torch.int32, device=y.device)
        count.scatter_add_(0, place, answer.view(-1).int())
        seen, count = seen.view(rows, vocab), count.view(rows, vocab)
        rep = s["repetition"].unsqueeze(1)
        y = torch.where(seen > 0, torch.where(y > 0, y / rep, y * rep), y)
        y = torch.where(count > 0, y - (s["frequency"].unsqueeze(1) * count + s["presence"].unsqueeze(1)), y)
    if "bias_ids" in s:
        width = s["bias_ids"].shape[1]
        at = torch.arange(width, device=y.device).unsqueeze(0)
        order = torch.where(at < s["bias_lengths"].unsqueeze(1), at + 1, 0)
        last = torch.zeros(rows * vocab, dtype=torch.int64, device=y.device)
        last.scatter_reduce_(0, (row * vocab + s["bias_ids"]).view(-1), order.reshape(-1), "amax")
        last = last.view(rows, vocab)
        value = s["bias_values"].gather(1, (last - 1).clamp(min=0))
        y = torch.where(last > 0, y + value, y)
    t = s["temperature"].unsqueeze(1)
    y = torch.where(t > 0, y / t, y)
    if "mask" in s:
        v = torch.arange(vocab, device=y.device)
        allowed = (s["mask"][:, v // 32] >> (v % 32)) & 1
        y = torch.where(allowed > 0, y, -math.inf)
    return y.to(s["out"].dtype)


def run(state):
    if own:
        if state["op"] == "linear":
            return state["layer"].forward(state["x"], residual=state["residual"], out=state["out"])
        return state["rules"].apply(state["logits"], out=state["out"])
    return _linear(state) if state["op"] == "linear" else _rules(state)


def work(case):
    if case["op"] == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        return {"bytes": n * k + 2 * n * (k // case["group"]) + 2 * t * k + n * BYTES[case["bias"]]
                + t * n * (BYTES[case["residual"]] + BYTES[case["out"]]),
                "flops": 2 * t * n * k}
    rows, vocab = case["rows"], case["vocab"]
    lists = 3 * case["history"] + 6 * case["biases"]   # rows are three quarters full on average
    return {"bytes": rows * (vocab * (BYTES[case["logits"]] + BYTES[case["out"]]) + lists
                             + (4 * ((vocab + 31) // 32) if case["mask"] else 0)),
            "flops": 6 * rows * vocab}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_linear(case, s):
    n, k, group = case["n"], case["k"], case["group"]
    x = s["x"].double()
    raw = s["packed"].contiguous().view(torch.uint8)
    y = torch.zeros(case["tokens"], n, dtype=torch.float64, device="cuda")
    for at in range(0, k, group):   # group by group: the scale outside the sum
        q = raw[:, at:at + group].double() - 128.0
        y += torch.mm(x[:, at:at + group].contiguous(), q.t().contiguous()) * s["scales"][:, at // group].double()
    if s["bias"] is not None:
        y += s["bias"].double()
    kind = case["activation"]
    if kind == "silu":
        y = y * torch.sigmoid(y)
    elif kind == "gelu":
        y = y * (torch.special.erfc(-y / math.sqrt(2.0)) / 2)
    elif kind == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)
        y = y * torch.sigmoid(2 * u)
    elif kind == "sigmoid":
        y = torch.sigmoid(y)
    elif kind == "relu":
        y = torch.maximum(y, torch.zeros_like(y))
    if s["residual"] is not None:
        y += s["residual"].double()
    return y


def _exact_rules(case, s):
    host = {k: v.float().cpu().numpy() if v.is_floating_point() else v.cpu().numpy()
            for k, v in s.items() if isinstance(v, torch.Tensor) and k != "out"}
    y = host["logits"].astype(np.float64)
    for r in range(case["rows"]):
        row = y[r]
        if "history" in host:
            said = host["history"][r, :host["lengths"][r]]
            ids = np.unique(said)
            rep = float(host["repetition"][r])
            row[ids] = np.where(row[ids] > 0, row[ids] / rep, row[ids] * rep)
            ids, count = np.unique(said[host["prompts"][r]:], return_counts=True)
            row[ids] -= float(host["frequency"][r]) * count + float(host["presence"][r])
        if "bias_ids" in host:
            pairs = {}
            for j in range(host["bias_lengths"][r]):
                pairs[int(host["bias_ids"][r, j])] = float(host["bias_values"][r, j])
            for i, b in pairs.items():
                row[i] += b
        if host["temperature"][r] > 0:
            row /= float(host["temperature"][r])
        if "mask" in host:
            bits = np.unpackbits(host["mask"][r].view(np.uint8), bitorder="little")[:case["vocab"]]
            row[bits == 0] = -np.inf
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_linear(case, s) if case["op"] == "linear" else _exact_rules(case, s)
