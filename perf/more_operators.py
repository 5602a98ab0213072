"""What a draft head runs beside the quantized layer, as it is measured: the
INT4 linear layer (its projections), the INT4 products grouped by expert (its
experts one product at a time, over the tables that the routing answers), and
the verification of drafted tokens against the target's logits.

`run` computes an operator in its plain form (torch in 32 bits; the choice of
tokens, which falls between borders, in 64), or, with `own` set, through the
package's entry points."""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "none": 0}

LINEAR = {"op": "linear", "group": 128, "strided": False, "bias": "none", "activation": "none", "residual": "none"}
GROUPED = {"op": "grouped", "group": 128, "experts": 512, "top_k": 10, "bias": "none", "activation": "none"}
VERIFY = {"op": "verify", "vocab": 248320, "strided": False}


def listed():
    return [
        # one drafted token through a square projection of the hidden state
        {**LINEAR, "name": "linear, 1 token", "tokens": 1, "n": 2560, "k": 2560, "out": "bf16"},
        # a batch of eight sequences through the widest projection
        {**LINEAR, "name": "linear, 8 tokens", "tokens": 8, "n": 10240, "k": 2560, "out": "fp32"},
        # a draft head's own vocabulary projection, one sequence
        {**LINEAR, "name": "linear, 1 token, vocabulary", "tokens": 1, "n": 248320, "k": 2560, "out": "fp32"},
        # a prefill chunk, added to the residual stream
        {**LINEAR, "name": "linear, 512 tokens", "tokens": 512, "n": 10240, "k": 2560, "residual": "bf16",
         "out": "bf16"},
        # an adapter of odd width inside wider rows
        {**LINEAR, "name": "odd linear, 77 tokens", "tokens": 77, "n": 1003, "k": 1152, "group": 64, "strided": True,
         "bias": "fp32", "activation": "gelu", "residual": "fp16", "out": "fp16"},
        # one drafted token's experts: gate and up
        {**GROUPED, "name": "grouped gate/up, 1 token", "tokens": 1, "n": 1280, "k": 2560, "down": False,
         "out": "bf16"},
        # a serving batch's down products, weighted and back in the tokens' order
        {**GROUPED, "name": "grouped down, 64 tokens", "tokens": 64, "n": 2560, "k": 640, "down": True,
         "out": "fp32"},
        # a prefill chunk's gate and up, many experts with few rows each
        {**GROUPED, "name": "grouped gate/up, 512 tokens", "tokens": 512, "n": 1280, "k": 2560, "down": False,
         "out": "bf16"},
        # a long prompt in one pass
        {**GROUPED, "name": "grouped gate/up, 8192 tokens", "tokens": 8192, "n": 1280, "k": 2560, "down": False,
         "out": "bf16"},
        # one chat stream with three drafted tokens
        {**VERIFY, "name": "verify, 1 sequence", "seqs": 1, "width": 3, "target": "fp32", "draft": "bf16",
         "mask": False},
        # a serving batch, some of its answers held to a grammar
        {**VERIFY, "name": "verify, 64 sequences", "seqs": 64, "width": 3, "target": "fp32", "draft": "fp32",
         "mask": True},
        # tokens drafted by lookup (no probabilities of their own), a small odd vocabulary in padded rows
        {**VERIFY, "name": "odd verify, 33 sequences", "seqs": 33, "width": 7, "vocab": 32003, "target": "fp16",
         "draft": "none", "mask": True, "strided": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "grouped", "verify"])
    out = rng.choice(["bf16", "fp16", "fp32"])
    if op == "linear":
        group = rng.choice([64, 128])
        tokens = _log(rng, 1, 8192)
        k = group * _log(rng, 1, 10240 // group)
        n = _log(rng, 33, 65536)
        # no more products, outputs or weights than a prefill chunk of 8192 tokens has
        n = max(1, min(n, 8192 * 10240 * 640 // (tokens * k), 8192 * 10240 // tokens))
        return {"op": op, "tokens": tokens, "n": n, "k": k, "group": group, "strided": rng.random() < 0.3,
                "bias": rng.choice(["none", "bf16", "fp32"]),
                "activation": rng.choice(["none", "silu", "gelu", "relu"]),
                "residual": rng.choice(["none", "bf16", "fp16", "fp32"]), "out": out}
    if op == "grouped":
        group = rng.choice([64, 128])
        experts = _log(rng, 1, 512)
        top_k = rng.randint(1, min(10, experts))
        tokens = _log(rng, 1, 4096)
        k = group * _log(rng, 1, 2560 // group)
        n = _log(rng, 33, 2560)
        return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "n": n, "k": k, "group": group,
                "down": rng.random() < 0.5, "bias": rng.choice(["none", "none", "bf16", "fp32"]),
                "activation": rng.choice(["none", "none", "silu"]), "out": out}
    width = rng.randint(0, 8)
    vocab = _log(rng, 1000, 248320)
    return {"op": op, "seqs": min(_log(rng, 1, 256), max(1, 64 * 7 * 248320 // ((2 * width + 1) * vocab))),
            "width": width, "vocab": vocab, "target": rng.choice(["bf16", "fp16", "fp32"]),
            "draft": rng.choice(["none", "bf16", "fp16", "fp32"]), "mask": rng.random() < 0.5,
            "strided": rng.random() < 0.3}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _wide(t, extra):
    """The same values inside rows that are `extra` elements longer."""
    wide = torch.zeros(t.shape[0], t.shape[1] + extra, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _weights(shape, k, group, normal, g):
    """Codes and scales of matrices [*shape, k] whose products with unit activations have about unit size."""
    packed = torch.randint(-2**31, 2**31 - 1, (*shape, k // 8), dtype=torch.int32, device="cuda", generator=g)
    return packed, (normal(*shape, k // group).abs() * (0.27 / math.sqrt(k))).to(torch.bfloat16)


def _prepare_linear(case, g):
    tokens, n, k, group = case["tokens"], case["n"], case["k"], case["group"]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    s = {"group": group, "activation": case["activation"], "x": normal(tokens, k).to(torch.bfloat16)}
    s["packed"], s["scales"] = _weights((n,), k, group, normal, g)
    s["bias"] = None if case["bias"] == "none" else (normal(n) * 0.5).to(TYPES[case["bias"]])
    s["residual"] = None if case["residual"] == "none" else normal(tokens, n).to(TYPES[case["residual"]])
    s["out"] = torch.empty(tokens, n, dtype=TYPES[case["out"]], device="cuda")
    if case["strided"]:
        s["x"] = _wide(s["x"], 24)
        s["out"] = _wide(s["out"], 5)
        s["residual"] = None if s["residual"] is None else _wide(s["residual"], 11)
    if own:  # the layer that a program holds: its weights as they are
        from quantized_moe_router_amd.layer import Int4Linear
        s["layer"] = Int4Linear(s["packed"], s["scales"], group, bias=s["bias"], activation=s["activation"])
    return s


def _prepare_grouped(case, g):
    tokens, experts, top_k, n, k = (case[i] for i in ("tokens", "experts", "top_k", "n", "k"))

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    s = {"group": case["group"], "activation": case["activation"], "top_k": top_k, "down": case["down"]}
    s["packed"], s["scales"] = _weights((experts, n), k, case["group"], normal, g)
    s["bias"] = None if case["bias"] == "none" else (normal(experts, n) * 0.5).to(TYPES[case["bias"]])
    # the tables that the routing answers: some experts are asked for more often than others
    rank = torch.randperm(experts, device="cuda", generator=g).float() + 1
    noise = -torch.log(-torch.log(torch.rand(tokens, experts, device="cuda", generator=g).clamp(1e-9, 1 - 1e-7)))
    ids = torch.topk(noise - 0.6 * torch.log(rank), top_k, dim=1).indices.reshape(-1)
    s["slots"] = torch.sort(ids, stable=True).indices.to(torch.int32)
    s["offsets"] = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    s["offsets"][1:] = torch.cumsum(torch.bincount(ids, minlength=experts), 0)
    rows = tokens * top_k
    s["x"] = normal(rows if case["down"] else tokens, k).to(torch.bfloat16)
    s["weights"] = torch.softmax(normal(tokens, top_k), 1)
    s["out"] = torch.empty(rows, n, dtype=TYPES[case["out"]], device="cuda")
    if own:  # the experts that a program holds: their weights as they are
        from quantized_moe_router_amd.layer import Int4GroupedLinear
        s["layer"] = Int4GroupedLinear(s["packed"], s["scales"], s["group"], bias=s["bias"],
                                       activation=s["activation"])
    return s


def _prepare_verify(case, g):
    seqs, width, vocab = case["seqs"], case["width"], case["vocab"]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    # the draft head is of the target's mind about most tokens
    target = normal(seqs, width + 1, vocab) * 2.5
    target[:, :, :32] += 6 * uniform(seqs, width + 1, 32)
    draft = target[:, :width] + 0.4 * normal(seqs, width, vocab)
    s = {"width": width, "vocab": vocab}
    s["temperature"] = 0.5 + uniform(seqs)
    s["temperature"][1::4] = 0.0   # greedy sequences
    s["lengths"] = torch.randint(0, width + 1, (seqs,), dtype=torch.int32, device="cuda", generator=g)
    s["lengths"][::2] = width      # half of the sequences have all their drafts
    gumbel = -torch.log(-torch.log(uniform(seqs, width, vocab).clamp(1e-9, 1 - 1e-7)))
    s["drafted"] = (draft + gumbel).argmax(2).to(torch.int32)
    s["drafted"][1::4] = draft[1::4].argmax(2).to(torch.int32)
    if case["draft"] == "none":    # a lookup finds the target's favourite more often than not
        best = target[:, :width].argmax(2).to(torch.int32)
        s["drafted"] = torch.where(uniform(seqs, width) < 0.7, best, s["drafted"])
    if case["mask"]:               # a grammar allows few tokens, in a dead end none
        banned = uniform(seqs, 1, vocab) < 0.9
        banned[::2] = False
        banned[7::16] = True
        target.masked_fill_(banned, -math.inf)
        draft.masked_fill_(banned, -math.inf)
    s["coins"], s["picks"] = uniform(seqs, width), uniform(seqs)
    s["target"] = target.view(-1, vocab).to(TYPES[case["target"]])
    s["draft"] = None if case["draft"] == "none" else draft.reshape(-1, vocab).to(TYPES[case["draft"]])
    if case["strided"]:
        s["target"] = _wide(s["target"], 29)
        s["draft"] = None if s["draft"] is None else _wide(s["draft"], 3)
    if own:  # what a program holds over its steps
        from quantized_moe_router_amd.layer import DraftVerifier
        s["verifier"] = DraftVerifier(vocab, temperature=s["temperature"])
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"linear": _prepare_linear, "grouped": _prepare_grouped, "verify": _prepare_verify}[case["op"]](case, g)
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
    return torch.clamp(y, min=0) if kind == "relu" else y


def _matrix(packed, scales, group):
    """fp32 matrices from their codes (8 a word, stored + 8) and a scale for every `group` inputs."""
    shifts = torch.arange(0, 32, 4, dtype=torch.int32, device=packed.device)
    codes = (((packed.unsqueeze(-1) >> shifts) & 15) - 8).float()
    w = codes.view(*packed.shape[:-1], -1, group) * scales.float().unsqueeze(-1)
    return w.view(*packed.shape[:-1], -1)


def _linear(s):
    y = s["x"].float() @ _matrix(s["packed"], s["scales"], s["group"]).T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _activate(y, s["activation"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["out"].dtype)


def _grouped(s):
    """Blocks of b sorted rows of one expert, as many as there can be, each with its expert's matrix."""
    experts, rows = s["packed"].shape[0], s["slots"].shape[0]
    b = 1
    if rows > experts:
        b = min(128, 1 << (rows // experts).bit_length())
    blocks = (rows + (b - 1) * min(experts, rows)) // b
    offsets = s["offsets"].long()
    tiles = torch.cumsum((offsets[1:] - offsets[:-1] + b - 1) // b, 0)   # blocks up to and with each expert
    at = torch.arange(blocks, device=tiles.device)
    e = torch.searchsorted(tiles, at, right=True).clamp(max=experts - 1)
    start = offsets[e] + (at - torch.where(e > 0, tiles[e - 1], 0)) * b
    place = start.unsqueeze(1) + torch.arange(b, device=at.device)
    live = place < offsets[e + 1].unsqueeze(1)
    place = torch.where(live, place, 0)
    slot = s["slots"].long()[place]
    x = s["x"][place if s["down"] else slot // s["top_k"]].float()
    if blocks >= experts:
        w = _matrix(s["packed"], s["scales"], s["group"])[e]
    else:
        w = _matrix(s["packed"][e], s["scales"][e], s["group"])
    y = torch.bmm(x, w.transpose(1, 2))
    if s["bias"] is not None:
        y = y + s["bias"][e].float().unsqueeze(1)
    y = _activate(y, s["activation"])
    if s["down"]:
        y = y * s["weights"].view(-1)[slot].unsqueeze(2)
    y = y.to(s["out"].dtype)
    # what is no row of its block goes to a row behind the last
    to = torch.where(live, slot if s["down"] else place, rows).view(-1)
    out = torch.empty(rows + 1, y.shape[2], dtype=y.dtype, device=y.device)
    out[to] = y.view(-1, y.shape[2])
    return out[:rows]


def _softmax(l):
    """In 64 bits; a row without any finite logit has no probabilities, and gets zeros."""
    l = l.double()
    e = torch.exp(l - l.amax(-1, keepdim=True))
    e = torch.where(torch.isnan(e), 0.0, e)
    return e / e.sum(-1, keepdim=True).clamp(min=1e-300)


def _verify(s):
    width, vocab = s["width"], s["vocab"]
    target = s["target"].view(-1, width + 1, vocab) if s["target"].is_contiguous() else \
        s["target"].unflatten(0, (-1, width + 1))
    seqs, dev = target.shape[0], target.device
    p = _softmax(target)
    drafted = s["drafted"].long()
    q = torch.zeros(seqs, width + 1, vocab, dtype=torch.float64, device=dev)
    if s["draft"] is not None:
        q[:, :width] = _softmax(s["draft"].unflatten(0, (seqs, width)) if width else q[:, :0])
    else:
        q[:, :width].scatter_(2, drafted.unsqueeze(2), 1.0)
    value, best = target.max(2)   # greedy: the first of the largest logits, if there is any
    first = (target == value.unsqueeze(2)).int().argmax(2)
    best = torch.where(torch.isneginf(value), -1, first)
    greedy = s["temperature"] <= 0
    px = p[:, :width].gather(2, drafted.unsqueeze(2)).squeeze(2)
    qx = q[:, :width].gather(2, drafted.unsqueeze(2)).squeeze(2)
    at = torch.arange(width + 1, device=dev)
    good = torch.where(greedy.unsqueeze(1), drafted == best[:, :width], s["coins"].double() * qx < px)
    good = good & (at[:width] < s["lengths"].unsqueeze(1))
    accepted = torch.cumprod(good.int(), 1).sum(1)
    # behind the last accepted draft: from what the target has over the draft,
    # or from the target where no draft was left
    row = torch.arange(seqs, device=dev)
    p, q, best = p[row, accepted], q[row, accepted], best[row, accepted]
    q = torch.where((accepted < s["lengths"]).unsqueeze(1), q, 0.0)
    r = torch.clamp(p - q, min=0)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, p)
    c = torch.cumsum(r, 1)
    over = c > (s["picks"].double() * c[:, -1]).unsqueeze(1)
    token = torch.where(over.any(1), over.int().argmax(1), -1)
    token = torch.where(greedy, best, token).unsqueeze(1)
    padded = torch.nn.functional.pad(drafted, (0, 1))
    tokens = torch.where(at < accepted.unsqueeze(1), padded, torch.where(at == accepted.unsqueeze(1), token, -1))
    return {"tokens": tokens.int(), "accepted": accepted.int()}


def run(state):
    op = state["op"]
    if own:
        if op == "linear":
            return state["layer"].forward(state["x"], residual=state["residual"], out=state["out"])
        if op == "grouped":
            if state["down"]:
                return state["layer"].forward(state["x"], state["offsets"], scatter=state["slots"],
                                              row_weights=state["weights"], out=state["out"])
            return state["layer"].forward(state["x"], state["offsets"], gather=state["slots"],
                                          gather_div=state["top_k"], out=state["out"])
        tokens, accepted = state["verifier"].verify(state["target"], state["drafted"], state["coins"], state["picks"],
                                                    draft=state["draft"], lengths=state["lengths"])
        return {"tokens": tokens, "accepted": accepted}
    return {"linear": _linear, "grouped": _grouped, "verify": _verify}[op](state)


def work(case):
    if case["op"] == "verify":
        seqs, width, vocab = case["seqs"], case["width"], case["vocab"]
        rows = seqs * ((width + 1) * BYTES[case["target"]] + width * BYTES[case["draft"]])
        logits = seqs * (width + 1 + (0 if case["draft"] == "none" else width)) * vocab
        return {"bytes": rows * vocab + 4 * seqs * (4 * width + 5), "flops": 4 * logits}
    n, k = case["n"], case["k"]
    matrix = n * k // 2 + 2 * n * (k // case["group"])
    if case["op"] == "linear":
        t = case["tokens"]
        return {"bytes": matrix + 2 * t * k + n * BYTES[case["bias"]]
                + t * n * (BYTES[case["residual"]] + BYTES[case["out"]]),
                "flops": 2 * t * n * k}
    rows, experts = case["tokens"] * case["top_k"], case["experts"]
    # the experts that the rows reach, with the popularity that the routing has
    popular = (np.arange(experts) + 1.0) ** -0.6
    reached = (1 - (1 - np.minimum(1.0, case["top_k"] * popular / popular.sum())) ** case["tokens"]).sum()
    return {"bytes": int(reached * (matrix + n * BYTES[case["bias"]])) + 2 * k * (rows if case["down"] else case["tokens"])
            + rows * (n * BYTES[case["out"]] + 4 + (4 if case["down"] else 0)) + 4 * (experts + 1),
            "flops": 2 * rows * n * k}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_activation(y, kind):
    if kind == "silu":
        return y * torch.sigmoid(y)
    if kind == "gelu":
        return y * (torch.special.erfc(-y / math.sqrt(2.0)) / 2)
    return torch.maximum(y, torch.zeros_like(y)) if kind == "relu" else y


def _exact_product(x, packed, scales, group):
    """x W^T, group by group, the scale outside the group's sum."""
    n, words = packed.shape
    y = torch.zeros(x.shape[0], n, dtype=torch.float64, device="cuda")
    per = group // 8
    for at in range(0, words, per):
        block = packed[:, at:at + per]
        q = torch.empty(n, group, dtype=torch.float64, device="cuda")
        for j in range(8):
            q[:, j::8] = (torch.div(block.long() % 2**32, 16**j, rounding_mode="floor") % 16).double() - 8.0
        y += torch.mm(x[:, 8 * at:8 * at + group].contiguous(), q.t().contiguous()) * scales[:, at // per].double()
    return y


def _exact_linear(case, s):
    y = _exact_product(s["x"].double(), s["packed"], s["scales"], s["group"])
    if s["bias"] is not None:
        y += s["bias"].double()
    y = _exact_activation(y, case["activation"])
    if s["residual"] is not None:
        y += s["residual"].double()
    return y


def _exact_grouped(case, s):
    offsets, slots = s["offsets"].tolist(), s["slots"].long()
    out = torch.zeros(slots.shape[0], case["n"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        begin, end = offsets[e], offsets[e + 1]
        if begin == end:
            continue
        mine = slots[begin:end]
        x = s["x"][begin:end] if case["down"] else s["x"][torch.div(mine, case["top_k"], rounding_mode="floor")]
        y = _exact_product(x.double(), s["packed"][e], s["scales"][e], s["group"])
        if s["bias"] is not None:
            y += s["bias"][e].double()
        y = _exact_activation(y, case["activation"])
        if case["down"]:
            out[mine] = y * s["weights"].double().view(-1)[mine].unsqueeze(1)
        else:
            out[begin:end] = y
    return out


def _exact_probabilities(l):
    top = l.max()
    if top == -np.inf:
        return np.zeros_like(l)
    e = np.exp(l - top)
    return e / e.sum()


def _exact_verify(case, s):
    seqs, width, vocab = case["seqs"], case["width"], case["vocab"]
    host = {k: v.float().cpu().numpy() if v.is_floating_point() else v.cpu().numpy()
            for k, v in s.items() if isinstance(v, torch.Tensor)}
    tokens, accepted = np.full((seqs, width + 1), -1, np.int32), np.zeros(seqs, np.int32)
    for b in range(seqs):
        n, drafts = 0, int(host["lengths"][b])
        while True:
            row = host["target"][b * (width + 1) + n].astype(np.float64)
            greedy = host["temperature"][b] <= 0
            x = int(host["drafted"][b, n]) if n < drafts else -1
            if greedy:
                best = int(row.argmax()) if row.max() > -np.inf else -1
                if n < drafts and x == best:
                    tokens[b, n] = x
                    n += 1
                    continue
                tokens[b, n] = best
                break
            p = _exact_probabilities(row)
            q = np.zeros(vocab)
            if n < drafts:
                if "draft" in host:
                    q = _exact_probabilities(host["draft"][b * width + n].astype(np.float64))
                else:
                    q[x] = 1.0
                if float(host["coins"][b, n]) * q[x] < p[x]:
                    tokens[b, n] = x
                    n += 1
                    continue
            r = np.maximum(p - q, 0.0)
            c = np.cumsum(r if r.sum() > 0 else p)
            if c[-1] > 0:
                tokens[b, n] = int(np.searchsorted(c, float(host["picks"][b]) * c[-1], side="right"))
            break
        accepted[b] = n
    return {"tokens": tokens, "accepted": accepted}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_linear(case, s)
    return _exact_grouped(case, s) if case["op"] == "grouped" else _exact_verify(case, s)
