"""Convenience wrapper: a resident MoE INT4 layer on the GPU.

Allocates outputs and a zero-filled workspace with torch and calls the C ABI;
no arithmetic of the layer happens here.
"""
from __future__ import annotations

import torch

from . import _binding as B


class MoeInt4Layer:
    """Holds device tensors of one layer (keys as produced by synth.to_device /
    synth.device_weights) and runs the library's entry points on them."""

    def __init__(self, weights: dict, top_k: int, group: int = 128, shared: dict | None = None):
        self.w = weights
        self.top_k = int(top_k)
        self.group = int(group)
        E, H = weights["router_w"].shape
        self.E, self.H = int(E), int(H)
        self.I = int(weights["w2_packed"].shape[2] * 8)
        self.shared = shared
        self._shared_c = B.make_shared(shared)
        self._ws = {}

    def shape(self, tokens: int) -> B.MoeShape:
        return B.make_shape(tokens, self.H, self.E, self.I, self.top_k, self.group)

    def workspace(self, tokens: int, device=None) -> torch.Tensor:
        key = (tokens, device)
        if key not in self._ws:
            self._ws[key] = B.new_workspace(self.shape(tokens), self._shared_c,
                                            device=device or self.w["router_w"].device)
        return self._ws[key]

    def workspaces(self) -> list:
        return list(self._ws.values())

    def forward(self, x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        T = x.shape[0]
        if out is None:
            out = torch.empty(T, self.H, dtype=torch.int16, device=x.device)
        w = self.w
        B.moe_int4_forward(x, w["router_w"], w["w13_packed"], w["w13_scales"], w["w2_packed"],
                           w["w2_scales"], self.top_k, out, self.shape(T), self._shared_c,
                           self.workspace(T), stream)
        return out

    def route(self, x: torch.Tensor, stream=None) -> dict:
        T, dev = x.shape[0], x.device
        r = {
            "ids": torch.empty(T, self.top_k, dtype=torch.int32, device=dev),
            "weights": torch.empty(T, self.top_k, dtype=torch.float32, device=dev),
            "counts": torch.empty(self.E, dtype=torch.int32, device=dev),
            "offsets": torch.empty(self.E + 1, dtype=torch.int32, device=dev),
            "sorted_slots": torch.empty(max(T * self.top_k, 1), dtype=torch.int32, device=dev),
        }
        B.moe_int4_route(x, self.w["router_w"], self.shape(T), r["ids"], r["weights"], r["counts"],
                         r["offsets"], r["sorted_slots"], self.workspace(T), stream)
        return r

    def experts(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        T = x.shape[0]
        if out is None:
            out = torch.empty(T, self.H, dtype=torch.int16, device=x.device)
        w = self.w
        B.moe_int4_experts(x, ids, weights, w["w13_packed"], w["w13_scales"], w["w2_packed"],
                           w["w2_scales"], self.shape(T), self._shared_c, out, self.workspace(T), stream)
        return out


class Int8Linear:
    """A resident INT8 W8A16 linear layer (hyper-connection mixer, lm_head)
    with its bias and activation: packed int32 [n, k/4], scales bf16
    [n, k/group], bias [n] in bf16, fp16 or fp32."""

    def __init__(self, packed: torch.Tensor, scales: torch.Tensor, group: int,
                 bias: torch.Tensor | None = None, activation: str = "none"):
        if packed.dim() != 2 or packed.dtype != torch.int32 or not packed.is_contiguous():
            raise ValueError(f"packed is {packed.dtype} {tuple(packed.shape)}, expected contiguous int32 [n, k/4]")
        self.n, self.k, self.group = int(packed.shape[0]), 4 * int(packed.shape[1]), int(group)
        if group <= 0 or self.k % group or tuple(scales.shape) != (self.n, self.k // group) \
                or B.type_code(scales.dtype) != B.TYPE_BF16 or not scales.is_contiguous():
            raise ValueError(f"scales is {scales.dtype} {tuple(scales.shape)}, expected contiguous bfloat16 "
                             f"({self.n}, {self.k} / {group})")
        if activation not in B.ACTIVATIONS:
            raise ValueError(f"activation {activation!r} is none of {', '.join(B.ACTIVATIONS)}")
        self.packed, self.scales, self.bias, self.activation = packed, scales, bias, activation
        self._need = {}

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """residual + act(x W^T + bias) on torch's current stream of x's
        device; x bf16 [tokens, k].  out may be the residual."""
        tokens = x.shape[0]
        if out is None:
            out = torch.empty(tokens, self.n, dtype=out_dtype, device=x.device)
        need = self._need.get(tokens)
        if need is None:
            need = self._need[tokens] = B.moe_int8_linear_fused_workspace_bytes(tokens, self.n, self.k, self.group)
        # taken anew for every call: the allocator orders it by stream, and
        # two calls in flight never share one
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
        B.int8_linear_fused(x, self.packed, self.scales, tokens, self.n, self.k, self.group, out, self.bias, residual,
                            self.activation, workspace)
        return out


class LogitsRules:
    """The rules of a serving batch on its logits: penalties for repeated
    tokens, biases, a grammar mask and a temperature per row.  Holds the
    caller's device tables as they are; what a program writes into them
    between calls (a new token, a length, a mask) is in force at the next.

      history int32 [rows, width], history_lengths, prompt_lengths int32 [rows]
      repetition, frequency, presence, temperature  float32 [rows]
      bias_ids int32, bias_values float32 [rows, width], bias_lengths int32 [rows]
      mask int32 [rows, ceil(vocab / 32)] (or one such row for all)

    include/moe_int4.h states what each does; any may be None."""

    def __init__(self, vocab: int, history=None, history_lengths=None, prompt_lengths=None, repetition=None,
                 frequency=None, presence=None, bias_ids=None, bias_values=None, bias_lengths=None,
                 temperature=None, mask=None):
        self.vocab = int(vocab)
        if history is None:
            for name, t in (("history_lengths", history_lengths), ("prompt_lengths", prompt_lengths),
                            ("repetition", repetition), ("frequency", frequency), ("presence", presence)):
                if t is not None:
                    raise ValueError(f"{name} is given without history")
        if (bias_ids is None) != (bias_values is None) or (bias_ids is None and bias_lengths is not None):
            raise ValueError("bias_ids and bias_values go together, bias_lengths with them")
        words = (self.vocab + 31) // 32
        if mask is not None and mask.dim() == 1:
            mask = mask.unsqueeze(0)
        shared_mask = mask is not None and mask.shape[0] == 1
        vectors = {"history_lengths": (history_lengths, torch.int32), "prompt_lengths": (prompt_lengths, torch.int32),
                   "repetition": (repetition, torch.float32), "frequency": (frequency, torch.float32),
                   "presence": (presence, torch.float32), "bias_lengths": (bias_lengths, torch.int32),
                   "temperature": (temperature, torch.float32)}
        matrices = {"history": (history, torch.int32), "bias_ids": (bias_ids, torch.int32),
                    "bias_values": (bias_values, torch.float32)}
        if not shared_mask:
            matrices["mask"] = (mask, torch.int32)
        given = {k: t for k, (t, _) in {**vectors, **matrices}.items() if t is not None}
        # the rows that every table has: None without any table by rows
        self.rows = next((int(t.shape[0]) for t in given.values()), None)
        c = B.MoeLogitsRules()
        for name, (t, dtype) in {**vectors, **matrices, "mask": (mask, torch.int32)}.items():
            if t is None:
                continue
            dims = 1 if name in vectors else 2
            if t.dtype != dtype or t.dim() != dims or (name in given and t.shape[0] != self.rows):
                raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}, expected {dtype} of {dims} dimension(s) "
                                 f"and {self.rows} rows")
            if t.shape[-1] > 1 and t.stride(-1) != 1:
                raise ValueError(f"{name}: the elements of a row must be consecutive")
            setattr(c, name, t.data_ptr())
        if history is not None:
            c.history_stride, c.history_width = history.stride(0), history.shape[1]
        if bias_ids is not None:
            if bias_ids.shape != bias_values.shape or (self.rows > 1 and bias_ids.stride(0) != bias_values.stride(0)):
                raise ValueError("bias_ids and bias_values differ in shape or row stride")
            c.bias_stride, c.bias_width = bias_ids.stride(0), bias_ids.shape[1]
        if mask is not None:
            if mask.shape[1] < words:
                raise ValueError(f"mask has {mask.shape[1]} words a row, {self.vocab} tokens need {words}")
            c.mask_stride = 0 if shared_mask else mask.stride(0)
        self._tables = {**given, **({} if mask is None else {"mask": mask})}
        self._index = None   # of the GPU that holds the tables
        for name, t in self._tables.items():
            self._index = B.device_index(t, name, self._index)
        self._c = c

    def apply(self, logits: torch.Tensor, out: torch.Tensor | None = None,
              out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
        """The rules applied to logits [rows, vocab] on torch's current stream
        of their device; the first rows of the tables where there are fewer
        logits than table rows.  out may be logits (in place)."""
        if logits.dim() != 2 or logits.shape[1] != self.vocab or (self.rows is not None
                                                                  and logits.shape[0] > self.rows):
            raise ValueError(f"logits is {tuple(logits.shape)}, expected at most {self.rows} rows of {self.vocab}")
        B.device_index(logits, "logits", self._index)
        if out is None:
            out = torch.empty(logits.shape, dtype=out_dtype, device=logits.device)
        B.moe_int4_logits_process(logits, self._c, out)
        return out


class Int4Linear:
    """A resident INT4 W4A16 linear layer (a draft head's projection, weights
    as moe_int4_quantize writes them) with its bias and activation: packed
    int32 [n, k/8], scales bf16 [n, k/group], bias [n] in bf16, fp16 or fp32."""

    def __init__(self, packed: torch.Tensor, scales: torch.Tensor, group: int = 128,
                 bias: torch.Tensor | None = None, activation: str = "none"):
        if packed.dim() != 2:
            raise ValueError(f"packed is {packed.dtype} {tuple(packed.shape)}, expected contiguous int32 [n, k/8]")
        self.n, self.k, self.group = int(packed.shape[0]), 8 * int(packed.shape[1]), int(group)
        B.check_int4_weights(packed, scales, (self.n,), self.k, self.group)
        if activation not in B.ACTIVATIONS:
            raise ValueError(f"activation {activation!r} is none of {', '.join(B.ACTIVATIONS)}")
        self.packed, self.scales, self.bias, self.activation = packed, scales, bias, activation
        self._need = {}

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """residual + act(x W^T + bias) on torch's current stream of x's
        device; x bf16 [tokens, k].  out may be the residual."""
        tokens = x.shape[0]
        if out is None:
            out = torch.empty(tokens, self.n, dtype=out_dtype, device=x.device)
        need = self._need.get(tokens)
        if need is None:
            need = self._need[tokens] = B.moe_int4_linear_workspace_bytes(tokens, self.n, self.k, self.group)
        # taken anew for every call, as in Int8Linear
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
        B.int4_linear(x, self.packed, self.scales, tokens, self.n, self.k, self.group, out, self.bias, residual,
                      self.activation, workspace)
        return out


class Int4GroupedLinear:
    """One product of resident INT4 experts over rows grouped by expert, as
    MoeInt4Layer.route answers them: packed int32 [experts, n, k/8], scales
    bf16 [experts, n, k/group], bias [experts, n] in bf16, fp16 or fp32."""

    def __init__(self, packed: torch.Tensor, scales: torch.Tensor, group: int = 128,
                 bias: torch.Tensor | None = None, activation: str = "none"):
        if packed.dim() != 3:
            raise ValueError(f"packed is {packed.dtype} {tuple(packed.shape)}, expected contiguous int32 "
                             "[experts, n, k/8]")
        self.experts, self.n, self.k = int(packed.shape[0]), int(packed.shape[1]), 8 * int(packed.shape[2])
        self.group = int(group)
        B.check_int4_weights(packed, scales, (self.experts, self.n), self.k, self.group)
        if activation not in B.ACTIVATIONS:
            raise ValueError(f"activation {activation!r} is none of {', '.join(B.ACTIVATIONS)}")
        self.packed, self.scales, self.bias, self.activation = packed, scales, bias, activation
        self._need = {}

    def forward(self, x: torch.Tensor, offsets: torch.Tensor, gather: torch.Tensor | None = None,
                gather_div: int = 1, scatter: torch.Tensor | None = None, row_weights: torch.Tensor | None = None,
                residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """residual + row_weights act(x W_e^T + bias_e) on torch's current
        stream of x's device; x bf16 [rows, k].  offsets int32 [experts + 1];
        place p of expert e (offsets[e] <= p < offsets[e + 1]) reads row
        gather[p] // gather_div of x and writes row scatter[p] of out (row p
        without the table), scaled by that row's entry of row_weights.  With r
        = MoeInt4Layer.route(x): a gate/up product takes gather =
        r["sorted_slots"] and gather_div = top_k, a down product scatter =
        r["sorted_slots"] and row_weights = r["weights"].  A new out has as
        many rows as there are places; rows that no place writes hold zeros
        where it is made here, and stay as they were in a given one."""
        if offsets.shape != (self.experts + 1,):
            raise ValueError(f"offsets is {tuple(offsets.shape)}, expected ({self.experts + 1},)")
        table = gather if gather is not None else scatter
        places = x.shape[0] if table is None else table.numel()
        if out is None:
            out = torch.zeros(places, self.n, dtype=out_dtype, device=x.device)
        c = B.make_groups(x.shape[0], out.shape[0], places, offsets, gather, gather_div, scatter, row_weights)
        index = B.device_index(x, "x")
        for name, t in (("offsets", offsets), ("gather", gather), ("scatter", scatter), ("row_weights", row_weights)):
            if t is not None:
                B.device_index(t, name, index)
        key = (places, c.x_rows, gather is None)
        need = self._need.get(key)
        if need is None:
            need = self._need[key] = B.moe_int4_grouped_linear_workspace_bytes(c, self.n, self.k, self.group)
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
        B.int4_grouped_linear(x, self.packed, self.scales, c, self.n, self.k, self.group, out, self.bias, residual,
                              self.activation, workspace)
        return out


class DraftVerifier:
    """Verifies the drafted tokens of a batch against the target's logits, and
    draws each sequence's next token.  temperature float32 [seqs] is the table
    that LogitsRules takes: sequences without one above zero are greedy."""

    def __init__(self, vocab: int, temperature: torch.Tensor | None = None):
        self.vocab = int(vocab)
        if temperature is not None and (temperature.dtype != torch.float32 or temperature.dim() != 1
                                        or not temperature.is_contiguous()):
            raise ValueError(f"temperature is {temperature.dtype} {tuple(temperature.shape)}, expected contiguous "
                             "float32 [seqs]")
        self.temperature = temperature
        self._need = {}

    def verify(self, target: torch.Tensor, drafted: torch.Tensor, coins: torch.Tensor, picks: torch.Tensor,
               draft: torch.Tensor | None = None, lengths: torch.Tensor | None = None,
               tokens: torch.Tensor | None = None, accepted: torch.Tensor | None = None) -> tuple:
        """target [seqs * (width + 1), vocab] and draft [seqs * width, vocab]
        (None: drafts found by lookup) logits in bf16, fp16 or fp32, as
        LogitsRules leaves them; drafted int32 [seqs, width], of which lengths
        int32 [seqs] count; coins float32 [seqs, width] and picks float32
        [seqs] random numbers in [0, 1).  Answers (tokens int32 [seqs, width +
        1]: the accepted drafts, the next token, -1 behind it; accepted int32
        [seqs])."""
        if drafted.dim() != 2:
            raise ValueError(f"drafted is {tuple(drafted.shape)}, expected [seqs, width]")
        seqs, width = drafted.shape
        if self.temperature is not None and self.temperature.shape[0] < seqs:
            raise ValueError(f"temperature has {self.temperature.shape[0]} sequences, drafted {seqs}")
        index = B.device_index(target, "target")
        c = B.MoeDrafts()
        for name, t, dtype, shape in (("tokens", drafted, torch.int32, (seqs, width)),
                                      ("lengths", lengths, torch.int32, (seqs,)),
                                      ("coins", coins, torch.float32, (seqs, width)),
                                      ("picks", picks, torch.float32, (seqs,))):
            if t is None:
                continue
            if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
                raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}, expected contiguous {dtype} {shape}")
            B.device_index(t, name, index)
            setattr(c, name, t.data_ptr())
        if self.temperature is not None:
            B.device_index(self.temperature, "temperature", index)
            c.temperature = self.temperature.data_ptr()
        c.target_stride = B.row_stride(target, "target", seqs * (width + 1), self.vocab)
        c.target, c.target_type = target.data_ptr(), B.type_code(target.dtype)
        if draft is not None:
            c.draft_stride = B.row_stride(draft, "draft", seqs * width, self.vocab)
            c.draft, c.draft_type = draft.data_ptr(), B.type_code(draft.dtype)
            B.device_index(draft, "draft", index)
        c.seqs, c.width, c.vocab = seqs, width, self.vocab
        if tokens is None:
            tokens = torch.empty(seqs, width + 1, dtype=torch.int32, device=target.device)
        if accepted is None:
            accepted = torch.empty(seqs, dtype=torch.int32, device=target.device)
        need = self._need.get((seqs, width))
        if need is None:
            need = self._need[seqs, width] = B.moe_int4_verify_drafts_workspace_bytes(seqs, width, self.vocab)
        workspace = torch.empty(need, dtype=torch.uint8, device=target.device)
        B.moe_int4_verify_drafts(c, accepted, tokens, workspace)
        return tokens, accepted
