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
