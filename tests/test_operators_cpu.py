"""Argument checks of moe_int8_linear_fused and moe_int4_logits_process, and
of the classes over them: every refusal happens on the host, before anything
touches a device, so none of these needs a GPU."""
import ctypes

import pytest
import torch

from quantized_moe_router_amd import _binding as B
from quantized_moe_router_amd.layer import Int8Linear, LogitsRules

FAKE = 1 << 24   # never dereferenced
BF16, F16, F32 = B.TYPE_BF16, B.TYPE_F16, B.TYPE_F32


def error():
    return B.lib().moe_int4_last_error().decode()


def no_device():
    return not torch.cuda.is_available()


def fused(tokens=4, n=320, k=2560, group=64, x=FAKE, xs=2560, wp=FAKE * 2, sc=FAKE * 3, out=FAKE * 4, ot=BF16,
          os_=320, ws=FAKE * 8, wb=1 << 40, epi=None, stream=None):
    e = None if epi is None else B.MoeInt8Epilogue(**epi)
    return B.lib().moe_int8_linear_fused(x, xs, wp, sc, tokens, n, k, group, ctypes.byref(e) if e else None, out, ot,
                                         os_, ws, wb, stream)


FINE = "a valid call"   # stops only where there is no gfx950 device; not made where there is one


@pytest.mark.parametrize("kw,code,msg", [
    (dict(group=32), B.EINVAL, "group"),
    (dict(k=2500, xs=2500), B.EINVAL, "k="),
    (dict(n=0), B.EINVAL, "n="),
    (dict(tokens=-1), B.EINVAL, "tokens"),
    (dict(tokens=1 << 20, n=1 << 12), B.EINVAL, "2^31"),
    (dict(x=None), B.EINVAL, "x is NULL"),
    (dict(wp=None), B.EINVAL, "w_packed is NULL"),
    (dict(sc=None), B.EINVAL, "w_scales is NULL"),
    (dict(out=None), B.EINVAL, "out is NULL"),
    (dict(x=FAKE + 8), B.EALIGN, "x is not 16-byte"),
    (dict(out=FAKE * 4 + 1), B.EALIGN, "out is not aligned"),
    (dict(out=FAKE * 4 + 2, ot=F32), B.EALIGN, "out is not aligned"),
    (dict(ot=3), B.EINVAL, "out: type 3"),
    (dict(ot=-1), B.EINVAL, "out: type -1"),
    (dict(xs=2559), B.EINVAL, "x: stride"),
    (dict(xs=0), B.EINVAL, "x: stride"),
    (dict(xs=-2560), B.EINVAL, "x: stride"),
    (dict(xs=2564), B.EALIGN, "x: stride 2564"),
    (dict(os_=319), B.EINVAL, "out: stride"),
    (dict(os_=1 << 41), B.EINVAL, "out: stride"),
    (dict(out=FAKE), B.EINVAL, "out overlaps x"),
    (dict(out=FAKE + 2 * 3 * 2560 + 100), B.EINVAL, "out overlaps x"),
    (dict(out=FAKE * 2 + 1000), B.EINVAL, "out overlaps w_packed"),
    (dict(out=FAKE * 3 + 64), B.EINVAL, "out overlaps w_scales"),
    (dict(tokens=64, k=10240, xs=10240, n=96, os_=96, ws=FAKE * 4 + 64), B.EINVAL, "workspace overlaps"),
    (dict(tokens=64, k=10240, xs=10240, n=96, os_=96, ws=FAKE * 2 + 64), B.EINVAL, "workspace overlaps"),
    (dict(tokens=64, k=10240, xs=10240, n=96, os_=96, ws=FAKE * 3 + 64), B.EINVAL, "workspace overlaps"),
    (dict(epi=dict(activation=6)), B.EINVAL, "activation 6"),
    (dict(epi=dict(activation=-1)), B.EINVAL, "activation -1"),
    (dict(epi=dict(bias=FAKE * 5, bias_type=7)), B.EINVAL, "bias: type 7"),
    (dict(epi=dict(bias=FAKE * 5 + 2, bias_type=F32)), B.EALIGN, "bias is not aligned"),
    (dict(epi=dict(bias=FAKE * 4 + 64, bias_type=BF16)), B.EINVAL, "out overlaps bias"),
    (dict(epi=dict(residual=FAKE * 5, residual_type=-2, residual_stride=320)), B.EINVAL, "residual: type -2"),
    (dict(epi=dict(residual=FAKE * 5, residual_type=F32, residual_stride=0)), B.EINVAL, "residual: stride 0"),
    (dict(epi=dict(residual=FAKE * 4, residual_type=F16, residual_stride=320)), B.EINVAL, "out overlaps residual"),
    (dict(epi=dict(residual=FAKE * 4 + 320, residual_type=BF16, residual_stride=320)), B.EINVAL, "out overlaps residual"),
    (dict(tokens=64, k=10240, xs=10240, ws=None), B.EINVAL, "workspace is NULL"),
    (dict(tokens=64, k=10240, xs=10240, ws=FAKE * 8 + 4), B.EALIGN, "workspace is not"),
    (dict(tokens=64, k=10240, xs=10240, wb=1024), B.EWORKSPACE, "workspace has 1024"),
    # fine up to the device check
    (dict(), B.EDEVICE, FINE),
    (dict(tokens=1, xs=0, os_=0), B.EDEVICE, FINE),
    (dict(out=FAKE * 4 + 2), B.EDEVICE, FINE),
    (dict(xs=4096, out=FAKE + 2 * 2560, os_=4096), B.EDEVICE, FINE),   # column ranges of one matrix
    (dict(epi=dict(residual=FAKE * 4, residual_type=BF16, residual_stride=320)), B.EDEVICE, FINE),   # in place
    (dict(os_=640, epi=dict(residual=FAKE * 4 + 640, residual_type=BF16, residual_stride=640)), B.EDEVICE, FINE),
    (dict(epi=dict(residual=None, residual_type=99, bias_type=99)), B.EDEVICE, FINE),   # not read
])
def test_fused_checks(kw, code, msg):
    if msg is FINE:
        if no_device():
            assert fused(**kw) == B.EDEVICE
        return
    assert fused(**kw) == code and msg in error(), error()


def test_fused_zero_tokens_and_workspace_query():
    assert fused(tokens=0, x=None, out=None) == B.OK
    assert fused(tokens=0, group=3) == B.EINVAL
    b = ctypes.c_size_t(1)
    q = B.lib().moe_int8_linear_fused_workspace_bytes
    assert q(1, 248320, 2560, 128, ctypes.byref(b)) == 0 and b.value == 0
    assert q(512, 320, 10240, 64, ctypes.byref(b)) == 0 and b.value == 0   # K over waves, whose sums meet in LDS
    assert q(64, 320, 10240, 64, ctypes.byref(b)) == 0 and b.value > 0     # and over workgroups
    assert q(512, 320, 10240, 65, ctypes.byref(b)) == B.EINVAL
    assert q(512, 320, 10240, 64, None) == B.EINVAL


def logits(rows=4, vocab=1000, p=FAKE, t=BF16, s=1000, out=FAKE * 2, ot=F32, os_=1000, rules=True, **u):
    r = B.MoeLogitsRules(**u) if rules else None
    return B.lib().moe_int4_logits_process(p, t, s, rows, vocab, ctypes.byref(r) if r else None, out, ot, os_, None)


HIST = dict(history=FAKE * 3, history_width=10, history_stride=10)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(rows=-1), B.EINVAL, "rows"),
    (dict(rows=65537), B.EINVAL, "rows"),
    (dict(vocab=0), B.EINVAL, "vocab"),
    (dict(vocab=(1 << 24) + 1), B.EINVAL, "vocab"),
    (dict(rows=1 << 16, vocab=1 << 20, s=1 << 20, os_=1 << 20), B.EINVAL, "2^34"),
    (dict(rules=False), B.EINVAL, "rules is NULL"),
    (dict(p=None), B.EINVAL, "logits is NULL"),
    (dict(out=None), B.EINVAL, "out is NULL"),
    (dict(t=5), B.EINVAL, "logits: type 5"),
    (dict(ot=-1), B.EINVAL, "out: type -1"),
    (dict(p=FAKE + 1), B.EALIGN, "logits is not aligned"),
    (dict(out=FAKE * 2 + 2), B.EALIGN, "out is not aligned"),
    (dict(s=999), B.EINVAL, "logits: stride"),
    (dict(os_=-1000), B.EINVAL, "out: stride"),
    (dict(out=FAKE), B.EINVAL, "out overlaps logits"),                       # another type in place
    (dict(out=FAKE + 500, ot=BF16), B.EINVAL, "out overlaps logits"),
    (dict(history_width=-1), B.EINVAL, "history_width"),
    (dict(history_width=(1 << 24) + 1), B.EINVAL, "history_width"),
    (dict(bias_width=-1), B.EINVAL, "bias_width"),
    (dict(HIST, history_stride=9), B.EINVAL, "history: stride 9"),
    (dict(HIST, history=FAKE * 3 + 2), B.EALIGN, "history is not aligned"),
    (dict(HIST, repetition=FAKE * 4 + 1), B.EALIGN, "repetition is not aligned"),
    (dict(HIST, history_lengths=FAKE * 2 + 16), B.EINVAL, "out overlaps history_lengths"),
    (dict(HIST, history=FAKE * 2 + 16), B.EINVAL, "out overlaps history"),
    (dict(bias_ids=FAKE * 4, bias_width=3, bias_stride=3), B.EINVAL, "bias_values is NULL"),
    (dict(bias_values=FAKE * 4, bias_width=3, bias_stride=3), B.EINVAL, "bias_ids is NULL"),
    (dict(bias_ids=FAKE * 4, bias_values=FAKE * 5, bias_width=3, bias_stride=2), B.EINVAL, "bias_ids: stride 2"),
    (dict(mask=FAKE * 4, mask_stride=31), B.EINVAL, "mask: stride 31"),
    (dict(mask=FAKE * 4 + 2, mask_stride=32), B.EALIGN, "mask is not aligned"),
    (dict(mask=FAKE * 2, mask_stride=0), B.EINVAL, "out overlaps mask"),
    (dict(), B.EDEVICE, FINE),
    (dict(p=FAKE, out=FAKE, ot=BF16), B.EDEVICE, FINE),                      # in place
    (dict(rows=1, s=0, os_=0), B.EDEVICE, FINE),
    (dict(HIST), B.EDEVICE, FINE),
    (dict(mask=FAKE * 4, mask_stride=0), B.EDEVICE, FINE),
])
def test_logits_checks(kw, code, msg):
    if msg is FINE:
        if no_device():
            assert logits(**kw) == B.EDEVICE
        return
    assert logits(**kw) == code and msg in error(), error()


def test_logits_no_rows():
    assert logits(rows=0, p=None, out=None) == B.OK


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(B.MoeInt8Epilogue) == 40
    assert ctypes.sizeof(B.MoeLogitsRules) == 11 * 8 + 3 * 8 + 2 * 4


def test_int8_linear_class_checks():
    p, s = torch.zeros(16, 32, dtype=torch.int32), torch.zeros(16, 2, dtype=torch.bfloat16)
    Int8Linear(p, s, 64)
    for bad in (dict(packed=p.float()), dict(packed=p[:, :31]), dict(scales=s[:, :1]), dict(scales=s.float()),
                dict(group=0), dict(group=48), dict(activation="swish")):
        with pytest.raises(ValueError):
            Int8Linear(**{"packed": p, "scales": s, "group": 64, **bad})
    lin = Int8Linear(p, s, 64, bias=torch.zeros(15))
    x = torch.zeros(3, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="bias is"):
        lin.forward(x)
    lin = Int8Linear(p, s, 64)
    with pytest.raises(ValueError, match="x is torch.float32"):
        lin.forward(x.float())
    with pytest.raises(ValueError, match="residual is"):
        lin.forward(x, residual=torch.zeros(3, 15))
    with pytest.raises(ValueError, match="none of bfloat16"):
        lin.forward(x, out_dtype=torch.float64)
    with pytest.raises(ValueError, match="must be on the GPU"):
        lin.forward(x)


@pytest.mark.parametrize("bad,msg", [
    (dict(w_packed=torch.zeros(16, 31, dtype=torch.int32)), "w_packed is"),          # too few words a row
    (dict(w_packed=torch.zeros(15, 32, dtype=torch.int32)), "w_packed is"),          # too few rows
    (dict(w_packed=torch.zeros(32, 16, dtype=torch.int32).t()), "w_packed is"),      # transposed
    (dict(w_packed=torch.zeros(16, 64, dtype=torch.int32)[:, :32]), "w_packed is"),  # inside wider rows
    (dict(w_packed=torch.zeros(16, 32, dtype=torch.int8)), "w_packed is"),           # a quarter of the bytes
    (dict(w_scales=torch.zeros(16, 1, dtype=torch.bfloat16)), "w_scales is"),        # of groups of 128
    (dict(w_scales=torch.zeros(16, 2)), "w_scales is"),
    (dict(w_scales=torch.zeros(16, 2, dtype=torch.float16)), "w_scales is"),
    (dict(w_scales=torch.zeros(2, 16, dtype=torch.bfloat16).t()), "w_scales is"),
    (dict(group=0), "w_scales is"),
    (dict(workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 20)), "workspace is"),
])
def test_fused_call_checks_what_it_dereferences(bad, msg):
    fine = dict(x=torch.zeros(3, 128, dtype=torch.bfloat16), w_packed=torch.zeros(16, 32, dtype=torch.int32),
                w_scales=torch.zeros(16, 2, dtype=torch.bfloat16), tokens=3, n=16, k=128, group=64,
                out=torch.zeros(3, 16))
    with pytest.raises(ValueError, match="x must be on the GPU"):
        B.moe_int8_linear_fused(**fine)
    with pytest.raises(ValueError, match=msg):
        B.moe_int8_linear_fused(**{**fine, **bad})


def test_logits_rules_class_checks():
    i, f = torch.int32, torch.float32
    ok = dict(history=torch.zeros(3, 5, dtype=i), repetition=torch.ones(3))
    for bad, msg in ((dict(repetition=torch.ones(3)), "without history"),
                     (dict(ok, presence=torch.ones(2)), "presence"),
                     (dict(ok, frequency=torch.ones(3, dtype=torch.float64)), "frequency"),
                     (dict(history=torch.zeros(3, 5)), "history"),
                     (dict(bias_ids=torch.zeros(3, 2, dtype=i)), "go together"),
                     (dict(bias_ids=torch.zeros(3, 2, dtype=i), bias_values=torch.zeros(3, 1)), "differ in shape"),
                     (dict(mask=torch.zeros(3, 3, dtype=i)), "words"),
                     (dict(mask=torch.zeros(3, 4)), "mask"),
                     (dict(history=torch.zeros(5, 3, dtype=i).t()), "consecutive"),
                     (dict(ok), "must be on the GPU")):
        with pytest.raises(ValueError, match=msg):
            LogitsRules(100, **bad)
    with pytest.raises(ValueError, match="rows of 100"):
        LogitsRules(100).apply(torch.zeros(2, 99, dtype=f))
