"""Argument checks of moe_int4_linear, moe_int4_grouped_linear and
moe_int4_verify_drafts and of the classes over them: every refusal happens on
the host, before anything touches a device, so none of these needs a GPU."""
import ctypes

import pytest
import torch

from quantized_moe_router_amd import _binding as B
from quantized_moe_router_amd.layer import DraftVerifier, Int4GroupedLinear, Int4Linear

FAKE = 1 << 24   # never dereferenced
BIG = 1 << 44
BF16, F16, F32 = B.TYPE_BF16, B.TYPE_F16, B.TYPE_F32
FINE = "a valid call"   # stops only where there is no gfx950 device; not made where there is one


def error():
    return B.lib().moe_int4_last_error().decode()


def outcome(call, kw, code, msg):
    if msg is FINE:
        if not torch.cuda.is_available():
            assert call(**kw) == B.EDEVICE, error()
        return
    assert call(**kw) == code and msg in error(), error()


def linear(tokens=4, n=320, k=2560, group=64, x=FAKE, xs=2560, wp=FAKE * 2, sc=FAKE * 3, out=FAKE * 4, ot=BF16,
           os_=320, ws=BIG, wb=1 << 40, epi=None):
    e = None if epi is None else B.MoeInt8Epilogue(**epi)
    return B.lib().moe_int4_linear(x, xs, wp, sc, tokens, n, k, group, ctypes.byref(e) if e else None, out, ot, os_,
                                   ws, wb, None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(group=32), B.EINVAL, "group"),
    (dict(k=2500, xs=2504), B.EINVAL, "k="),
    (dict(k=65536 + 64, xs=65536 + 64), B.EINVAL, "k="),
    (dict(n=0), B.EINVAL, "n="),
    (dict(n=(1 << 24) + 1), B.EINVAL, "n="),
    (dict(tokens=-1), B.EINVAL, "tokens"),
    (dict(tokens=(1 << 20) + 1), B.EINVAL, "tokens"),
    (dict(tokens=1 << 20, n=1 << 12), B.EINVAL, "2^31"),
    (dict(x=None), B.EINVAL, "x is NULL"),
    (dict(wp=None), B.EINVAL, "w_packed is NULL"),
    (dict(sc=None), B.EINVAL, "w_scales is NULL"),
    (dict(out=None), B.EINVAL, "out is NULL"),
    (dict(x=FAKE + 8), B.EALIGN, "x is not 16-byte"),
    (dict(wp=FAKE * 2 + 4), B.EALIGN, "w_packed is not 16-byte"),
    (dict(out=FAKE * 4 + 1), B.EALIGN, "out is not aligned"),
    (dict(ot=3), B.EINVAL, "out: type 3"),
    (dict(xs=2559), B.EINVAL, "x: stride"),
    (dict(xs=2564), B.EALIGN, "x: stride 2564"),
    (dict(os_=319), B.EINVAL, "out: stride"),
    (dict(out=FAKE), B.EINVAL, "out overlaps x"),
    (dict(out=FAKE * 2 + 1000), B.EINVAL, "out overlaps w_packed"),
    (dict(out=FAKE * 3 + 64), B.EINVAL, "out overlaps w_scales"),
    (dict(epi=dict(activation=6)), B.EINVAL, "activation 6"),
    (dict(epi=dict(bias=FAKE * 5, bias_type=7)), B.EINVAL, "bias: type 7"),
    (dict(epi=dict(bias=FAKE * 4 + 64, bias_type=BF16)), B.EINVAL, "out overlaps bias"),
    (dict(epi=dict(residual=FAKE * 5, residual_type=F32, residual_stride=0)), B.EINVAL, "residual: stride 0"),
    (dict(epi=dict(residual=FAKE * 4, residual_type=F16, residual_stride=320)), B.EINVAL, "out overlaps residual"),
    # fine up to the device check
    (dict(), B.EDEVICE, FINE),
    (dict(tokens=1, xs=0, os_=0), B.EDEVICE, FINE),
    (dict(xs=4096, out=FAKE + 2 * 2560, os_=4096), B.EDEVICE, FINE),   # column ranges of one matrix
    (dict(epi=dict(residual=FAKE * 4, residual_type=BF16, residual_stride=320)), B.EDEVICE, FINE),   # in place
    (dict(epi=dict(residual=None, residual_type=99, bias_type=99)), B.EDEVICE, FINE),   # not read
])
def test_linear_checks(kw, code, msg):
    outcome(linear, kw, code, msg)


GROUPS = dict(offsets=FAKE * 6, gather=None, scatter=None, row_weights=None, experts=4, places=20, gather_div=1,
              x_rows=20, out_rows=20)


def grouped(n=320, k=2560, group=64, x=FAKE, xs=2560, wp=FAKE * 2, sc=FAKE * 3, out=FAKE * 5, ot=BF16, os_=320,
            ws=BIG, wb=1 << 40, epi=None, groups=True, **u):
    e = None if epi is None else B.MoeInt8Epilogue(**epi)
    g = B.MoeGroups(**{**GROUPS, **u}) if groups else None
    return B.lib().moe_int4_grouped_linear(x, xs, wp, sc, ctypes.byref(g) if g else None, n, k, group,
                                           ctypes.byref(e) if e else None, out, ot, os_, ws, wb, None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(groups=False), B.EINVAL, "groups is NULL"),
    (dict(offsets=None), B.EINVAL, "offsets is NULL"),
    (dict(offsets=FAKE * 6 + 2), B.EALIGN, "offsets is not aligned"),
    (dict(experts=0), B.EINVAL, "experts=0"),
    (dict(experts=1025), B.EINVAL, "experts=1025"),
    (dict(places=-1), B.EINVAL, "places=-1"),
    (dict(places=1 << 20, x_rows=1 << 20, out_rows=1 << 20, n=1 << 12), B.EINVAL, "2^31"),
    (dict(out_rows=1 << 20, scatter=FAKE * 7, n=1 << 12), B.EINVAL, "2^31"),
    (dict(x_rows=19), B.EINVAL, "x_rows=19"),
    (dict(x_rows=0, gather=FAKE * 7), B.EINVAL, "x_rows=0"),
    (dict(out_rows=19), B.EINVAL, "out_rows=19"),
    (dict(out_rows=0, scatter=FAKE * 7), B.EINVAL, "out_rows=0"),
    (dict(gather=FAKE * 7, gather_div=0), B.EINVAL, "gather_div=0"),
    (dict(gather=FAKE * 7 + 1), B.EALIGN, "gather is not aligned"),
    (dict(scatter=FAKE * 7 + 2), B.EALIGN, "scatter is not aligned"),
    (dict(row_weights=FAKE * 7 + 2), B.EALIGN, "row_weights is not aligned"),
    (dict(group=96), B.EINVAL, "group=96"),
    (dict(out=FAKE), B.EINVAL, "out overlaps x"),
    (dict(out=FAKE * 6), B.EINVAL, "out overlaps offsets"),
    (dict(gather=FAKE * 5 + 64), B.EINVAL, "out overlaps gather"),
    (dict(scatter=FAKE * 5 + 64), B.EINVAL, "out overlaps scatter"),
    (dict(row_weights=FAKE * 5 + 64), B.EINVAL, "out overlaps row_weights"),
    # the last expert's codes and scales, and the bias of all
    (dict(out=FAKE * 2 + 4 * 3 * 320 * 320), B.EINVAL, "out overlaps w_packed"),
    (dict(out=FAKE * 3 + 2 * 3 * 320 * 40), B.EINVAL, "out overlaps w_scales"),
    (dict(epi=dict(bias=FAKE * 5 - 2 * 3 * 320, bias_type=BF16)), B.EINVAL, "out overlaps bias"),
    (dict(), B.EDEVICE, FINE),
    (dict(gather=FAKE * 7, gather_div=10, x_rows=2), B.EDEVICE, FINE),
    (dict(scatter=FAKE * 7, out_rows=3, row_weights=FAKE * 8), B.EDEVICE, FINE),
    (dict(epi=dict(bias=FAKE * 5 - 2 * 4 * 320, bias_type=BF16)), B.EDEVICE, FINE),
])
def test_grouped_checks(kw, code, msg):
    outcome(grouped, kw, code, msg)


def test_nothing_to_do_and_workspace_queries():
    assert linear(tokens=0, x=None, out=None) == B.OK
    assert linear(tokens=0, group=3) == B.EINVAL
    assert grouped(places=0, x=None, out=None) == B.OK
    assert verify(seqs=0, target=None) == B.OK
    b = ctypes.c_size_t(1)
    L = B.lib()
    assert L.moe_int4_linear_workspace_bytes(1, 248320, 2560, 128, ctypes.byref(b)) == 0 and b.value == 0
    assert L.moe_int4_linear_workspace_bytes(512, 320, 10240, 65, ctypes.byref(b)) == B.EINVAL
    assert L.moe_int4_linear_workspace_bytes(512, 320, 10240, 64, None) == B.EINVAL
    g = B.MoeGroups(**GROUPS)
    assert L.moe_int4_grouped_linear_workspace_bytes(ctypes.byref(g), 320, 2560, 128, ctypes.byref(b)) == 0
    assert L.moe_int4_grouped_linear_workspace_bytes(None, 320, 2560, 128, ctypes.byref(b)) == B.EINVAL
    assert L.moe_int4_verify_drafts_workspace_bytes(64, 3, 248320, ctypes.byref(b)) == 0 and b.value > 0
    assert L.moe_int4_verify_drafts_workspace_bytes(64, 65, 248320, ctypes.byref(b)) == B.EINVAL
    assert L.moe_int4_verify_drafts_workspace_bytes(64, 3, 248320, None) == B.EINVAL


DRAFTS = dict(target=FAKE * 64, draft=FAKE * 128, tokens=FAKE, lengths=FAKE * 2, coins=FAKE * 3, picks=FAKE * 4,
              temperature=FAKE * 5, target_stride=1000, draft_stride=1000, target_type=F32, draft_type=BF16, seqs=4,
              width=3, vocab=1000)


def verify(accepted=FAKE * 6, tokens_out=FAKE * 7, ws=BIG, wb=1 << 30, drafts=True, **u):
    d = B.MoeDrafts(**{**DRAFTS, **u}) if drafts else None
    return B.lib().moe_int4_verify_drafts(ctypes.byref(d) if d else None, accepted, tokens_out, ws, wb, None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(drafts=False), B.EINVAL, "drafts is NULL"),
    (dict(seqs=-1), B.EINVAL, "seqs=-1"),
    (dict(seqs=65537), B.EINVAL, "seqs=65537"),
    (dict(width=-1), B.EINVAL, "width=-1"),
    (dict(width=65), B.EINVAL, "width=65"),
    (dict(vocab=0), B.EINVAL, "vocab=0"),
    (dict(vocab=(1 << 24) + 1), B.EINVAL, "vocab="),
    (dict(seqs=65536, width=8), B.EINVAL, "2^20"),
    (dict(seqs=65536, width=0, vocab=(1 << 20) + 1, target_stride=1 << 21), B.EINVAL, "2^36"),
    (dict(target=None), B.EINVAL, "target is NULL"),
    (dict(tokens=None), B.EINVAL, "tokens is NULL"),
    (dict(coins=None), B.EINVAL, "coins is NULL"),
    (dict(picks=None), B.EINVAL, "picks is NULL"),
    (dict(accepted=None), B.EINVAL, "accepted is NULL"),
    (dict(tokens_out=None), B.EINVAL, "out_tokens is NULL"),
    (dict(target_type=3), B.EINVAL, "target: type 3"),
    (dict(draft_type=-1), B.EINVAL, "draft: type -1"),
    (dict(target=FAKE * 64 + 2), B.EALIGN, "target is not aligned"),
    (dict(draft=FAKE * 128 + 1), B.EALIGN, "draft is not aligned"),
    (dict(lengths=FAKE * 2 + 2), B.EALIGN, "lengths is not aligned"),
    (dict(target_stride=999), B.EINVAL, "target: stride"),
    (dict(draft_stride=(1 << 24) + 1), B.EINVAL, "draft: stride"),
    (dict(accepted=FAKE * 7), B.EINVAL, "accepted overlaps out_tokens"),
    (dict(accepted=FAKE * 4), B.EINVAL, "accepted overlaps picks"),
    (dict(tokens_out=FAKE * 64 + 400), B.EINVAL, "out_tokens overlaps target"),
    (dict(tokens_out=FAKE), B.EINVAL, "out_tokens overlaps tokens"),
    (dict(ws=None), B.EINVAL, "workspace is NULL"),
    (dict(ws=BIG + 4), B.EALIGN, "workspace is not"),
    (dict(wb=16), B.EWORKSPACE, "workspace has 16"),
    (dict(ws=FAKE * 128), B.EINVAL, "workspace overlaps draft"),
    (dict(), B.EDEVICE, FINE),
    (dict(draft=None, lengths=None, temperature=None, draft_type=9), B.EDEVICE, FINE),
    (dict(width=0, tokens=None, coins=None, draft=None), B.EDEVICE, FINE),
    (dict(seqs=1, width=0, target_stride=0), B.EDEVICE, FINE),
])
def test_verify_checks(kw, code, msg):
    outcome(verify, kw, code, msg)


def test_classes_check_their_tensors():
    packed, scales = torch.zeros(6, 16, dtype=torch.int32), torch.zeros(6, 2, dtype=torch.bfloat16)
    for bad in (dict(packed=packed[:, ::2]), dict(packed=packed.float()), dict(packed=packed[0]),
                dict(scales=scales[:5]), dict(scales=scales.float()), dict(group=128), dict(group=0),
                dict(activation="tanh")):
        with pytest.raises(ValueError):
            Int4Linear(**{**dict(packed=packed, scales=scales, group=64), **bad})
    layer = Int4Linear(packed, scales, 64)
    with pytest.raises(ValueError, match="GPU"):
        layer.forward(torch.zeros(3, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="x is"):
        layer.forward(torch.zeros(3, 128))
    with pytest.raises(ValueError, match="x is"):
        layer.forward(torch.zeros(3, 120, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="residual"):
        layer.forward(torch.zeros(3, 128, dtype=torch.bfloat16), residual=torch.zeros(3, 5))
    packed, scales = packed.view(2, 3, 16), scales.view(2, 3, 2)
    experts = Int4GroupedLinear(packed, scales, 64)
    x, off = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="offsets"):
        experts.forward(x, off[:2])
    with pytest.raises(ValueError, match="offsets"):
        experts.forward(x, off.long())
    with pytest.raises(ValueError, match="scatter"):
        experts.forward(x, off, gather=torch.zeros(4, dtype=torch.int32), scatter=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="row_weights"):
        experts.forward(x, off, row_weights=torch.zeros(5))
    with pytest.raises(ValueError, match="GPU"):
        experts.forward(x, off)
    with pytest.raises(ValueError):
        Int4GroupedLinear(packed[0], scales[0], 64)
    v = DraftVerifier(50)
    with pytest.raises(ValueError, match="GPU"):
        v.verify(torch.zeros(4, 50), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1), torch.zeros(2))
    with pytest.raises(ValueError, match="drafted"):
        v.verify(torch.zeros(4, 50), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 1), torch.zeros(2))
    with pytest.raises(ValueError, match="temperature"):
        DraftVerifier(50, temperature=torch.zeros(3, dtype=torch.float64))
    with pytest.raises(ValueError, match="temperature has 1"):
        DraftVerifier(50, temperature=torch.zeros(1)).verify(
            torch.zeros(4, 50), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1), torch.zeros(2))
