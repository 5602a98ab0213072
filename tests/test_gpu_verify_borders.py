"""moe_int4_verify_drafts where a pick lies close below a border: the first of
two tokens with logits l0 < l1 has the share p = e^(l0 - l1) / (1 + e^(l0 - l1)),
and is the answer as long as p exceeds the pick, here by 1.5 to 3.5 times 10^-15
of itself.

What the kernels may be off by, in units of u = 2^-53: the exponential 2 (its
bound is 2^-52), times 1 - p < 0.9 in the share; the sum, the product with the
pick and their difference 3.  5 u = 5.6 * 10^-16 is a third of the smallest
gap."""
from decimal import Decimal, getcontext

import pytest
import torch

from quantized_moe_router_amd import _binding as B
from quantized_moe_router_amd.layer import DraftVerifier

pytestmark = pytest.mark.gpu

CASES = [
    ("-0x1.4c2ac4p-2", "0x1.78cb4ep-11", "0x1.ad7fe6p-2"),
    ("-0x1.54c8f8p-2", "0x1.6c0a88p-11", "0x1.ab6896p-2"),
    ("-0x1.5bff3cp-2", "0x1.25664ap-11", "0x1.a9b076p-2"),
    ("-0x1.5be45cp-2", "0x1.5b264ap-11", "0x1.a9b076p-2"),
    ("-0x1.0350fcp+0", "0x1.f053a8p-12", "0x1.10b374p-2"),
    ("-0x1.06df7ep+0", "0x1.c4d7e8p-12", "0x1.0df044p-2"),
    ("-0x1.034506p+0", "0x1.57d9d4p-11", "0x1.10b374p-2"),
    ("-0x1.b81a16p+0", "0x1.aceae6p-11", "0x1.370a84p-3"),
    ("-0x1.b71736p+0", "0x1.fe2e42p-12", "0x1.382c1ap-3"),
    ("-0x1.baef98p+0", "0x1.ad8506p-16", "0x1.3456e6p-3"),
    ("-0x1.b814dap+0", "0x1.0a0f78p-11", "0x1.3724e4p-3"),
]


def share(l0, l1):
    getcontext().prec = 60
    e = (Decimal(l0) - Decimal(l1)).exp()
    return e / (1 + e)


def test_picks_just_below_a_border():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    B.lib()
    rows = [[float.fromhex(h) for h in c] for c in CASES]
    for l0, l1, pick in rows:
        p = share(l0, l1)
        assert Decimal("1.5e-15") < (p - Decimal(pick)) / p < Decimal("3.5e-15")
    logits = torch.tensor([r[:2] for r in rows], device="cuda")
    picks = torch.tensor([r[2] for r in rows], device="cuda")
    assert logits.double().tolist() == [r[:2] for r in rows] and picks.double().tolist() == [r[2] for r in rows]
    none = torch.zeros(len(rows), 0, device="cuda")
    tokens, _ = DraftVerifier(2).verify(logits, none.to(torch.int32), none, picks)
    assert tokens[:, 0].tolist() == [0] * len(rows)
    # a step of fp32 above: the other token
    tokens, _ = DraftVerifier(2).verify(logits, none.to(torch.int32), none, torch.nextafter(picks, torch.ones_like(picks)))
    assert tokens[:, 0].tolist() == [1] * len(rows)
