"""moe_int4_logits_process at the sizes of serving batches: rows that fill the
chip take slabs of 8192 logits (more than 512 of them in a call), and long
histories whose rows do not begin on 16 bytes.

Tolerances as in test_gpu_logits.py."""
import sys

import numpy as np
import pytest
import torch

from quantized_moe_router_amd.layer import LogitsRules
from test_gpu_logits import FILL, TYPES, check, expected, inside, make

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def ends(u, width, seed):
    """Lengths and prompts at, before and behind the ends of the scan's turns
    (512 threads, four groups of four ids each), groups and tables."""
    edges = np.array([0, 1, 2, 3, 4, 5, 8191, 8192, 8193, 16383, 16384, 16385, width - 1, width, width + 1]).clip(0, width + 1)
    rng = np.random.default_rng(seed)
    for name in ("history_lengths", "prompt_lengths"):
        u[name].copy_(torch.from_numpy(rng.choice(edges, len(u[name])).astype(np.int32)))
    u["history_lengths"][0] = width


BATCHES = [
    # (rows, vocab, history width, biases, mask, in, out, strided): vocabularies
    # of whole slabs, of one token less and more, of a small part of a slab
    (65, 65537, 300, 20, True, "bf16", "fp32", False),
    (65, 65536, 9000, 0, True, "bf16", "bf16", False),
    (65, 65535, 20003, 700, False, "fp32", "fp32", False),
    (65, 65537, 20004, 40, True, "fp16", "fp16", True),
    (20, 248323, 1024, 300, True, "fp32", "fp32", True),
    (20, 248320, 4097, 64, True, "bf16", "fp32", True),
    (20, 248320, 0, 513, True, "fp32", "bf16", False),
    (130, 32003, 77, 40, True, "fp16", "fp32", False),
    (130, 32768, 1, 0, True, "fp16", "fp16", False),
    (300, 16391, 513, 5, False, "bf16", "fp16", True),
    (515, 1000, 64, 3, True, "bf16", "fp32", False),
    (513, 33, 40, 2, True, "fp32", "fp16", True),
    (520, 7, 9, 1, True, "bf16", "bf16", False),
]


@pytest.mark.parametrize("rows,vocab,width,biases,mask,tin,tout,strided", BATCHES)
def test_rules_of_a_batch(rows, vocab, width, biases, mask, tin, tout, strided):
    assert rows * -(-vocab // 8192) > 512
    label = f"batch {rows}x{vocab} history {width} biases {biases} mask {mask} {tin}->{tout} {strided}"
    say(label)
    logits, u = make(rows, vocab, width, biases, mask, rows + vocab, strided, tin)
    if width:
        ends(u, width, rows)
    out = torch.full((rows, vocab), FILL, dtype=TYPES[tout], device="cuda")
    wide = None
    if strided:
        wide, out = inside(out, 9, FILL)
    LogitsRules(vocab, **u).apply(logits, out=out)
    torch.cuda.synchronize()
    check(out, *expected(logits, u), label)
    if strided:
        assert bool((wide[:, vocab:] == FILL).all())


@pytest.mark.parametrize("rows,vocab,t", [(65, 65537, "fp32"), (65, 65536, "bf16"), (40, 131075, "fp16")])
def test_rules_of_a_batch_in_place_and_repeated(rows, vocab, t):
    say(f"in place {rows}x{vocab} {t}")
    logits, u = make(rows, vocab, 700, 30, True, 9, in_type=t)
    rules = LogitsRules(vocab, **u)
    want = expected(logits, u)
    first = rules.apply(logits, out_dtype=TYPES[t])
    for i in range(4):
        torch.randn(1 << 18, device="cuda").sort()   # other kernels leave LDS and caches otherwise
        few = logits.clone()
        got = rules.apply(few, out=few)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.uint8), first.view(torch.uint8)), f"call {i}"
    check(first, *want, "in place")


@pytest.mark.parametrize("rows,vocab,width,tin,tout", [
    (2, 30001, 65539, "bf16", "fp32"), (5, 30001, 16385, "fp32", "fp32"), (9, 300001, 20003, "fp16", "fp16"),
    (3, 50000, 32770, "bf16", "bf16"), (4, 40003, 65537, "fp32", "bf16")])
@pytest.mark.parametrize("shift", [0, 1, 2, 3])
def test_rules_long_history_at_any_place(rows, vocab, width, tin, tout, shift):
    # rows of ids that begin at any word of a 16-byte unit, and logits that
    # share no aligned word
    say(f"{rows}x{vocab} history {width} from word {shift} {tin}->{tout}")
    logits, u = make(rows, vocab, width, 9, True, width + shift, in_type=tin)
    ends(u, width, shift)
    table = torch.full((rows, width + 5), vocab - 1, dtype=torch.int32, device="cuda")
    table[:, shift:shift + width] = u["history"]
    u["history"] = table[:, shift:shift + width]
    out = LogitsRules(vocab, **u).apply(logits, out_dtype=TYPES[tout])
    torch.cuda.synchronize()
    check(out, *expected(logits, u), f"from word {shift}")
