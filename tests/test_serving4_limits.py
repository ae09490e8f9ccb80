"""Host-side refusals of the serving step's other operators that need no GPU: arrays over one another."""
import ctypes as C

import pytest

from mxfp4_mixture_experts_rms_gb300 import build, moe


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.load()


def verify(L, **over):
    """moe_verify on 6 rows of 10 fp32 logits (10 draft probabilities, each 12 apart) of 2 sequences, at made-up addresses."""
    a = dict(x=0x10000, bf=0, stride=12, drafts=0x20000, probs=0x30000, probs_stride=12, starts=0x40000, t=0x50000, k=0x60000, p=0x70000,
             mp=0x80000, u=0x90000, draws=0xa0000, ids=0xb0000, acc=0xc0000, ws=0xd0000)
    a.update(over)
    P = C.c_void_p
    return L.moe_verify(P(a["x"]), a["bf"], 6, 10, a["stride"], P(a["drafts"]), P(a["probs"]), a["probs_stride"], P(a["starts"]), 2, P(a["t"]), P(a["k"]),
                        P(a["p"]), P(a["mp"]), P(a["u"]), P(a["draws"]), P(a["ids"]), P(a["acc"]), P(a["ws"]), 6 * 24, None)


@pytest.mark.parametrize("what", ["x", "probs"])
def test_verify_refuses_outputs_over_the_rows_that_it_reads(L, what):
    base = dict(x=0x10000, probs=0x30000)[what]
    for out, size in (("ids", 24), ("acc", 8)):
        for at in (base, base + 4 * 11 - size, base + 4 * 12, base + 4 * (5 * 12 + 9), base - size + 4, base + 4 * 30):
            assert verify(L, **{out: at}) == moe.MOE_EINVAL, (out, at - base)
            assert b"overlap" in L.moe_last_error()


def test_verify_refuses_outputs_over_bf16_rows(L):
    for at in (0x10000 + 2 * (5 * 12 + 8), 0x10000 + 2 * 12, 0x10000 - 4):
        assert verify(L, bf=1, acc=at) == moe.MOE_EINVAL


def test_verify_refuses_a_workspace_over_anything_else(L):
    for name, size in (("ids", 24), ("acc", 8), ("drafts", 24), ("starts", 12), ("u", 24), ("draws", 8), ("t", 8), ("k", 8), ("p", 8), ("mp", 8)):
        for at in (0xd0000, 0xd0000 + 6 * 24 - 4, 0xd0000 - size + 4):
            assert verify(L, **{name: at}) == moe.MOE_EINVAL, (name, at - 0xd0000)
            assert b"overlap" in L.moe_last_error()
    for name in ("x", "probs"):
        for at in (0xd0000, 0xd0000 + 6 * 24 - 4, 0xd0000 - 4 * (5 * 12 + 9)):
            assert verify(L, **{name: at}) == moe.MOE_EINVAL, (name, at - 0xd0000)


def test_verify_takes_outputs_beside_the_rows(L):
    # behind a row's logits, where rows lie apart, and right before and behind the arrays: no overlap (the call then has no GPU)
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where no kernel can be launched")
    for over in (dict(acc=0x10000 + 4 * 10), dict(acc=0x30000 + 4 * (2 * 12 + 10)), dict(ids=0x10000 + 4 * (5 * 12 + 10)), dict(ids=0x10000 - 24),
                 dict(ids=0xd0000 - 24), dict(acc=0xd0000 + 6 * 24), dict(stride=16, ids=0x10000 + 4 * 26), dict(probs=0)):
        assert verify(L, **over) == moe.MOE_ECUDA, over
