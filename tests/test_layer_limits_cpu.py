"""Refusals of the layer operators that need no GPU.

A call that passes the checks would launch on made-up addresses, so every call here is refused."""
import pytest

import linear_attention_chunked_02_gb300 as kda
from test_layer_abi_cpu import INVALID, L, P, prefill, step  # noqa: F401

WS = kda.delta_prefill_workspace_size


# 64 tokens, two heads of 128: q, k, v, o 32 KiB each (BF16), g 64 KiB, beta 256 B, states 128 KiB
SIZES = {"q": 64 * 512, "k": 64 * 512, "v": 64 * 512, "g": 64 * 1024, "beta": 64 * 4, "o": 64 * 512, "sin": 1 << 17,
         "sout": 1 << 17}


@pytest.mark.parametrize("written", ["o", "sout", "ws"])
@pytest.mark.parametrize("other", ["q", "k", "v", "g", "beta", "sin", "sout", "o", "slots", "cu", "ws"])
def test_prefill_refuses_overlapping_buffers(L, written, other):  # noqa: F811
    if other == written or {written, other} == {"sout", "sin"}:
        pytest.skip("the same buffer, or states in place")
    sizes = dict(SIZES, ws=WS(1, 64, 2, 1 if other == "cu" else 0), slots=4, cu=8)
    base = {"q": P[0], "k": P[1], "v": P[2], "g": P[3], "beta": P[4], "o": P[5], "sout": P[6], "ws": P[7], "sin": P[8],
            "slots": P[10], "cu": P[11]}
    for name, count in (("slots", "nslots"), ("cu", "nseq")):
        if name == other:
            base[count] = 1
        else:
            del base[name]
    at = base[other]
    for start in (at, at - sizes[written] + 16, at + max(0, sizes[other] - 16)):
        assert prefill(L, **dict(base, **{written: start}), wsb=sizes["ws"]) == INVALID, (start, at)


@pytest.mark.parametrize("written", ["o", "state"])
@pytest.mark.parametrize("other", ["q", "k", "v", "g", "beta", "slots", "o", "state"])
def test_step_refuses_overlapping_buffers(L, written, other):  # noqa: F811
    if other == written:
        pytest.skip("the same buffer")
    sizes = {"q": 4 * 512, "k": 4 * 512, "v": 4 * 512, "g": 4 * 1024, "beta": 16, "o": 4 * 512, "state": 4 << 17,
             "slots": 16}
    base = {"q": P[0], "k": P[1], "v": P[2], "g": P[3], "beta": P[4], "o": P[5], "state": P[6], "slots": P[7]}
    at = base[other]
    for start in (at, at - sizes[written] + 16, at + sizes[other] - 16):
        assert step(L, **dict(base, **{written: start})) == INVALID, (start, at)
