"""Refusals of the layer operators that need no GPU, and their sizes at the limits.

A call that passes the checks would launch on made-up addresses, so every call here is refused: where a
size is just allowed, a missing pointer refuses it after the sizes were looked at."""
import pytest

import linear_attention_chunked_02_gb300 as kda
from test_layer_abi_cpu import INVALID, L, P, UNSUPPORTED, WORKSPACE, prefill, step  # noqa: F401

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


def test_prefill_limits(L):  # noqa: F811
    """Each limit of the header from both sides."""
    def sized(**kw):
        return prefill(L, q=None, **kw)                    # INVALID where the sizes pass

    top = 1 << 17
    assert sized(Hk=1, H=top - 1) == INVALID and sized(Hk=1, H=top) == UNSUPPORTED
    assert sized(Hk=1, H=top - 1, K=32, V=32) == INVALID and sized(Hk=1, H=top, K=32, V=32) == UNSUPPORTED
    assert sized(T=(1 << 31) - 129, Hk=1, H=1) == INVALID and sized(T=(1 << 31) - 128, Hk=1, H=1) == UNSUPPORTED
    # sequences x heads
    assert sized(cu=P[8], nseq=(1 << 20) - 1, T=1, Hk=1, H=256) == INVALID
    assert sized(cu=P[8], nseq=1 << 20, T=1, Hk=1, H=256) == UNSUPPORTED
    # chunks x heads
    assert sized(T=64 * ((1 << 20) - 1), Hk=1, H=1024) == INVALID
    assert sized(T=64 * (1 << 20), Hk=1, H=1024) == UNSUPPORTED


def test_step_limits(L):  # noqa: F811
    assert step(L, q=None, N=(1 << 20) - 1, nslots=1 << 20, Hk=1, H=256) == INVALID
    assert step(L, q=None, N=1 << 20, nslots=1 << 20, Hk=1, H=256) == UNSUPPORTED
    assert step(L, q=None, Hk=1, H=(1 << 17) - 1) == INVALID and step(L, q=None, Hk=1, H=1 << 17) == UNSUPPORTED


@pytest.mark.parametrize("T, seqs", [(1000, 0), (1000, 7), (16384, 0), (16384, 1), (20000, 3), (40, 7)])
@pytest.mark.parametrize("K, V, H", [(128, 128, 2), (32, 96, 1), (64, 128, 300)])
def test_prefill_workspace_is_what_the_header_says(L, T, seqs, K, V, H):  # noqa: F811
    got = WS(1, T, H, seqs, K, V)
    if T < 16 * seqs:
        assert got == 0
        return
    chunks = (T + 63) // 64 if seqs == 0 else (T + 63 * seqs) // 64
    rest = got - 32896 * chunks * H
    if H * max(1, seqs) >= 152:                            # never split
        assert rest == 16 * seqs
        return
    unit = K * (K + V) * 4 * H + (16 if seqs else 0)
    assert rest == 16 * seqs or (rest % unit == 0 and rest // unit > max(1, seqs))


def test_prefill_workspace_of_split_sequences(L):  # noqa: F811
    """One long sequence is split, packed or not: the segments' maps, and 16 bytes each where packed."""
    dense, packed = WS(1, 16384, 2), WS(1, 16384, 2, 1)
    images, unit = 32896 * 256 * 2, 128 * 256 * 4 * 2
    parts = (dense - images) // unit
    assert parts > 1 and dense == images + parts * unit
    assert packed - images in [n * (unit + 16) for n in (parts, parts + 1)]


def test_prefill_workspace_serves_smaller_prompts(L):  # noqa: F811
    """The size for one T is refused for no smaller one; what has no room for the images is, for every T."""
    def given(T, ws, H, seqs):                             # a misplaced o refuses the call after the workspace's size
        packed = {"cu": P[8], "nseq": seqs} if seqs else {}
        return prefill(L, T=T, Hk=1, H=H, o=P[0], ws=P[11] * 64, wsb=ws, **packed)

    for H, seqs in ((1, 0), (16, 0), (32, 0), (16, 4), (2, 3)):
        largest, shrinks = 0, 0
        for T in range(64, 20000, 320):
            size = WS(1, T, H, seqs)
            shrinks += size < largest
            largest = max(largest, size)
            chunks = (T + 63) // 64 if seqs == 0 else (T + 63 * seqs) // 64
            least = 32896 * chunks * H + 16 * seqs
            if size:
                assert given(T, least, H, seqs) == INVALID and given(T, least - 1, H, seqs) == WORKSPACE
                for longer in range(T, T + 3000, 320):
                    assert WS(1, longer, H, seqs) >= least
        assert shrinks > 0


def test_stream_of_another_device():
    """Refused, not left for the tensors' device's current stream."""
    class Stream:
        device_index = 1

    from linear_attention_chunked_02_gb300 import layer
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        layer._elsewhere(0, Stream())
