"""The gated delta rule over sequences that are split into segments: states updated in place,
packed batches with more walks than the GPU has SMs.

Tolerances are those of test_layer_gpu.py, fixed there.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from test_layer_gpu import BF16, DEV, F16, F32, Rule, close, kda  # noqa: F401

pytestmark = pytest.mark.gpu


def pooled(kda, x, in_place, slots, entries):
    """The rule over x with its states in a pool; (o, the pool written)."""
    pool = torch.full((entries, x.H, x.K, x.V), 7.0, device=DEV)
    pool[slots.long()] = x.state.to(DEV)
    out = pool if in_place else torch.full_like(pool, 7.0)
    o, S = kda.delta_prefill(*x.args(), cu_seqlens=x.cu.to(DEV), initial_state=pool, final_state=out, slots=slots)
    torch.cuda.synchronize()
    assert S is out
    return o[0], out


# Lengths and heads for which sequences are split and the first segment of the last sequence is walked
# after its last segment (which has fewer chunks, on a CTA that had less to do before).
LATE = [([384, 640, 1024, 2048, 384], 10), ([2568, 13017, 153, 2713], 16), ([4160, 1, 16384, 4160], 16)]


@pytest.mark.parametrize("lens, H", LATE[:1], ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_split_states_in_place(kda, lens, H, dtype):  # noqa: F811
    x = Rule(lens, Hk=H, H=H, dtype=dtype, seed=51, rate=0.02, initial=True)
    wo, wS = x.want()
    slots = torch.tensor([5, 2, 6, 0, 3], dtype=torch.int32, device=DEV)
    o, pool = pooled(kda, x, True, slots, 7)
    for n, (a, b) in enumerate(x.rows()):
        close(o[a:b], wo[n], dtype, f"o of sequence {n}")
        close(pool[int(slots[n])], wS[n], F32, f"state of sequence {n}")
    assert torch.all(pool[1] == 7) and torch.all(pool[4] == 7)
    # without slots, the final states over the initial ones
    S0 = x.state.to(DEV)
    o2, S = kda.delta_prefill(*x.args(), cu_seqlens=x.cu.to(DEV), initial_state=S0, final_state=S0)
    torch.cuda.synchronize()
    assert S is S0 and torch.equal(o2[0], o) and torch.equal(S, pool[slots.long()])


@pytest.mark.parametrize("lens, H", LATE, ids=str)
def test_split_in_place_is_out_of_place(kda, lens, H):  # noqa: F811
    """Bit for bit, whichever CTA is first."""
    x = Rule(lens, Hk=H, H=H, K=64, V=128, dtype=BF16, seed=52, rate=0.02, initial=True)
    slots = torch.tensor(np.random.default_rng(0).permutation(len(lens)), dtype=torch.int32, device=DEV)
    o, S = pooled(kda, x, False, slots, len(lens))
    for _ in range(3):
        o2, S2 = pooled(kda, x, True, slots, len(lens))
        assert torch.equal(o2, o) and torch.equal(S2, S)


def test_split_in_place_dense(kda):  # noqa: F811
    for B, T, H in ((2, 8192, 16), (7, 2048, 3), (1, 5000, 32)):
        x = Rule([T] * B, Hk=H, H=H, K=32, V=96, dtype=BF16, packed=False, seed=53, rate=0.02, initial=True)
        o, S = x.run(kda)
        S0 = x.state.to(DEV)
        o2, _ = kda.delta_prefill(*x.args(), initial_state=S0, final_state=S0)
        torch.cuda.synchronize()
        assert torch.equal(o2.reshape(-1, H, 96), o) and torch.equal(S0, S)


def test_split_slots_of_none(kda):  # noqa: F811
    """Split sequences among which one has no slot: it starts from zero and is not stored."""
    x = Rule([2500, 3100, 0, 2000], Hk=2, H=2, dtype=F32, seed=54, rate=0.02, initial=True)
    slots = torch.tensor([3, -1, 1, 9], dtype=torch.int32, device=DEV)
    pool = torch.randn(5, 2, 128, 128, device=DEV)
    before = pool.clone()
    x.state = torch.stack([before[s].cpu() if 0 <= s < 5 else torch.zeros(2, 128, 128) for s in slots.tolist()])
    wo, wS = x.want()
    o, _ = kda.delta_prefill(*x.args(), cu_seqlens=x.cu.to(DEV), initial_state=pool, slots=slots)
    torch.cuda.synchronize()
    for n, (a, b) in enumerate(x.rows()):
        close(o[0, a:b], wo[n], F32, f"o {n}")
    close(pool[3], wS[0], F32, "state 0")
    assert all(torch.equal(pool[e], before[e]) for e in (0, 1, 2, 4))


@pytest.mark.parametrize("packed", [False, True])
def test_workspace_without_room_for_segments(kda, packed):  # noqa: F811
    """A workspace that holds all but the segments' maps: the sequences are walked whole."""
    x = Rule([2500, 2500], Hk=2, H=2, dtype=F32, packed=packed, seed=55, rate=0.02, initial=True)
    size = kda.delta_prefill_workspace_size(*((1, 5000, 2, 2) if packed else (2, 2500, 2)))
    chunks = (5000 + 126) // 64 if packed else 80
    least = 32896 * chunks * 2 + (32 if packed else 0)
    assert size > least
    for given in (least, size - 1, size):
        ws = torch.full((given + 256,), 255, dtype=torch.uint8, device=DEV)
        x.check(kda, f"{given} bytes", workspace=ws[:given])
        assert torch.all(ws[given:] == 255)
    with pytest.raises(kda.KdaError, match="workspace"):
        x.run(kda, workspace=ws[:least - 1])


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("lens, H, reps", [([384, 640, 1024, 2048, 384], 10, 300), ([4160, 1, 16384, 4160], 16, 30),
                                           ([320] * 40, 16, 60)], ids=str)
def test_prefill_repeats_bit_for_bit_over_many_walks(kda, dtype, lens, H, reps):  # noqa: F811
    """Several walks to a CTA, so that their buffers go from one to the next while other warps still read; one
    chunk's row read too late shows in some runs only."""
    x = Rule(lens, Hk=H, H=H, dtype=dtype, seed=57, rate=0.02, initial=True)
    args, cu, S0 = x.args(), x.cu.to(DEV), x.state.to(DEV)
    o, S = (t.clone() for t in kda.delta_prefill(*args, cu_seqlens=cu, initial_state=S0))
    out, S1 = torch.empty_like(o), torch.empty_like(S)
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(reps):
        out.zero_()
        kda.delta_prefill(*args, cu_seqlens=cu, initial_state=S0, final_state=S1, out=out)
        differ += (out != o).any() | (S1 != S).any()
    assert int(differ) == 0


def test_workspace_of_repeated_bytes(kda):  # noqa: F811
    """A view with more elements than memory is refused before anything is launched."""
    x = Rule([130, 64], dtype=BF16, seed=56)
    need = kda.delta_prefill_workspace_size(1, 194, 2, 2)
    one = torch.zeros(16, dtype=torch.uint8, device=DEV)
    for ws in (one.repeat(2)[::2], one[:1].expand(need), torch.zeros(2 * need, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            x.run(kda, workspace=ws)
