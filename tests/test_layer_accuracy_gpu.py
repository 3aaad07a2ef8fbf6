"""How near the layer's operators come to 64 bits, beyond the bounds of test_layer_gpu.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.layer as ref

from test_layer_gpu import BF16, DEV, F16, F32, Rule, close, f64, kda  # noqa: F401

pytestmark = pytest.mark.gpu


# A 16-bit output is an FP32 one rounded once.  With e the FP32 result's error (the header's 1e-6 of the
# result's norm), an element rounds to another neighbour than the 64-bit result does with probability
# |e| / ulp, by one ulp: the mean square of the difference is E|e| ulp <= rms(e) rms(ulp), where an ulp is at
# most 2^-7 (BF16) or 2^-10 (FP16) of its value.  Twice the root of that allows for the sample.
@pytest.mark.parametrize("dtype, ulp", [(BF16, 2.0 ** -7), (F16, 2.0 ** -10)], ids=str)
@pytest.mark.parametrize("K, gate", [(128, "channel"), (64, "head"), (96, "channel")])
def test_prefill_output_is_rounded_once(kda, dtype, ulp, K, gate):  # noqa: F811
    x = Rule([300, 64, 130], Hk=2, H=4, K=K, dtype=dtype, gate=gate, seed=61, rate=0.2, initial=True)
    o, _ = x.run(kda)
    want = np.concatenate(x.want()[0])
    rounded = f64(torch.from_numpy(want).to(dtype))
    off = np.linalg.norm(f64(o) - rounded) / np.linalg.norm(want)
    assert off <= 2 * np.sqrt(1e-6 * ulp), off


CHUNK = 64


def faded(x, big, clear, fall):
    """One sequence whose values are of 1e8 in its first `big` chunks and of 1e-6 after them, and whose chunk
    `clear` leaves next to nothing of the state: each row of it the same share, or the first ten rows all.  Rows
    from the end of that chunk on see 1e8 e^-64 or 1e8 e^-28 of what was before."""
    x.v[0, :CHUNK * big] *= 1e8
    x.v[0, CHUNK * big:] *= 1e-6
    if fall == "even":
        x.g[0, CHUNK * clear:CHUNK * (clear + 1)] = -1.0
    else:
        x.g[0, CHUNK * clear:CHUNK * clear + 10] = -2.8
    return CHUNK * (clear + 1)


# 32 chunks of one head, which are walked in segments of four to eleven chunks: the chunk that clears the state
# stands in all places of several segments, after the large values at once (a segment's own state) or later (the
# state that comes into a segment).
@pytest.mark.parametrize("big, clear", [(2, c) for c in range(3, 24, 2)] + [(c, c) for c in (3, 7, 8, 11, 14, 15, 17)])
@pytest.mark.parametrize("fall", ["even", "first rows"])
@pytest.mark.parametrize("K, V, dtype, gate", [(64, 32, F32, "channel"), (128, 128, F32, "head"), (96, 64, BF16, "channel")],
                         ids=str)
def test_split_sequence_forgets_what_a_chunk_clears(kda, big, clear, fall, K, V, dtype, gate):  # noqa: F811
    x = Rule([32 * CHUNK], Hk=1, H=1, K=K, V=V, dtype=dtype, gate=gate, seed=big + clear, rate=0.002)
    a = faded(x, big, clear, fall)
    o, S = x.run(kda)
    wo, wS = x.want()
    close(o[a:], wo[0][a:], dtype, "outputs after the chunk")
    close(S[0], wS[0], F32, "state")
    close(o, wo[0], dtype, "all outputs")


# In FP32, units of 2^-24: the exponential 2, the sum with one 1, the quotient 1, four products 4, the root 4, the
# mean of 128 squares (a chain of four and five steps between lanes, halved by the root) 5: 17, and 20 allowed.
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gated_norm_gates_far_out(kda, act):  # noqa: F811
    rng = np.random.default_rng(71)
    gate = torch.from_numpy(np.linspace(-86, 40, 128 * 512).reshape(512, 128)).float()
    x = torch.from_numpy(rng.standard_normal((512, 128))).float()
    w = torch.from_numpy(1 + 0.1 * rng.standard_normal(128)).float()
    want = ref.gated_norm(f64(x), f64(gate), f64(w), 1e-6, act)
    got = f64(kda.gated_norm(x.to(DEV), gate.to(DEV), w.to(DEV), activation=act))
    worst = np.max(np.abs(got - want) / (np.abs(want) + 1e-38))
    assert worst <= 20 * 2.0 ** -24, f"{worst * 2 ** 24:.1f} units of 2^-24"


# Both ways round at the same places to a type of unit roundoff u, and differ where a value falls on the other side:
# some eight roundings a layer, each at most u / sqrt(3) sqrt(2) in the mean, two layers and a last norm: 17 of them
# make 3.4 u in the mean square, 4 times that for the largest of 4000 outputs, which are up to 4 times their mean
# themselves; four times the 3.4 u that this comes to allows for what the layers amplify.
@pytest.mark.parametrize("dtype, u", [(F16, 2.0 ** -11), (BF16, 2.0 ** -8)], ids=str)
def test_example_differs_by_roundings(dtype, u):
    from test_layer_example_gpu import _example

    _, off = _example().run(dtype, layers=2, dim=256, heads=4, width=64, lengths=(70, 1, 33), new_tokens=5)
    assert off <= 14 * u, off / u
