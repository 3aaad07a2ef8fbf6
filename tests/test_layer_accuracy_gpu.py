"""How near the layer's operators come to 64 bits, beyond the bounds of test_layer_gpu.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

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
