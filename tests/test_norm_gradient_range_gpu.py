"""The gated norm's gradients where the gate is far below zero: at the type's lowest value, as masks have it, and on the way there.

Tolerances, from the arithmetic: that of test_recurrence_gpu.py (2^-17 of the oracle's sums of absolute values) and, for each
of the two factors that come from the sigmoid, the fast exponential's |z| 2^-24 + 2^-21 for arguments down to -88: 2^-15
in all.  A sigmoid below 2^-126 may be taken as 0, so that act(z) and its slope are off by at most
88 * 2^-126 < 2^-119: that much of dy w, and of what the mean makes of it, in absolute terms."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.recurrence as ref
from test_recurrence_gpu import BF16, DEV, DTYPES, F32, f64, kda, near  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("rows, dim", [(5, 64), (3, 33), (4, 513), (2, 4096), (2, 16384)])
def test_gates_far_below_zero(kda, dtype, act, rows, dim):  # noqa: F811
    rng = np.random.default_rng(dim)
    low = float(torch.finfo(dtype).min)
    values = [v for v in (low, low / 2, -1e38, -1e30, -1e20, -1e4, -1000.0, -200.0, -104.0, -100.0, -90.0, -88.0, -87.0, -80.0, -50.0,
                          -20.0, 0.0, 3.0, 100.0) if v >= low]
    x, dy = (torch.from_numpy(s * rng.standard_normal((rows, dim))).to(dtype) for s in (0.3, 1.0))
    w = torch.from_numpy(1 + 0.1 * rng.standard_normal(dim)).to(dtype)
    mixed = torch.tensor([values[i % len(values)] for i in range(rows * dim)], dtype=torch.float64).reshape(rows, dim).to(dtype)
    masked = torch.full((rows, dim), low, dtype=dtype)      # a row that leaves nothing
    masked[0, : dim // 2] = 1.0
    for z, name in ((mixed, "mixed"), (masked, "masked")):
        for saved in (False, True):
            gz, wz = z.to(DEV), f64(z)
            if saved:
                gz, wz = kda.checkpoint_save(gz), ref.checkpoint(wz, -low)[2]
            dx, dz, dw = kda.gated_norm_backward(dy.to(DEV), x.to(DEV), gz, w.to(DEV), eps=1e-5, activation=act)
            rx, rz, rw, sx, sz, sw = ref.gated_norm_backward(f64(dy), f64(x), wz, f64(w), 1e-5, act)
            r = 1 / np.sqrt(np.mean(f64(x) ** 2, -1, keepdims=True) + 1e-5)
            n, into = np.abs(f64(x)) * r, np.abs(f64(dy) * f64(w))
            least = 2.0 ** -119
            near(dx, rx, 2.0 ** -15 * sx + least * r * (into + n * np.mean(into * n, -1, keepdims=True)), f"dx {name} {saved}")
            near(dz, rz, 2.0 ** -15 * sz + least * into * n, f"dgate {name} {saved}")
            near(dw, rw, 2.0 ** -14 * sw + least * (np.abs(f64(dy)) * n).sum(0), f"dweight {name} {saved}")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_masked_gate_gives_no_gradient(kda, dtype):  # noqa: F811
    """The lowest gate behind SiLU: nothing passes, as in the forward operator."""
    low = float(torch.finfo(dtype).min)
    x, dy = (torch.randn(4, 128, device=DEV).to(dtype) for _ in range(2))
    w, z = torch.ones(128, dtype=dtype, device=DEV), torch.full((4, 128), low, dtype=dtype, device=DEV)
    assert (kda.gated_norm(x, z, w, activation="silu") == 0).all()
    for gate in (z, kda.checkpoint_save(z)):
        assert all((t == 0).all() for t in kda.gated_norm_backward(dy, x, gate, w, activation="silu"))
