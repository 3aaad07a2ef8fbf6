"""The example that serves a stack of layers with the four operators together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "kda_layers.py")


def _example():
    spec = importlib.util.spec_from_file_location("kda_layers", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


# Both ways round every intermediate to the dtype (unit roundoff u) at the same places, so that they differ
# by single roundings: some twenty a layer, carried through two layers and a residual sum of unit gain.
# 256 u covers them with room: 1.5e-5 in FP32, 0.125 for FP16, as a share of the largest output.
@pytest.mark.parametrize("dtype, u", [(torch.float32, 2.0 ** -24), (torch.float16, 2.0 ** -11)])
def test_example_decodes_what_it_prefills(dtype, u):
    figures, off = _example().run(dtype, layers=2, dim=256, heads=4, width=64, lengths=(70, 1, 33), new_tokens=5)
    assert off <= 256 * u
    assert all(value > 0 for value in figures.values())
