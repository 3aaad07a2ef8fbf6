"""Calls at the edge of what the recurrence's entries accept, in buffers that are there: the counterparts of the
refusals in test_recurrence_abi_cpu.py, whose addresses are made up and which can therefore only be refused."""
from __future__ import annotations

import pytest
import torch

from test_recurrence_gpu import BF16, DEV, F32, kda  # noqa: F401

pytestmark = pytest.mark.gpu
B, T, D, ROWS = 2, 64, 512, 128


def _inputs():
    gen = torch.Generator(device=DEV).manual_seed(1)
    return [torch.randn(B, T, D, generator=gen, device=DEV).to(BF16) for _ in range(3)]


def test_an_output_right_behind_an_input(kda):  # noqa: F811
    x, g, _ = _inputs()
    want, final = kda.gated_scan(x, g, gate="sigmoid")
    both = torch.empty(2, B, T, D, dtype=BF16, device=DEV)
    both[0] = x
    y, state = kda.gated_scan(both[0], g, gate="sigmoid", out=both[1])
    assert torch.equal(y, want) and torch.equal(state, final) and torch.equal(both[0], x)
    with pytest.raises(kda.KdaError):                       # one element earlier it would lie on the input's last
        kda.gated_scan(both[0], g, gate="sigmoid", out=both.view(-1)[ROWS * D - 1:-1].view(B, T, D))


def test_states_in_place_and_inputs_that_share_rows(kda):  # noqa: F811
    x, g, _ = _inputs()
    state = torch.randn(B, D, device=DEV)
    want, final = kda.gated_scan(x, g, gate="sigmoid", initial_state=state)
    both = torch.cat([x, g], -1)
    y, same = kda.gated_scan(both[..., :D], both[..., D:], gate="sigmoid", initial_state=state, final_state=state)
    assert same is state and torch.equal(y, want) and torch.equal(state, final)
    # the same tensor twice
    assert torch.equal(kda.gated_scan(x, x, gate="sigmoid")[0], kda.gated_scan(x, x.clone(), gate="sigmoid")[0])


def test_codes_at_odd_addresses(kda):  # noqa: F811
    x, g, dy = _inputs()
    chunks = torch.empty(kda.gated_scan_chunks(B, T), D, device=DEV)
    kda.gated_scan(x, g, gate="sigmoid", chunk_states=chunks)
    saved = kda.checkpoint_save(x)
    box = torch.empty(ROWS * D + 1, dtype=torch.int8, device=DEV)
    codes = box[1:].view(B, T, D)
    codes.copy_(saved.codes)
    odd = kda.Checkpoint(codes, saved.exponents)
    # codes at odd addresses are read one by one, in another order of sums.  Decays near 1/2 keep the chains' sums of absolute
    # values below 2^11, of which FP32 loses 2^-21; dweight sums 128 products of size 1 within 2^-14; each output is rounded once,
    # by half a step of BF16
    for a, b in zip(kda.gated_scan_backward(dy, odd, g, chunks, gate="sigmoid")[:2],
                    kda.gated_scan_backward(dy, saved, g, chunks, gate="sigmoid")[:2]):
        assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=2.0 ** -10)
    w = torch.ones(D, dtype=BF16, device=DEV)
    for a, b in zip(kda.gated_norm_backward(dy, odd, g, w), kda.gated_norm_backward(dy, saved, g, w)):
        assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=2.0 ** -7 if a.dim() == 1 else 2.0 ** -10)
    assert torch.equal(kda.checkpoint_load(odd, BF16), kda.checkpoint_load(saved, BF16))


def test_a_pool_of_no_states(kda):  # noqa: F811
    x, g, _ = _inputs()
    pool, slots = torch.empty(0, D, device=DEV), torch.zeros(8, dtype=torch.int32, device=DEV)
    y = kda.gated_step(x[0, :8], g[0, :8], pool, slots=slots)
    assert torch.equal(y, x[0, :8])                         # a state of zeros, and nothing stored


def test_the_least_workspace(kda):  # noqa: F811
    x, g, dy = _inputs()
    w = torch.ones(D, dtype=BF16, device=DEV)
    need = kda.gated_norm_backward_workspace_size(ROWS, D)
    box = torch.full((need + 64,), 9, dtype=torch.uint8, device=DEV)
    got = kda.gated_norm_backward(dy, x, g, w, workspace=box[16:16 + need])
    assert all(torch.equal(a, b) for a, b in zip(got, kda.gated_norm_backward(dy, x, g, w)))
    assert (box[:16] == 9).all() and (box[16 + need:] == 9).all()
    with pytest.raises(kda.KdaError):
        kda.gated_norm_backward(dy, x, g, w, workspace=box[16:15 + need])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_checkpoints_of_plain_buffers(kda, dtype):  # noqa: F811
    x = torch.randn(10, 100, device=DEV).to(dtype)
    got = kda.checkpoint_load(kda.checkpoint_save(x), dtype)
    # half a step, 1 / 127 of the block's largest at most
    top = torch.nn.functional.pad(x.float(), (0, 28)).view(10, 4, 32).abs().amax(-1).repeat_interleave(32, -1)[:, :100]
    assert ((got.float() - x.float()).abs() <= top / 127).all()
