"""The recurrence on rows of whole 16-byte pieces whose outputs and states lie at addresses that are aligned to their
elements alone, and whose inputs are slices of wider rows: the values within the oracle's bounds and,
where the same kernels can take them, the same bits as from buffers of their own; nothing written beside them.

Tolerances: those of test_recurrence_gpu.py, which follow from the oracle's bounds on FP32 arithmetic."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.recurrence as ref
from test_recurrence_gpu import BF16, DEV, F16, F32, Case, f64, kda, near  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16)]
GUARD = 64


def boxed(t, offset, fill=None):
    """A contiguous copy of t `offset` elements past a 256-byte boundary (or that place, filled), and the buffer around it."""
    whole = torch.full((2 * GUARD + offset + t.numel(),), 5.0, dtype=t.dtype, device=DEV)
    inner = whole[GUARD + offset:GUARD + offset + t.numel()].view(t.shape)
    if fill is None:
        inner.copy_(t)
    else:
        inner.fill_(fill)
    return whole, inner


def untouched(whole, inner):
    at = inner.storage_offset()
    return bool((whole[:at] == 5.0).all() and (whole[at + inner.numel():] == 5.0).all())


def _lens(n, longest, seed):
    return [int(v) for v in np.random.default_rng(seed).integers(0, longest + 1, n)]


# Walked by single warps (8 bytes of x to a lane, or 4), packed and dense; chained, by clusters or by blocks alone.
SHAPES = {"walked": (512, _lens(400, 12, 1), True), "walked dense": (512, [9] * 230, False), "walked narrow": (256, [9] * 300, True),
          "chained": (64, [3000, 1, 0, 900, 70], True), "chained dense": (72, [400] * 3, False)}


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype, gdtype", TYPES)
def test_scans_into_buffers_at_any_element(kda, shape, dtype, gdtype):  # noqa: F811
    D, lens, packed = SHAPES[shape]
    c = Case(lens, D, dtype, gdtype, "sigmoid", True, packed=packed, seed=D)
    x, g, cu, state = c.gpu(c.x), c.gpu(c.g), c.gpu(c.cu), c.gpu(c.state)
    wy, wf, wc, by, bf, bc = c.want()
    empty = np.isnan(wc)
    new = torch.empty(kda.gated_scan_chunks(*x.shape[:2]), D, device=DEV)
    y, final = kda.gated_scan(x, g, cu, initial_state=state, chunk_states=new, **c.form)
    for offset in (0, 1, 2, 3, 4):
        for which in ("y", "state_in", "state_out", "chunks", "in place", "all"):
            def at(name):
                return offset if which in (name, "all") or (which == "in place" and name in ("state_in", "state_out")) else 0

            boxes = {"y": boxed(y, at("y"), 3.0), "state_in": boxed(state, at("state_in")),
                     "state_out": boxed(final, at("state_out"), 3.0), "chunks": boxed(new, at("chunks"), 7.0)}
            if which == "in place":
                boxes["state_out"] = boxes["state_in"]
            out, first, last, chunks = (boxes[n][1] for n in ("y", "state_in", "state_out", "chunks"))
            assert out.data_ptr() % 16 == at("y") * out.element_size() % 16
            got = kda.gated_scan(x, g, cu, initial_state=first, final_state=last, chunk_states=chunks, out=out, **c.form)
            label = f"{shape} {offset} {which}"
            near(got[0], wy, by, f"{label} y")
            near(got[1], wf, bf, f"{label} final")
            near(chunks, wc, bc, f"{label} chunk states")
            assert all(untouched(*b) for b in boxes.values()), label
            assert (f64(chunks)[empty] == 7.0).all()
            if offset % 2 == 0:                             # vectors of two elements: the same arithmetic, row by row
                assert torch.equal(got[0], y) and torch.equal(got[1], final), label
                assert torch.equal(chunks[torch.from_numpy(~empty).to(DEV)], new[torch.from_numpy(~empty).to(DEV)]), label
            if which != "in place":
                assert torch.equal(first, state), label


@pytest.mark.parametrize("shape", ["walked", "chained", "chained dense"])
@pytest.mark.parametrize("dtype, gdtype", TYPES)
@pytest.mark.parametrize("saved", [False, True])
def test_gradients_into_buffers_at_any_element(kda, shape, dtype, gdtype, saved):  # noqa: F811
    D, lens, packed = SHAPES[shape]
    c = Case(lens, D, dtype, gdtype, "sigmoid", True, packed=packed, seed=D)
    chunks = torch.from_numpy(np.nan_to_num(c.want()[2], nan=5.0)).to(F32).to(DEV)
    x, g, dy, cu, state, dfinal = (c.gpu(t) for t in (c.x, c.g, c.dy, c.cu, c.state, c.dfinal))
    wx, wg = c.flat(c.x), c.flat(c.g)
    if saved:
        x, g, wx, wg = kda.checkpoint_save(x), kda.checkpoint_save(g), ref.checkpoint(wx)[2], ref.checkpoint(wg)[2]
    like = torch.empty(c.dy.shape, dtype=gdtype, device=DEV)
    wdx, wdg, wds, bx, bg, bs = ref.scan_backward(c.flat(c.dy), wx, wg, f64(chunks), c.spans, c.start, f64(c.dfinal), **c.form,
                                                  coarse=c.coarse(saved))
    plain = kda.gated_scan_backward(dy, x, g, chunks, cu, initial_state=state, dfinal_state=dfinal, dg=like, **c.form)
    plain = [t.clone() for t in plain]
    for offset in (0, 1, 2, 3, 4):
        for which in ("dx", "dg", "ds", "chunks", "state", "dfinal", "all"):
            def at(name):
                return offset if which in (name, "all") else 0

            out = {"dx": boxed(plain[0], at("dx"), 3.0), "dg": boxed(plain[1], at("dg"), 3.0), "ds": boxed(plain[2], at("ds"), 3.0)}
            got = kda.gated_scan_backward(dy, x, g, boxed(chunks, at("chunks"))[1], cu, initial_state=boxed(state, at("state"))[1],
                                          dfinal_state=boxed(dfinal, at("dfinal"))[1], dx=out["dx"][1], dg=out["dg"][1],
                                          dinitial_state=out["ds"][1], **c.form)
            label = f"{shape} {offset} {which}"
            near(got[0], wdx, bx, f"{label} dx")
            near(got[1], wdg, bg, f"{label} dg")
            near(got[2], wds, bs, f"{label} dinitial")
            assert all(untouched(*b) for b in out.values()), label
            if offset % 2 == 0:
                assert all(torch.equal(a, b) for a, b in zip(got, plain)), label


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype, gdtype", TYPES)
def test_slices_of_wider_rows_at_whole_pieces(kda, shape, dtype, gdtype):  # noqa: F811
    """x, g and dy as slices of projections of several widths, at 16-byte boundaries: the bits of contiguous ones."""
    D, lens, packed = SHAPES[shape]
    c = Case(lens, D, dtype, gdtype, "log", False, packed=packed, seed=D)
    x, g, dy, cu, state, dfinal = (c.gpu(t) for t in (c.x, c.g, c.dy, c.cu, c.state, c.dfinal))
    chunks = torch.full((kda.gated_scan_chunks(*x.shape[:2]), D), 7.0, device=DEV)
    y, final, chunks = c.check(kda, shape)
    grads = kda.gated_scan_backward(dy, x, g, chunks, cu, initial_state=state, dfinal_state=dfinal, **c.form)

    def inside(t, before, behind):
        wide = torch.full((*t.shape[:2], before + D + behind), float("nan"), dtype=t.dtype, device=DEV)
        part = wide[..., before:before + D]
        part.copy_(t)
        return part

    for x_at, g_at, dy_at in (((0, 8), (8, 0), (16, 8)), ((2 * D, D), (D, 2 * D), (0, D)), ((8, 0), (0, 0), (0, 0)),
                              ((0, 0), (8, 64), (0, 0)), ((0, 0), (0, 0), (64, 8))):
        xs, gs, ds = inside(x, *x_at), inside(g, *g_at), inside(dy, *dy_at)
        again = torch.full_like(chunks, 7.0)
        got = kda.gated_scan(xs, gs, cu, initial_state=state, chunk_states=again, **c.form)
        assert torch.equal(got[0], y) and torch.equal(got[1], final) and torch.equal(again, chunks), (x_at, g_at)
        got = kda.gated_scan_backward(ds, xs, gs, chunks, cu, initial_state=state, dfinal_state=dfinal, **c.form)
        assert all(torch.equal(a, b) for a, b in zip(got, grads)), (x_at, g_at, dy_at)
        pool, want = state.clone(), state.clone()
        n = min(len(lens), xs.shape[1])
        token = kda.gated_step(xs[0, :n], gs[0, :n], pool[:n], **c.form)
        assert torch.equal(token, kda.gated_step(x[0, :n], g[0, :n], want[:n], **c.form)) and torch.equal(pool, want)
