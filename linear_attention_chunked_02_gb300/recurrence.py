"""The gated linear recurrence, 8-bit checkpoints and the gated norm's gradients: binding of
include/kda_recurrent.h.

The block of a gated recurrent layer between its projections: ``gated_scan`` over whole sequences
or ``gated_step`` for one token of each running request, with ``gated_norm`` behind it.  Training
keeps the chunk states of ``gated_scan`` and the inputs, as they are or as ``checkpoint_save`` packs
them, and calls ``gated_norm_backward`` and ``gated_scan_backward``; no operator records gradients by itself.

With ``stream``, everything a call does happens on that stream, as for the operators in layer.py.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple, Union

import torch

from ._lib import DTYPE_CODE, check, lib
from .layer import ACT_CODE, _current_stream, _elsewhere, _int32, _on_gpu, _ptr

DECAY_CODE = {"log": 0, "sigmoid": 1}
SCAN_CHUNK = 64          # rows to a chunk state
CHECKPOINT_BLOCK = 32    # elements of a row that share an exponent


class Checkpoint(NamedTuple):
    """A tensor in 8 bits: the value of codes[.., i] is codes[.., i] * 2 ** (exponents[.., i // 32] - 127)."""
    codes: torch.Tensor        # int8, the tensor's shape
    exponents: torch.Tensor    # uint8, its last dimension divided by 32, rounded up


Saved = Union[torch.Tensor, Checkpoint]


def _form(gate: str, complement: bool) -> Tuple[int, int]:
    if gate not in DECAY_CODE:
        raise ValueError(f"unknown gate {gate!r}")
    return DECAY_CODE[gate], int(bool(complement))


def _pitched(t: torch.Tensor) -> Tuple[torch.Tensor, int]:
    """t, or a contiguous copy where its rows (all dimensions but the last) have no common pitch; the pitch."""
    width = t.shape[-1]
    if t.is_contiguous():
        return t, max(width, 1)
    if t.stride(-1) == 1 or width == 1:
        pitch, n = None, 1                                 # n rows so far, counted from the last dimension on
        for size, stride in zip(t.shape[-2::-1], t.stride()[-2::-1]):
            if size == 1:
                continue
            if pitch is None:
                pitch, n = stride, size
            elif stride == pitch * n:
                n *= size
            else:
                pitch = -1
                break
        if pitch is None or pitch >= width:
            return t, pitch or max(width, 1)
    return t.contiguous(), max(width, 1)


def _saved(name: str, t: Saved, shape, dtypes) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The tensor or the codes, and their exponents; checked against the shape and the types of a plain tensor."""
    if torch.is_tensor(t):
        if t.shape != shape or t.dtype not in dtypes:
            raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
        return t, None
    codes, exponents = t
    blocks = (*shape[:-1], -(-shape[-1] // CHECKPOINT_BLOCK))
    if codes.shape != shape or codes.dtype != torch.int8 or not codes.is_contiguous():
        raise ValueError(f"{name}'s codes must be contiguous int8 {tuple(shape)}, got {codes.dtype} {tuple(codes.shape)}")
    if exponents.numel() != _numel(blocks) or exponents.dtype != torch.uint8 or not exponents.is_contiguous():
        raise ValueError(f"{name}'s exponents must be contiguous uint8 {blocks}, got {exponents.dtype} {tuple(exponents.shape)}")
    return codes, exponents


def _numel(shape) -> int:
    n = 1
    for size in shape:
        n *= size
    return n


def _tensors(*saved):
    """The tensors of plain and checkpointed arguments, in pairs."""
    out = []
    for t in saved:
        out += [t, None] if t is None or torch.is_tensor(t) else list(t)
    return out


def _stream_rows(x: torch.Tensor, cu_seqlens: Optional[torch.Tensor]):
    """(B, T, D, sequences given by cu_seqlens, sequences) of a [B, T, D] tensor."""
    shape = x.shape
    if len(shape) != 3 or shape[2] < 1:
        raise ValueError(f"x must be [B, T, D], got {tuple(shape)}")
    B, T, D = shape
    if cu_seqlens is None:
        return B, T, D, 0, B
    nseq = _int32("cu_seqlens", cu_seqlens).numel() - 1
    if B != 1 or nseq < 1:
        raise ValueError("cu_seqlens needs B == 1 and at least one sequence")
    return B, T, D, nseq, nseq


def _states(name: str, t: torch.Tensor, entries: Optional[int], D: int) -> None:
    shape = t.shape
    if t.dtype != torch.float32 or len(shape) != 2 or shape[1] != D or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 [entries, {D}], got {t.dtype} {tuple(shape)}")
    if entries is not None and shape[0] != entries:
        raise ValueError(f"{name} must have {entries} entries, got {shape[0]}")


def _out(name: str, out: Optional[torch.Tensor], shape, dtype: torch.dtype, device) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if out.shape != shape or out.dtype != dtype or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    return out


def _types(x: torch.Tensor, g: torch.Tensor) -> Tuple[int, int]:
    xt, gt = x.dtype, g.dtype
    if xt not in DTYPE_CODE or (gt != xt and gt != torch.float32):
        raise ValueError(f"unsupported dtypes x {xt}, g {gt}")
    return DTYPE_CODE[xt], DTYPE_CODE[gt]


def _like(name: str, out: Optional[torch.Tensor], t: torch.Tensor) -> torch.Tensor:
    """_out for a tensor of t's shape and type."""
    if out is None and t.is_contiguous():
        return torch.empty_like(t)                         # the quickest way
    return _out(name, out, t.shape, t.dtype, t.device)


def gated_scan_chunks(B: int, T: int) -> int:
    """Rows of gated_scan's chunk_states for x [B, T, D]: one to 64 rows of the stream of B * T."""
    return -(-B * T // SCAN_CHUNK)


def gated_scan(x: torch.Tensor, g: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None, gate: str = "log",
               complement: bool = False, initial_state: Optional[torch.Tensor] = None,
               final_state: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
               chunk_states: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """h <- a h + c x over whole sequences, channel by channel; returns (y, final states), y the states h.

    x: [B, T, D] (float32 / bfloat16 / float16); g: [B, T, D] of x's dtype or float32.  a is
    exp(g) (gate "log": log decays, none positive) or sigmoid(g) ("sigmoid"); c is 1, or 1 - a
    with complement.  x and g may be slices of wider rows.  cu_seqlens: int32 CUDA tensor [N+1]
    for the packed layout (then B == 1).  initial_state, final_state, slots: as for delta_prefill,
    with states [N, D] or pools [entries, D].  chunk_states: float32 [gated_scan_chunks(B, T), D],
    written for gated_scan_backward.
    """
    device = _on_gpu("x g cu_seqlens initial_state final_state slots chunk_states out", x, g, cu_seqlens, initial_state,
                     final_state, slots, chunk_states, out)
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return gated_scan(x, g, cu_seqlens, gate, complement, initial_state, final_state, slots, chunk_states, out)
    decay, comp = _form(gate, complement)
    B, T, D, nseq, N = _stream_rows(x, cu_seqlens)
    xt, gt = _types(x, g)
    if g.shape != x.shape:
        raise ValueError(f"g must be {tuple(x.shape)}, got {tuple(g.shape)}")
    entries = N
    if slots is not None:
        slots = _int32("slots", slots, N).contiguous()
        if initial_state is None and final_state is None:
            raise ValueError("slots need a state pool")
        if final_state is None:
            final_state = initial_state
        entries = final_state.shape[0]
    if initial_state is not None:
        _states("initial_state", initial_state, entries, D)
    if final_state is None:
        final_state = torch.empty((N, D), dtype=torch.float32, device=x.device)
    elif final_state is not initial_state:
        _states("final_state", final_state, entries, D)
    if chunk_states is not None:
        _states("chunk_states", chunk_states, gated_scan_chunks(B, T), D)
    if cu_seqlens is not None:
        cu_seqlens = cu_seqlens.contiguous()
    out = _like("out", out, x)
    x, ldx = _pitched(x)
    g, ldg = _pitched(g)
    st = lib().kda_gated_scan(x.data_ptr(), ldx, g.data_ptr(), ldg, out.data_ptr(), _ptr(initial_state),
                              final_state.data_ptr(), _ptr(slots), entries, _ptr(chunk_states), _ptr(cu_seqlens), nseq,
                              B, T, D, xt, gt, decay, comp, _current_stream(device))
    check(st, "kda_gated_scan")
    return out, final_state


def gated_scan_backward(dy: torch.Tensor, x: Saved, g: Saved, chunk_states: torch.Tensor,
                        cu_seqlens: Optional[torch.Tensor] = None, gate: str = "log", complement: bool = False,
                        initial_state: Optional[torch.Tensor] = None, dfinal_state: Optional[torch.Tensor] = None,
                        dx: Optional[torch.Tensor] = None, dg: Optional[torch.Tensor] = None,
                        dinitial_state: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """The gradients of gated_scan; returns (dx, dg, dinitial_state).

    dy: [B, T, D], the gradient of y; dfinal_state: that of the final states, float32 [N, D] (zeros if
    not given).  x, g: as given to gated_scan, or checkpoints of them.  chunk_states: as gated_scan
    left them.  initial_state: float32 [N, D], what the sequences started from (with slots: the pool's
    entries before the call, in the sequences' order); zeros if not given, dinitial_state is then None unless given.
    dx is of dy's dtype; dg of g's, for a checkpoint of dy's, unless given (dy's dtype or float32).
    """
    device = _on_gpu("dy x x_exponents g g_exponents chunk_states cu_seqlens initial_state dfinal_state dx dg "
                     "dinitial_state", dy, *_tensors(x, g), chunk_states, cu_seqlens, initial_state, dfinal_state, dx, dg,
                     dinitial_state)
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return gated_scan_backward(dy, x, g, chunk_states, cu_seqlens, gate, complement, initial_state, dfinal_state,
                                       dx, dg, dinitial_state)
    decay, comp = _form(gate, complement)
    B, T, D, nseq, N = _stream_rows(dy, cu_seqlens)
    dt, f32 = dy.dtype, torch.float32
    if dt not in DTYPE_CODE:
        raise ValueError(f"unsupported dtype dy {dt}")
    x, xe = _saved("x", x, dy.shape, (dt,))
    g_dtypes = (dt,) if dt == f32 else (dt, f32)
    g, ge = _saved("g", g, dy.shape, g_dtypes)
    g_dtype = dg.dtype if dg is not None else dt if ge is not None else g.dtype
    if g_dtype not in g_dtypes or (ge is None and g_dtype != g.dtype):
        raise ValueError(f"unsupported dtypes dy {dt}, g {g.dtype}, dg {g_dtype}")
    _states("chunk_states", chunk_states, gated_scan_chunks(B, T), D)
    if initial_state is not None:
        _states("initial_state", initial_state, N, D)
    if dfinal_state is not None:
        _states("dfinal_state", dfinal_state, N, D)
    if dinitial_state is not None:
        _states("dinitial_state", dinitial_state, N, D)
    elif initial_state is not None:
        dinitial_state = torch.empty_like(initial_state)
    if cu_seqlens is not None:
        cu_seqlens = cu_seqlens.contiguous()
    dx = _like("dx", dx, dy)
    dg = _like("dg", dg, dy) if g_dtype == dt else _out("dg", dg, dy.shape, g_dtype, dy.device)
    dy, lddy = _pitched(dy)
    x, ldx = _pitched(x)
    g, ldg = _pitched(g)
    st = lib().kda_gated_scan_backward(dy.data_ptr(), lddy, x.data_ptr(), _ptr(xe), ldx, g.data_ptr(), _ptr(ge), ldg,
                                       chunk_states.data_ptr(), _ptr(initial_state), _ptr(dfinal_state), dx.data_ptr(),
                                       dg.data_ptr(), _ptr(dinitial_state), _ptr(cu_seqlens), nseq, B, T, D,
                                       DTYPE_CODE[dt], DTYPE_CODE[g_dtype], decay, comp, _current_stream(device))
    check(st, "kda_gated_scan_backward")
    return dx, dg, dinitial_state


def gated_step(x: torch.Tensor, g: torch.Tensor, state: torch.Tensor, slots: Optional[torch.Tensor] = None,
               gate: str = "log", complement: bool = False, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One token of each of N running requests; updates the states in place and returns y.

    x: [N, D]; g: [N, D] of x's dtype or float32; state: float32 pool [entries, D], of which request n
    uses entry slots[n] (int32 [N]), or n without slots.  A slot outside the pool (-1 for padding) reads
    zeros and stores nothing.
    """
    device = _on_gpu("x g state slots out", x, g, state, slots, out)
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return gated_step(x, g, state, slots, gate, complement, out)
    decay, comp = _form(gate, complement)
    shape = x.shape
    if len(shape) != 2 or shape[1] < 1 or g.shape != shape:
        raise ValueError(f"x and g must be [N, D], got {tuple(shape)} and {tuple(g.shape)}")
    xt, gt = _types(x, g)
    N, D = shape
    _states("state", state, None, D)
    entries = state.shape[0]
    if slots is not None:
        slots = _int32("slots", slots, N).contiguous()
    elif entries < N:
        raise ValueError(f"{N} requests and a pool of {entries} states")
    out = _like("out", out, x)
    x, ldx = _pitched(x)
    g, ldg = _pitched(g)
    st = lib().kda_gated_step(x.data_ptr(), ldx, g.data_ptr(), ldg, out.data_ptr(), state.data_ptr(), _ptr(slots),
                              entries, N, D, xt, gt, decay, comp, _current_stream(device))
    check(st, "kda_gated_step")
    return out


def checkpoint_save(x: torch.Tensor, out: Optional[Checkpoint] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> Checkpoint:
    """x [.., dim] in 8 bits, a power-of-two scale to 32 elements of a row; each value within 1 / 127 of the
    largest of its 32, or 2 ** -128 if that is more; 1 / 64 where the largest is so near its type's own that its
    code is cut.  A block with a NaN or an infinity reads back as NaN."""
    device = _on_gpu("x codes exponents", x, *(out if out is not None else ()))
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return checkpoint_save(x, out)
    if x.dim() < 1 or x.dtype not in DTYPE_CODE or x.shape[-1] < 1:
        raise ValueError(f"unsupported x {x.dtype} {tuple(x.shape)}")
    dim = x.shape[-1]
    blocks = (*x.shape[:-1], -(-dim // CHECKPOINT_BLOCK))
    codes = _out("codes", out.codes if out is not None else None, x.shape, torch.int8, x.device)
    exponents = _out("exponents", out.exponents if out is not None else None, blocks, torch.uint8, x.device)
    x, ldx = _pitched(x)
    st = lib().kda_checkpoint_save(x.data_ptr(), ldx, codes.data_ptr(), exponents.data_ptr(), x.numel() // dim, dim,
                                   DTYPE_CODE[x.dtype], _current_stream(device))
    check(st, "kda_checkpoint_save")
    return Checkpoint(codes, exponents)


def checkpoint_load(saved: Checkpoint, dtype: torch.dtype, out: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The values that a checkpoint stands for, in dtype; exact where dtype is the saved tensor's or float32."""
    device = _on_gpu("codes exponents out", *saved, out)
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return checkpoint_load(saved, dtype, out)
    if dtype not in DTYPE_CODE or saved.codes.dim() < 1 or saved.codes.shape[-1] < 1:
        raise ValueError(f"unsupported codes {tuple(saved.codes.shape)} or dtype {dtype}")
    codes, exponents = _saved("saved", saved, saved.codes.shape, ())
    dim = codes.shape[-1]
    out = _out("out", out, codes.shape, dtype, codes.device)
    st = lib().kda_checkpoint_load(codes.data_ptr(), exponents.data_ptr(), out.data_ptr(), codes.numel() // dim, dim,
                                   DTYPE_CODE[dtype], _current_stream(device))
    check(st, "kda_checkpoint_load")
    return out


def gated_norm_backward_workspace_size(rows: int, dim: int) -> int:
    """Bytes of workspace gated_norm_backward needs."""
    return int(lib().kda_gated_norm_backward_workspace_size(rows, dim))


def gated_norm_backward(dy: torch.Tensor, x: Saved, gate: Saved, weight: torch.Tensor, eps: float = 1e-6,
                        activation: str = "sigmoid", dx: Optional[torch.Tensor] = None,
                        dgate: Optional[torch.Tensor] = None, dweight: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """The gradients of gated_norm; returns (dx, dgate, dweight).

    dy: [.., dim], the gradient of gated_norm's result.  x, gate: as given to gated_norm, or checkpoints of them
    (saved in any shape whose rows are multiples of 32 and whose elements lie in the same order).
    weight: [dim] of dy's dtype.  dx and dgate are of dy's dtype, dweight float32.
    workspace: optional contiguous CUDA buffer of gated_norm_backward_workspace_size() bytes.
    """
    if activation not in ACT_CODE:
        raise ValueError(f"unknown activation {activation!r}")
    device = _on_gpu("dy x x_exponents gate gate_exponents weight dx dgate dweight workspace", dy, *_tensors(x, gate),
                     weight, dx, dgate, dweight, workspace)
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return gated_norm_backward(dy, x, gate, weight, eps, activation, dx, dgate, dweight, workspace)
    if dy.dim() < 1 or dy.dtype not in DTYPE_CODE or dy.shape[-1] < 1:
        raise ValueError(f"unsupported dy {dy.dtype} {tuple(dy.shape)}")
    dim = dy.shape[-1]
    rows = dy.numel() // dim
    if weight.dim() != 1 or weight.shape[0] != dim or weight.dtype != dy.dtype:
        raise ValueError(f"weight must be a {dy.dtype} [{dim}], got {weight.dtype} {tuple(weight.shape)}")
    x, xe = _saved("x", _reshaped(x, dy.shape), dy.shape, (dy.dtype,))
    gate, ze = _saved("gate", _reshaped(gate, dy.shape), dy.shape, (dy.dtype,))
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    dy, x, gate, weight = dy.contiguous(), x.contiguous(), gate.contiguous(), weight.contiguous()
    dx, dgate = _like("dx", dx, dy), _like("dgate", dgate, dy)
    dweight = _out("dweight", dweight, weight.shape, torch.float32, dy.device)
    need = gated_norm_backward_workspace_size(rows, dim)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dy.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().kda_gated_norm_backward(dy.data_ptr(), x.data_ptr(), _ptr(xe), gate.data_ptr(), _ptr(ze),
                                       weight.data_ptr(), dx.data_ptr(), dgate.data_ptr(), dweight.data_ptr(), rows, dim,
                                       eps, ACT_CODE[activation], DTYPE_CODE[dy.dtype], _ptr(workspace), ws_bytes,
                                       _current_stream(device))
    check(st, "kda_gated_norm_backward")
    return dx, dgate, dweight


def _reshaped(saved: Saved, shape) -> Saved:
    """A checkpoint of wider or narrower rows in this shape, where blocks of 32 stay what they are."""
    if torch.is_tensor(saved) or saved.codes.shape == shape or saved.codes.dim() < 1:
        return saved
    if saved.codes.numel() != _numel(shape) or saved.codes.shape[-1] % CHECKPOINT_BLOCK or shape[-1] % CHECKPOINT_BLOCK:
        return saved
    if not (saved.codes.is_contiguous() and saved.exponents.is_contiguous()):
        return saved
    return Checkpoint(saved.codes.view(shape), saved.exponents)
