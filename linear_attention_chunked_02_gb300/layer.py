"""The gated delta rule and the norms around it: binding of include/kda_layer.h.

A layer's operators between its projections, as a server runs them: ``add_norm``
before the block, ``delta_prefill`` over prompts or ``delta_step`` for one token of
each running request, ``gated_norm`` on the heads' outputs.  Inference only: no
operator records gradients.

With ``stream`` (one of the tensors' device), everything a call does (copies of tensors whose layout does not fit
and new outputs among it) happens on that stream; ordering it after the work that
produced the inputs, and the outputs' use on other streams, is the caller's.
"""
from __future__ import annotations

from typing import Optional

import torch

from ._lib import DTYPE_CODE, check, lib

WIDTHS = (32, 64, 96, 128)
ACT_CODE = {"sigmoid": 0, "silu": 1}


def _elsewhere(device: int, stream: Optional[torch.cuda.Stream]):
    """None where the call can run as it is; else the context in which it can: `stream`, or `device` made current."""
    if stream is not None:
        if stream.device_index != device:
            raise ValueError(f"stream is on cuda:{stream.device_index}, the tensors on cuda:{device}")
        return torch.cuda.stream(stream)
    return None if device == torch._C._cuda_getDevice() else torch.cuda.device(device)


def _current_stream(device: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device)


def _on_gpu(names: str, *tensors) -> int:
    """The device index of the tensors (named in `names`; None ones are skipped), which must be on one GPU."""
    device = tensors[0].get_device()                       # one integer a tensor; -1 on the CPU
    for t in tensors:
        if t is not None and (t.get_device() != device or not t.is_cuda):
            _refuse_devices(names, tensors)
    return device


def _refuse_devices(names: str, tensors) -> None:
    for name, t in zip(names.split(), tensors):
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
    for name, t in zip(names.split(), tensors):
        if t is not None and t.device != tensors[0].device:
            raise ValueError(f"{name} is on {t.device}, {names.split()[0]} on {tensors[0].device}")


def _ptr(t: Optional[torch.Tensor]):
    return t.data_ptr() if t is not None else None


def _aligned(t: torch.Tensor) -> torch.Tensor:
    """t itself, or a contiguous copy where its layout or address does not fit the kernels' vectors."""
    if not t.is_contiguous():
        t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


def _rule_shapes(q, k, v, g, beta, lead: int):
    """Checks of the token tensors, which have `lead` leading dimensions; (Hk, H, K, V, gate code)."""
    qs, vs, gs = q.shape, v.shape, g.shape
    if len(qs) != lead + 2 or len(vs) != lead + 2 or k.shape != qs or qs[:lead] != vs[:lead]:
        raise ValueError(f"shapes q {tuple(qs)}, k {tuple(k.shape)}, v {tuple(vs)} do not match")
    Hk, K = qs[-2:]
    H, V = vs[-2:]
    if K not in WIDTHS or V not in WIDTHS:
        raise ValueError(f"K and V must be among {WIDTHS}, got {K} and {V}")
    if Hk < 1 or H < 1 or H % Hk != 0:
        raise ValueError(f"{H} heads cannot share {Hk} key heads")
    heads = vs[:-1]
    if beta.shape != heads:
        raise ValueError(f"beta must be {tuple(heads)}, got {tuple(beta.shape)}")
    if len(gs) == lead + 2 and gs[:-1] == heads and gs[-1] == K:
        gate = 0
    elif gs == heads:
        gate = 1
    else:
        raise ValueError(f"g must be {tuple(heads)} or that with {K} channels, got {tuple(gs)}")
    dt = q.dtype
    if dt not in DTYPE_CODE or k.dtype != dt or v.dtype != dt or beta.dtype != dt or g.dtype != torch.float32:
        raise ValueError(f"unsupported dtypes q {q.dtype}, k {k.dtype}, v {v.dtype}, beta {beta.dtype}, g {g.dtype}")
    return Hk, H, K, V, gate


def _int32(name: str, t: Optional[torch.Tensor], numel: Optional[int] = None) -> Optional[torch.Tensor]:
    if t is None:
        return None
    if t.dtype != torch.int32 or t.dim() != 1 or (numel is not None and t.numel() != numel):
        raise ValueError(f"{name} must be a 1-D int32 CUDA tensor" + (f" of {numel}" if numel is not None else ""))
    return t


def _state(name: str, t: torch.Tensor, entries: Optional[int], H: int, K: int, V: int) -> None:
    if t.dtype != torch.float32 or t.shape[1:] != (H, K, V) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 [entries, {H}, {K}, {V}], got {t.dtype} {tuple(t.shape)}")
    if entries is not None and t.shape[0] != entries:
        raise ValueError(f"{name} must have {entries} entries, got {t.shape[0]}")


def _output(name: str, out: Optional[torch.Tensor], like: torch.Tensor) -> torch.Tensor:
    if out is None:
        return torch.empty_like(like)
    if out.shape != like.shape or out.dtype != like.dtype or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {like.dtype} tensor of shape {tuple(like.shape)}")
    return out


def delta_prefill_workspace_size(B: int, T: int, H: int, num_seqs: int = 0, K: int = 128, V: int = 128) -> int:
    """Bytes of workspace delta_prefill needs for this shape; enough for every smaller T too."""
    return int(lib().kda_delta_prefill_workspace_size(B, T, H, num_seqs, K, V))


def delta_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                  cu_seqlens: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                  initial_state: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
                  slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """The gated delta rule over whole sequences; returns (o, final states).

    q, k: [B, T, Hk, K]; v: [B, T, H, V], H a multiple of Hk; beta: [B, T, H], all of one
    dtype (float32 / bfloat16 / float16).  g: the tokens' log decays, float32, [B, T, H, K]
    or [B, T, H], none positive.  cu_seqlens: int32 CUDA tensor [N+1] for the packed layout
    (then B == 1).  scale: factor on the output, K ** -0.5 if not given.
    initial_state, final_state: float32 [N, H, K, V] (N = B for the dense layout); zeros and
    a new tensor if not given.  With slots (int32 [N]) both are pools of which sequence n
    uses entry slots[n], final_state is written in place and defaults to initial_state.
    workspace: optional contiguous CUDA buffer of delta_prefill_workspace_size() bytes.
    """
    device = _on_gpu("q k v g beta cu_seqlens initial_state final_state slots out workspace", q, k, v, g, beta,
                     cu_seqlens, initial_state, final_state, slots, out, workspace)
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return delta_prefill(q, k, v, g, beta, cu_seqlens, scale, initial_state, final_state, slots, out, workspace)
    Hk, H, K, V, gate = _rule_shapes(q, k, v, g, beta, 2)
    B, T = q.shape[:2]
    cu_seqlens = _int32("cu_seqlens", cu_seqlens)
    if cu_seqlens is not None and (B != 1 or cu_seqlens.numel() < 2):
        raise ValueError("cu_seqlens needs B == 1 and at least one sequence")
    nseq = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    N = nseq if cu_seqlens is not None else B
    slots = _int32("slots", slots, N)
    if slots is not None and initial_state is None and final_state is None:
        raise ValueError("slots need a state pool")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")   # its elements are counted as consecutive bytes
    if final_state is None and slots is not None:
        final_state = initial_state
    entries = N if slots is None else final_state.shape[0]
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        if t is not None:
            _state(name, t, entries, H, K, V)
    q, k, v, g, beta = _aligned(q), _aligned(k), _aligned(v), _aligned(g), _aligned(beta)
    slots = slots.contiguous() if slots is not None else None
    out = _output("out", out, v)
    cu_seqlens = cu_seqlens.contiguous() if cu_seqlens is not None else None
    if final_state is None:
        final_state = torch.empty((N, H, K, V), dtype=torch.float32, device=q.device)
    need = delta_prefill_workspace_size(B, T, H, nseq, K, V)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().kda_delta_prefill(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), out.data_ptr(),
        _ptr(initial_state), final_state.data_ptr(), _ptr(slots), entries, _ptr(cu_seqlens), nseq, B, T,
        Hk, H, K, V, DTYPE_CODE[q.dtype], gate, float(K ** -0.5 if scale is None else scale), _ptr(workspace), ws_bytes,
        _current_stream(device))
    check(st, "kda_delta_prefill")
    return out, final_state


def delta_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
               state: torch.Tensor, slots: Optional[torch.Tensor] = None, scale: Optional[float] = None,
               out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One token of each of N running requests; updates the states in place and returns o.

    q, k: [N, Hk, K]; v: [N, H, V]; beta: [N, H], of one dtype; g: float32 [N, H, K] or [N, H].
    state: float32 pool [entries, H, K, V]; request n uses entry slots[n] (int32 [N]), or n
    without slots.  A slot outside the pool (-1 for padding) reads zeros and stores nothing.
    """
    device = _on_gpu("q k v g beta state slots out", q, k, v, g, beta, state, slots, out)
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return delta_step(q, k, v, g, beta, state, slots, scale, out)
    Hk, H, K, V, gate = _rule_shapes(q, k, v, g, beta, 1)
    N = q.shape[0]
    slots = _int32("slots", slots, N)
    _state("state", state, None, H, K, V)
    if slots is None and state.shape[0] < N:
        raise ValueError(f"{N} requests and a pool of {state.shape[0]} states")
    q, k, v, g, beta = _aligned(q), _aligned(k), _aligned(v), _aligned(g), _aligned(beta)
    slots = slots.contiguous() if slots is not None else None
    out = _output("out", out, v)
    st = lib().kda_delta_step(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), out.data_ptr(), state.data_ptr(),
        _ptr(slots), state.shape[0], N, Hk, H, K, V, DTYPE_CODE[q.dtype], gate,
        float(K ** -0.5 if scale is None else scale), _current_stream(device))
    check(st, "kda_delta_step")
    return out


def _norm_shapes(x: torch.Tensor, weight: torch.Tensor, other: Optional[torch.Tensor], name: str) -> None:
    if x.dim() < 1 or x.dtype not in DTYPE_CODE:
        raise ValueError(f"unsupported x {x.dtype} {tuple(x.shape)}")
    if weight.dim() != 1 or weight.shape[0] != x.shape[-1] or weight.dtype != x.dtype:
        raise ValueError(f"weight must be a {x.dtype} [{x.shape[-1]}], got {weight.dtype} {tuple(weight.shape)}")
    if other is not None and (other.shape != x.shape or other.dtype != x.dtype):
        raise ValueError(f"{name} must match x, a {x.dtype} {tuple(x.shape)}; got {other.dtype} {tuple(other.shape)}")


def add_norm(x: torch.Tensor, residual: Optional[torch.Tensor], weight: torch.Tensor, eps: float = 1e-6,
             alpha: float = 1.0, out: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None):
    """r = residual + alpha x, y = r / sqrt(mean(r^2) + eps) * weight over the last dimension; returns (y, r).

    residual may be None (r = alpha x); residual_out may be residual and out may be x.
    """
    device = _on_gpu("x residual weight out residual_out", x, residual, weight, out, residual_out)
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return add_norm(x, residual, weight, eps, alpha, out, residual_out)
    _norm_shapes(x, weight, residual, "residual")
    dim = x.shape[-1]
    x, weight = x.contiguous(), weight.contiguous()
    residual = residual.contiguous() if residual is not None else None
    out, residual_out = _output("out", out, x), _output("residual_out", residual_out, x)
    st = lib().kda_add_norm(x.data_ptr(), _ptr(residual), weight.data_ptr(), out.data_ptr(),
                            residual_out.data_ptr(), x.numel() // dim if dim else 0, dim, alpha, eps,
                            DTYPE_CODE[x.dtype], _current_stream(device))
    check(st, "kda_add_norm")
    return out, residual_out


def gated_norm(x: torch.Tensor, gate: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
               activation: str = "sigmoid", out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """x / sqrt(mean(x^2) + eps) * weight * act(gate) over the last dimension; act is "sigmoid" or "silu".

    out may be x or gate.
    """
    if activation not in ACT_CODE:
        raise ValueError(f"unknown activation {activation!r}")
    device = _on_gpu("x gate weight out", x, gate, weight, out)
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return gated_norm(x, gate, weight, eps, activation, out)
    _norm_shapes(x, weight, gate, "gate")
    dim = x.shape[-1]
    x, gate, weight = x.contiguous(), gate.contiguous(), weight.contiguous()
    out = _output("out", out, x)
    st = lib().kda_gated_norm(x.data_ptr(), gate.data_ptr(), weight.data_ptr(), out.data_ptr(),
                              x.numel() // dim if dim else 0, dim, eps, ACT_CODE[activation], DTYPE_CODE[x.dtype],
                              _current_stream(device))
    check(st, "kda_gated_norm")
    return out
