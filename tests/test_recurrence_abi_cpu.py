"""The argument checks of the gated linear recurrence, the checkpoints and the norm's gradients on a
machine without a GPU: every refusal comes before any CUDA call, which would give KDA_ERR_CUDA here.

The addresses are made up, so every call here is refused or has nothing to do: one that nothing refuses would go on to a
launch, which would read and write them.  What is just allowed is called with real buffers in test_recurrence_edges_gpu.py."""
import pytest
import torch

import linear_attention_chunked_02_gb300 as kda
from linear_attention_chunked_02_gb300 import build as kbuild
from linear_attention_chunked_02_gb300 import recurrence

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a GPU is present, and a refusal that was lost would use made-up addresses")

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = [1 << (30 + i) for i in range(20)]                     # distinct, aligned, far apart


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kda.lib()


def scan(L, x=P[0], ldx=512, g=P[1], ldg=512, y=P[2], sin=None, sout=P[3], slots=None, nslots=0, chunk=P[4], cu=None,
         nseq=0, B=2, T=64, D=512, dt=1, gdt=1, decay=0, comp=0):
    return L.kda_gated_scan(x, ldx, g, ldg, y, sin, sout, slots, nslots, chunk, cu, nseq, B, T, D, dt, gdt, decay, comp, None)


def back(L, dy=P[0], lddy=512, x=P[1], xe=None, ldx=512, g=P[2], ge=None, ldg=512, chunk=P[3], sin=None, dout=None, dx=P[4],
         dg=P[5], din=None, cu=None, nseq=0, B=2, T=64, D=512, dt=1, gdt=1, decay=0, comp=0):
    return L.kda_gated_scan_backward(dy, lddy, x, xe, ldx, g, ge, ldg, chunk, sin, dout, dx, dg, din, cu, nseq, B, T, D, dt,
                                     gdt, decay, comp, None)


def step(L, x=P[0], ldx=512, g=P[1], ldg=512, y=P[2], state=P[3], slots=None, nslots=8, N=8, D=512, dt=1, gdt=1, decay=0,
         comp=0):
    return L.kda_gated_step(x, ldx, g, ldg, y, state, slots, nslots, N, D, dt, gdt, decay, comp, None)


def norm(L, dy=P[0], x=P[1], xe=None, z=P[2], ze=None, w=P[3], dx=P[4], dz=P[5], dw=P[6], rows=100, dim=128, eps=1e-6, act=0,
         dt=1, ws=P[7], wsb=1 << 30):
    return L.kda_gated_norm_backward(dy, x, xe, z, ze, w, dx, dz, dw, rows, dim, eps, act, dt, ws, wsb, None)


@pytest.mark.parametrize("call", [scan, back, step])
def test_forms_that_are_refused(L, call):
    for dt, gdt in ((3, 3), (-1, 0), (0, 1), (1, 2), (2, 1), (1, 3)):
        assert call(L, dt=dt, gdt=gdt) == UNSUPPORTED
    for decay in (-1, 2):
        assert call(L, decay=decay) == INVALID
    for comp in (-1, 2):
        assert call(L, comp=comp) == INVALID
    assert call(L, D=0) == INVALID and call(L, D=-4) == INVALID
    wide = {"ldx": 1 << 21, "ldg": 1 << 21, **({"lddy": 1 << 21} if call is back else {})}
    assert call(L, D=(1 << 20) + 1, **wide) == UNSUPPORTED


@pytest.mark.parametrize("call", [scan, back])
def test_streams_that_are_refused(L, call):
    assert call(L, B=-1) == INVALID and call(L, T=-1) == INVALID and call(L, nseq=-1) == INVALID
    assert call(L, cu=P[8], nseq=0) == INVALID and call(L, nseq=2) == INVALID
    assert call(L, cu=P[8], nseq=2, B=2) == INVALID and call(L, cu=P[8] + 2, nseq=2, B=1) == INVALID
    assert call(L, B=1 << 30, T=0) == UNSUPPORTED and call(L, B=1, T=(1 << 31) - (1 << 16)) == UNSUPPORTED
    assert call(L, B=1 << 16, T=1 << 15) == UNSUPPORTED and call(L, B=1, cu=P[8], nseq=1 << 30) == UNSUPPORTED
    assert call(L, B=0) == OK


def test_scan_refusals(L):
    for name in ("x", "g", "y"):
        assert scan(L, **{name: None}) == INVALID
        assert scan(L, **{name: P[9] + 1}) == INVALID
    for name in ("sin", "sout", "chunk", "slots"):
        assert scan(L, **{name: P[9] + 2}) == INVALID
    assert scan(L, g=P[9] + 2, gdt=0) == INVALID
    assert scan(L, ldx=511) == INVALID and scan(L, ldg=0) == INVALID
    assert scan(L, slots=P[9], nslots=-1) == INVALID
    # what is written may lie on nothing else, up to its last byte
    rows, row = 128, 512 * 2
    for name, other in (("y", P[0]), ("y", P[1]), ("chunk", P[0]), ("sout", P[0]), ("sout", P[2]), ("chunk", P[2]), ("chunk", P[3])):
        assert scan(L, **{name: other}) == INVALID, (name, other)
    assert scan(L, y=P[0] + rows * row - 2) == INVALID
    assert scan(L, x=P[0], ldx=1024, y=P[0] + rows * 2048 - 1024 - 2) == INVALID
    assert scan(L, sin=P[9], sout=P[9] + 4) == INVALID and scan(L, sin=P[9], y=P[9]) == INVALID
    assert scan(L, sin=P[9], chunk=P[9]) == INVALID
    assert scan(L, cu=P[9], nseq=3, B=1, sout=P[9]) == INVALID and scan(L, slots=P[9], nslots=9, y=P[9]) == INVALID
    assert scan(L, B=2, T=0, sout=None) == OK               # nothing to do


def test_backward_refusals(L):
    for name in ("dy", "x", "g", "chunk", "dx", "dg"):
        assert back(L, **{name: None}) == INVALID
        assert back(L, **{name: P[9] + 1}) == INVALID
    for name in ("sin", "dout", "din", "chunk"):
        assert back(L, **{name: P[9] + 2}) == INVALID
    for name in ("lddy", "ldx", "ldg"):
        assert back(L, **{name: 511}) == INVALID
    assert back(L, xe=P[9], ldx=513) == INVALID and back(L, ge=P[9], ldg=1024) == INVALID
    for out in ("dx", "dg", "din"):
        for at in (P[0], P[1], P[2], P[3]):
            assert back(L, **{out: at}) == INVALID
    assert back(L, dx=P[9], dg=P[9]) == INVALID and back(L, din=P[9], dout=P[9]) == INVALID
    assert back(L, din=P[9], sin=P[9]) == INVALID and back(L, xe=P[9], dx=P[9]) == INVALID
    assert back(L, ge=P[9], dg=P[9]) == INVALID
    assert back(L, T=0) == OK


def test_step_refusals(L):
    for name in ("x", "g", "y", "state"):
        assert step(L, **{name: None}) == INVALID
        assert step(L, **{name: P[9] + 1}) == INVALID
    assert step(L, slots=P[9] + 2) == INVALID
    assert step(L, N=-1) == INVALID and step(L, nslots=-1) == INVALID and step(L, nslots=7) == INVALID
    assert step(L, ldx=511) == INVALID and step(L, ldg=511) == INVALID
    assert step(L, N=1 << 30, nslots=1 << 30) == UNSUPPORTED
    for out in ("y", "state"):
        for at in (P[0], P[1]):
            assert step(L, **{out: at}) == INVALID
    assert step(L, y=P[3]) == INVALID and step(L, slots=P[9], y=P[9]) == INVALID and step(L, slots=P[9], state=P[9]) == INVALID
    assert step(L, N=0) == OK


def test_checkpoint_refusals(L):
    def save(x=P[0], ldx=100, codes=P[1], exps=P[2], rows=10, dim=100, dt=1):
        return L.kda_checkpoint_save(x, ldx, codes, exps, rows, dim, dt, None)

    def load(codes=P[1], exps=P[2], x=P[0], rows=10, dim=100, dt=1):
        return L.kda_checkpoint_load(codes, exps, x, rows, dim, dt, None)

    for call in (save, load):
        assert call(dt=3) == UNSUPPORTED and call(dim=(1 << 20) + 1) == UNSUPPORTED and call(rows=1 << 35) == UNSUPPORTED
        assert call(rows=-1) == INVALID and call(dim=0) == INVALID and call(rows=0) == OK
        for name in ("x", "codes", "exps"):
            assert call(**{name: None}) == INVALID
        assert call(x=P[9] + 1) == INVALID
        assert call(codes=P[0] + 10 * 200 - 1) == INVALID and call(exps=P[0]) == INVALID and call(codes=P[2]) == INVALID
    assert save(ldx=99) == INVALID


def test_norm_gradient_refusals(L):
    need = L.kda_gated_norm_backward_workspace_size(100, 128)
    assert need >= 128 * 4 and L.kda_gated_norm_backward_workspace_size(0, 128) == 0
    assert L.kda_gated_norm_backward_workspace_size(5, 0) == 0 and L.kda_gated_norm_backward_workspace_size(5, 16385) == 0
    for name in ("dy", "x", "z", "w", "dx", "dz", "dw"):
        assert norm(L, **{name: None}) == INVALID
        assert norm(L, **{name: P[9] + 1}) == INVALID
    assert norm(L, dt=3) == UNSUPPORTED and norm(L, dim=16385) == UNSUPPORTED and norm(L, rows=1 << 31) == UNSUPPORTED
    assert norm(L, rows=-1) == INVALID and norm(L, dim=0) == INVALID and norm(L, act=2) == INVALID
    assert norm(L, eps=-1.0) == INVALID and norm(L, eps=float("nan")) == INVALID
    assert norm(L, ws=None) == WORKSPACE and norm(L, wsb=need - 1) == WORKSPACE and norm(L, ws=P[9] + 4) == INVALID
    for out in ("dx", "dz", "dw", "ws"):
        for at in (P[0], P[1], P[2], P[3]):
            assert norm(L, **{out: at}) == INVALID, (out, at)
    for a, b in (("dx", "dz"), ("dx", "dw"), ("dz", "ws"), ("dw", "ws")):
        assert norm(L, **{a: P[9], b: P[9]}) == INVALID
    assert norm(L, xe=P[9], dx=P[9]) == INVALID and norm(L, ze=P[9], dz=P[9]) == INVALID


def test_python_refusals_without_a_gpu():
    x = torch.zeros(1, 4, 8)
    for call in (lambda: kda.gated_scan(x, x), lambda: kda.gated_step(x[0], x[0], x[0]), lambda: kda.checkpoint_save(x),
                 lambda: kda.gated_scan_backward(x, x, x, x[0]), lambda: kda.gated_norm_backward(x, x, x, x[0, 0])):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="unknown activation"):
        kda.gated_norm_backward(x, x, x, x[0, 0], activation="tanh")


def test_pitches():
    """Which layouts are read as they are, and at what pitch."""
    base = torch.zeros(4, 30, 140)
    for t, pitch in ((base, 140), (base[:, :, 3:69], 140), (base[1:2, :, 5:6], 140), (base[:, :1, :66], 30 * 140),
                     (base[:, ::2, :66], 280), (base[0], 140), (base[0, :, :7], 140), (base[0, 0], 140), (base[:0], 140)):
        got, at = recurrence._pitched(t)
        assert got is t and at == pitch, (t.shape, t.stride(), at)
    for t in (base.transpose(1, 2), base[:, :, ::2], base[:, :20, :66], base[:, :1].expand(4, 5, 140), base[:, ::7, :66],
              torch.zeros(140).expand(3, 5, 140)):
        got, at = recurrence._pitched(t)
        assert got.is_contiguous() and torch.equal(got, t) and at == t.shape[-1], (t.shape, t.stride())
