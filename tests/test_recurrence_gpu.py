"""The gated linear recurrence, its gradients and its step, 8-bit checkpoints and the gated norm's
gradients against the 64-bit oracle on the same rounded inputs.

Tolerances: the oracle's bounds on what FP32 arithmetic may lose (oracle/recurrence.py says where they come from;
that of sigmoids of 16-bit arguments was derived when they took the faster exponential, after the first
run), plus half a unit in the last place of a 16-bit output's type where there is one (2^-8 and 2^-11 of the
value, half the least subnormal below the normal range).
Checkpoints are exact.  Norm gradients: sums over up to 16384 elements in a tree carry less than 32 * 2^-24
relative to the sum of absolute values, and there are two of them in dx beside some ten roundings and
functions of 2 units each: 2^-17 of the oracle's sums of absolute values.  dweight adds up
rows / 304 + 1 products in a thread at most, 256 threads' sums, 38 blocks' in each of 8 warps and those 8: for the rows below
less than 2^-24 (rows / 304 + 303) + 2^-19, taken as 2^-14 of the sum of absolute values.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.recurrence as ref

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
DTYPES = [F32, BF16, F16]
DEV = "cuda:0"


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_chunked_02_gb300 import build as kbuild
    kbuild.build()
    import linear_attention_chunked_02_gb300 as k
    yield k
    assert k.device_error(0) == 0


def f64(t):
    return t.to(torch.float64).cpu().numpy()


def rounding(value, dtype):
    """Half a unit in the last place of the type: what one rounding to it may add."""
    half = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}[dtype]
    least = {F32: 2.0 ** -150, BF16: 2.0 ** -134, F16: 2.0 ** -25}[dtype]
    return np.maximum(half * np.abs(value), least)


def near(got, want, bound, label):
    """got within bound of want, and of one rounding to its type; NaN in want: not looked at."""
    dtype, got = got.dtype, f64(got).reshape(want.shape)
    tol = bound + rounding(np.abs(want) + bound, dtype)
    bad = ~(np.abs(got - want) <= tol) & ~np.isnan(want)
    assert not bad.any(), (f"{label}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]}, allowed {tol[bad][0]}")


class Case:
    """Inputs in their types on the CPU, and the oracle's view of them."""

    def __init__(self, lens, D, dtype=F32, gdtype=None, gate="log", complement=False, packed=True, initial=True, seed=0,
                 before=0, after=0):
        rng = np.random.default_rng(seed)
        self.lens, self.D, self.dtype, self.gdtype = list(lens), D, dtype, gdtype or dtype
        self.form = {"gate": gate, "complement": complement}
        rows = sum(lens) + before + after
        ends = before + np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        self.spans = [(int(a), int(b)) for a, b in zip(ends[:-1], ends[1:])]
        self.cu = torch.tensor(ends.astype(np.int32)) if packed else None
        lead = (1, rows) if packed else (len(lens), lens[0] if lens else 0)

        def t(a, dt=dtype):
            return torch.from_numpy(np.ascontiguousarray(a)).to(dt).reshape(*lead, D)

        self.x, self.dy = t(rng.standard_normal((rows, D))), t(rng.standard_normal((rows, D)))
        g = rng.standard_normal((rows, D))
        if gate == "log":                                   # memories from a token to some hundred, by channel
            g = -(0.003 * 300 ** rng.uniform(size=D)) * np.logaddexp(0, g)
        else:
            g = g + 5 * rng.uniform(size=D)
        self.g = t(g, self.gdtype)
        self.state = torch.from_numpy(rng.standard_normal((len(lens), D))).to(F32) if initial else None
        self.dfinal = torch.from_numpy(rng.standard_normal((len(lens), D))).to(F32)
        self.start = f64(self.state) if initial else np.zeros((len(lens), D))

    def coarse(self, saved=False):
        """The largest argument where the sigmoid's faster form is taken (the oracle says what it costs)."""
        if self.form["gate"] != "sigmoid" or (self.gdtype == F32 and not saved):
            return 0
        g = np.abs(f64(self.g))
        return float(np.max(g[np.isfinite(g)], initial=0))

    def flat(self, t):
        return f64(t).reshape(-1, self.D)

    def want(self):
        return ref.scan(self.flat(self.x), self.flat(self.g), self.spans, self.start, **self.form, coarse=self.coarse())

    def gpu(self, t):
        return t.to(DEV) if t is not None else None

    def scan(self, kda, **kw):
        chunks = torch.full((kda.gated_scan_chunks(*self.x.shape[:2]), self.D), 7.0, device=DEV)
        kw = {"initial_state": self.gpu(self.state), "chunk_states": chunks, **kw}
        y, final = kda.gated_scan(self.gpu(self.x), self.gpu(self.g), self.gpu(self.cu), **self.form, **kw)
        return y, final, chunks

    def check(self, kda, label="", **kw):
        y, final, chunks = self.scan(kda, **kw)
        wy, wf, wc, by, bf, bc = self.want()
        near(y, wy, by, f"{label} y")
        near(final, wf, bf, f"{label} final")
        near(chunks, wc, bc, f"{label} chunk states")
        return y, final, chunks

    def check_backward(self, kda, save_x=False, save_g=False, with_final=True, dg=None, label=""):
        chunks = torch.from_numpy(np.nan_to_num(self.want()[2], nan=5.0)).to(F32)
        x, g = self.gpu(self.x), self.gpu(self.g)
        wx, wg = self.flat(self.x), self.flat(self.g)
        if save_x:
            x, wx = kda.checkpoint_save(x), ref.checkpoint(wx)[2]
        if save_g:
            g, wg = kda.checkpoint_save(g), ref.checkpoint(wg)[2]
        dfinal = self.dfinal if with_final else None
        out = kda.gated_scan_backward(self.gpu(self.dy), x, g, self.gpu(chunks), self.gpu(self.cu),
                                      initial_state=self.gpu(self.state), dfinal_state=self.gpu(dfinal), dg=dg, **self.form)
        *want, bx, bg, bs = ref.scan_backward(self.flat(self.dy), wx, wg, f64(chunks), self.spans, self.start,
                                              f64(self.dfinal) * with_final, **self.form, coarse=self.coarse(save_g))
        assert out[0].dtype == self.dtype and out[1].dtype == (self.gdtype if not save_g or dg is not None else self.dtype)
        near(out[0], want[0], bx, f"{label} dx")
        near(out[1], want[1], bg, f"{label} dg")
        if self.state is not None:
            near(out[2], want[2], bs, f"{label} dinitial")
        else:
            assert out[2] is None
        return out


LENS = {"one": [1], "chunk": [64], "past": [65], "singles": [1] * 5, "mixed": [0, 3, 0, 0, 70, 0, 129, 1], "long": [700],
        "many": [1] * 40 + [0] * 70 + [2] * 20 + [0] * 3, "edges": [64, 64, 1, 63, 128, 16, 8, 7, 9]}


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("dtype, gdtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
def test_scan_and_gradients_over_lengths(kda, lens, dtype, gdtype):
    for D, gate, complement in ((64, "log", False), (33, "sigmoid", True)):
        c = Case(LENS[lens], D, dtype, gdtype, gate, complement, seed=len(lens))
        c.check(kda, f"{lens} {D}")
        c.check_backward(kda, label=f"{lens} {D}")


@pytest.mark.parametrize("D", [1, 2, 31, 32, 63, 66, 128, 200, 2305])
@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("complement", [False, True])
def test_scan_and_gradients_over_widths(kda, D, gate, complement):
    c = Case([5, 130, 64], D, BF16, F32, gate, complement, seed=D)
    c.check(kda, str(D))
    c.check_backward(kda, label=str(D))


@pytest.mark.parametrize("B, T", [(1, 1), (3, 1), (1, 300), (4, 64), (5, 100), (2, 1000), (700, 3)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_dense(kda, B, T, dtype):
    for initial in (False, True):
        c = Case([T] * B, 70, dtype, packed=False, gate="sigmoid", complement=initial, initial=initial, seed=B)
        c.check(kda, f"{B}x{T}")
        c.check_backward(kda, label=f"{B}x{T}", with_final=initial)


@pytest.mark.parametrize("lens", [[20000], [9000, 1, 0, 5000, 3]], ids=str)
def test_long_sequences(kda, lens):
    c = Case(lens, 34, BF16, F32, "log", False, seed=3)
    c.check(kda, "long")
    c.check_backward(kda, label="long")
    c = Case(lens, 3, F32, F32, "sigmoid", True, seed=4)
    c.check(kda, "long")
    c.check_backward(kda, label="long")


def _many(n, longest, seed, zeros=0.1):
    rng = np.random.default_rng(seed)
    return [0 if rng.uniform() < zeros else int(rng.integers(1, longest + 1)) for _ in range(n)]


# Enough sequences that single warps walk them (8 bytes of x to a lane, or 4), alike or not; and one so long beside them that
# they are chained after all.
@pytest.mark.parametrize("dtype, gdtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16)])
@pytest.mark.parametrize("D, lens", [(512, _many(400, 12, 1)), (256, _many(300, 20, 2)), (136, [9] * 470), (512, [1] * 300 + [64] + [0] * 5),
                                     (512, [2] * 200 + [1500] + [3] * 250), (1024, _many(240, 9, 3, 0.5))], ids=lambda v: str(v)[:12])
def test_many_sequences(kda, dtype, gdtype, D, lens):
    for gate, complement in (("sigmoid", True), ("log", False), ("log", True)):
        c = Case(lens, D, dtype, gdtype, gate, complement, seed=D)
        c.check(kda, f"{D}")
    c.check_backward(kda, label=f"{D}")


# So many sequences that a block looks through their lengths for long, or (past 65536) does not: walked, or chained for a long one
# among them, by clusters or by parts alone.
@pytest.mark.parametrize("D, lens", [(64, _many(2600, 3, 5)), (32, [1] * 33000), (16, _many(70000, 1, 6, 0.5)),
                                     (64, [1] * 2500 + [1200] + [0] * 50 + [1] * 700), (40, [2] * 12000)], ids=lambda v: str(v)[:12])
def test_very_many_sequences(kda, D, lens):
    c = Case(lens, D, BF16, F32, "log", True, seed=D)
    c.check(kda, f"{D}")
    c.check_backward(kda, label=f"{D}")


@pytest.mark.parametrize("B, T, D", [(230, 9, 512), (460, 3, 256), (920, 2, 64), (40, 65, 2000), (2, 700, 64), (3, 1, 4096)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_dense_batches_of_whole_pieces(kda, B, T, D, dtype):
    c = Case([T] * B, D, dtype, packed=False, gate="sigmoid", complement=True, seed=B)
    c.check(kda, f"{B}x{T}x{D}")
    c.check_backward(kda, label=f"{B}x{T}x{D}")


# One sequence, or a few of any lengths, that the blocks of a cluster share tile by tile; parts of their own where they are alike.
@pytest.mark.parametrize("lens", [[9000], [3000, 1, 0, 2500, 700], [512] * 16, [64] * 90, [40] * 300, [1] * 70 + [4000]], ids=lambda v: str(v)[:14])
@pytest.mark.parametrize("dtype, gdtype", [(F32, F32), (BF16, BF16), (F16, F32)])
def test_clusters(kda, lens, dtype, gdtype):
    for D, gate, complement in ((64, "sigmoid", True), (72, "log", False)):
        c = Case(lens, D, dtype, gdtype, gate, complement, seed=len(lens))
        c.check(kda, f"{D}")
        c.check_backward(kda, label=f"{D}")
    c = Case(lens, 96, dtype, gdtype, "sigmoid", False, seed=5)
    c.check_backward(kda, True, True, dg=torch.empty(c.dy.shape, dtype=gdtype, device=DEV), label="codes")


def test_offsets_past_32_bits(kda):
    """More than 2^31 elements: the last rows and channels are those of a narrower tensor."""
    T, D, keep = 33000, 65600, 64
    x = torch.empty(1, T, D, dtype=BF16, device=DEV)
    g = torch.empty_like(x)
    small = [torch.randn(1, T, keep, device=DEV).to(BF16), (torch.randn(1, T, keep, device=DEV) + 2).to(BF16)]
    for big, part in zip((x, g), small):
        big.zero_()
        big[..., -keep:] = part
    form = {"gate": "sigmoid", "complement": True}
    chunks = torch.empty(kda.gated_scan_chunks(1, T), D, device=DEV)
    few = torch.empty(kda.gated_scan_chunks(1, T), keep, device=DEV)
    y, final = kda.gated_scan(x, g, chunk_states=chunks, **form)
    want, end = kda.gated_scan(*small, chunk_states=few, **form)
    # the same chains cut differently: both within the bound of the exact one, whose size is at most the values'
    assert torch.allclose(chunks[:, -keep:], few, rtol=1e-4, atol=1e-5) and torch.allclose(final[:, -keep:], end, rtol=1e-4, atol=1e-5)
    assert float((y[..., -keep:].float() - want.float()).abs().max()) <= 2.0 ** -7 * float(want.float().abs().max())
    sx = kda.checkpoint_save(x)
    assert torch.equal(sx.codes[..., -keep:], kda.checkpoint_save(small[0]).codes)
    assert torch.equal(kda.checkpoint_load(sx, BF16)[..., -keep:], kda.checkpoint_load(kda.checkpoint_save(small[0]), BF16))
    dx, dg, _ = kda.gated_scan_backward(y, sx, g, chunks, **form)
    wx, wg, _ = kda.gated_scan_backward(want, kda.checkpoint_save(small[0]), small[1], few, **form)
    for a, b in ((dx, wx), (dg, wg)):
        # inputs that differ by roundings of y, results by theirs: a few of 2^-8
        assert float((a[..., -keep:].float() - b.float()).abs().max()) <= 2.0 ** -6 * float(b.float().abs().max())


@pytest.mark.parametrize("save_x, save_g", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("dtype, gdtype", [(F32, F32), (BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("D", [31, 32, 33, 64, 98, 130, 240])
def test_gradients_from_checkpoints(kda, save_x, save_g, dtype, gdtype, D):
    c = Case([5, 0, 130, 64], D, dtype, gdtype, "sigmoid", True, seed=D)
    c.check_backward(kda, save_x, save_g, dg=torch.empty(c.dy.shape, dtype=gdtype, device=DEV))
    c = Case([77], D, dtype, gdtype, "log", False, initial=False, seed=D)
    c.check_backward(kda, save_x, save_g)


def test_rows_of_no_sequence_are_left_alone(kda):
    c = Case([70, 0, 3], 66, BF16, F32, before=9, after=150, seed=1)
    plain = c.check(kda, "outside")
    outside = [i for i in range(c.x.shape[1]) if not 9 <= i < 82]
    for value in (float("nan"), float("inf")):
        for t in (c.x, c.g, c.dy):
            t[0, outside] = value
        y = torch.full(c.x.shape, 3.0, dtype=BF16, device=DEV)
        got = c.scan(kda, out=y)
        assert (f64(y)[0, outside] == 3.0).all()
        assert torch.equal(y[0, 9:82], plain[0][0, 9:82]) and torch.equal(got[1], plain[1])
        assert (f64(got[2])[[0, 2, 3]] == 7.0).all() and torch.equal(got[2][1], plain[2][1])
        dx, dg = torch.full(c.x.shape, 3.0, dtype=BF16, device=DEV), torch.full(c.x.shape, 3.0, device=DEV)
        chunks = got[2].clone()
        chunks[[0, 2, 3]] = value
        out = kda.gated_scan_backward(c.gpu(c.dy), c.gpu(c.x), c.gpu(c.g), chunks, c.gpu(c.cu),
                                      initial_state=c.gpu(c.state), dfinal_state=c.gpu(c.dfinal), dx=dx, dg=dg, **c.form)
        assert (f64(dx)[0, outside] == 3.0).all() and (f64(dg)[0, outside] == 3.0).all()
        assert all(torch.isfinite(t[0, 9:82] if t.dim() == 3 else t).all() for t in out)


def test_nothing_leaks_between_sequences_and_channels(kda):
    c = Case([40, 50, 1, 200, 30], 66, F32, seed=2)
    y, final, chunks = c.scan(kda)
    grads = c.check_backward(kda)
    for value in (float("nan"), float("inf"), -float("inf")):
        bad = Case([40, 50, 1, 200, 30], 66, F32, seed=2)
        bad.x[0, 60, 5] = value                              # in the second sequence, its 21st token
        y2, final2, _ = bad.scan(kda)
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[0, 60:90, 5] = True
        assert torch.equal(y2[~hit], y[~hit]) and not torch.isfinite(y2[hit]).any()
        keep = torch.ones_like(final, dtype=torch.bool)
        keep[1, 5] = False
        assert torch.equal(final2[keep], final[keep])
        for n, name in enumerate(("x", "g", "dy")):
            bad = Case([40, 50, 1, 200, 30], 66, F32, seed=2)
            getattr(bad, name)[0, 60, 5] = value if name != "g" else float("nan")
            got = kda.gated_scan_backward(bad.gpu(bad.dy), bad.gpu(bad.x), bad.gpu(bad.g), chunks, bad.gpu(bad.cu),
                                          initial_state=bad.gpu(bad.state), dfinal_state=bad.gpu(bad.dfinal), **bad.form)
            hit = torch.zeros_like(y, dtype=torch.bool)
            hit[0, 40:90, 5] = True
            # the chunk states are those of the forward pass on finite inputs
            want = kda.gated_scan_backward(c.gpu(c.dy), c.gpu(c.x), c.gpu(c.g), chunks, c.gpu(c.cu),
                                           initial_state=c.gpu(c.state), dfinal_state=c.gpu(c.dfinal), **c.form)
            for a, b in zip(got[:2], want[:2]):
                assert torch.equal(a[~hit], b[~hit]), name
            assert torch.equal(got[2][keep], want[2][keep])
    assert torch.isfinite(grads[0]).all()


def test_decays_at_the_ends_of_their_range(kda):
    for gate, values in (("log", [0.0, -0.0, -1e-30, -100.0, -float("inf"), -3.0]),
                         ("sigmoid", [0.0, 40.0, -40.0, 100.0, -100.0, float("inf"), -float("inf")])):
        for complement in (False, True):
            c = Case([90, 33], 64, F32, F32, gate, complement, seed=7)
            c.g[0] = torch.tensor([values[i % len(values)] for i in range(123 * 64)]).reshape(123, 64)
            with np.errstate(invalid="ignore"):
                c.check(kda, f"{gate} {complement}")
                c.check_backward(kda, label=f"{gate} {complement}")
            if gate == "sigmoid":                           # the faster form of 16-bit arguments; rows of whole 16-byte pieces or not
                for D in (64, 63):
                    c = Case([90, 33], D, F16, F16, gate, complement, seed=8)
                    c.g[0] = torch.tensor([values[i % len(values)] for i in range(123 * D)]).reshape(123, D)
                    c.check(kda, f"{gate} {complement}")
                    c.check_backward(kda, label=f"{gate} {complement}")


def test_slots_and_states_in_place(kda):
    c = Case([5, 70, 0, 200, 1], 66, BF16, BF16, "sigmoid", True, seed=5)
    slots = torch.tensor([6, 2, 0, -1, 9], dtype=torch.int32, device=DEV)   # the fourth has none; 9 is past the pool
    pool = torch.from_numpy(np.random.default_rng(1).standard_normal((8, 66))).to(F32)
    for n, s in enumerate(slots.tolist()):
        c.start[n] = f64(pool[s]) if 0 <= s < 8 else 0.0
    wy, wf, _, by, bf, _ = c.want()
    before = pool.to(DEV)
    for in_place in (True, False):
        mine = before.clone()
        target = mine if in_place else torch.full_like(mine, 4.0)
        y, final = kda.gated_scan(c.gpu(c.x), c.gpu(c.g), c.gpu(c.cu), initial_state=mine,
                                  final_state=None if in_place else target, slots=slots, **c.form)
        near(y, wy, by, "y")
        assert final is target
        for n, s in enumerate(slots.tolist()):
            if 0 <= s < 8:
                near(final[s], wf[n], bf[n], f"state {n}")
        others = [i for i in range(8) if i not in slots.tolist()]
        assert torch.equal(target[others], before[others] if in_place else torch.full_like(target[others], 4.0))
    # in place without slots, repeated: the second call goes on from the first
    state = c.state.to(DEV)
    first = kda.gated_scan(c.gpu(c.x), c.gpu(c.g), c.gpu(c.cu), initial_state=state, final_state=state, **c.form)[1]
    c.start = f64(first)
    wy, wf, _, by, bf, _ = c.want()
    y, final = kda.gated_scan(c.gpu(c.x), c.gpu(c.g), c.gpu(c.cu), initial_state=state, final_state=state, **c.form)
    near(y, wy, by, "y again")
    near(final, wf, bf, "state again")


def test_empty_batches(kda):
    for x in (torch.empty(2, 0, 5, device=DEV), torch.empty(0, 7, 5, device=DEV)):
        state = torch.ones(x.shape[0], 5, device=DEV)
        y, final = kda.gated_scan(x, x, initial_state=state)
        assert y.shape == x.shape and torch.equal(final, state)
        assert torch.equal(kda.gated_scan(x, x)[1], torch.zeros_like(state))
        chunks = torch.empty(0, 5, device=DEV)
        dx, dg, ds = kda.gated_scan_backward(x, x, x, chunks, initial_state=state, dfinal_state=2 * state)
        assert dx.shape == x.shape and torch.equal(ds, 2 * state)
        assert torch.equal(kda.gated_scan_backward(x, x, x, chunks, initial_state=state)[2], torch.zeros_like(state))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_pitches_and_alignment(kda, dtype):
    c = Case([5, 130, 64], 66, dtype, dtype, "sigmoid", True, seed=8)
    rows = c.x.shape[1]
    y, final, chunks = c.check(kda)
    grads = c.check_backward(kda)
    x, g, dy = c.gpu(c.x), c.gpu(c.g), c.gpu(c.dy)
    cu, state, dfinal = c.gpu(c.cu), c.gpu(c.state), c.gpu(c.dfinal)
    for offset, pitch in ((0, 200), (66, 200), (67, 199), (1, 301)):
        wide = [torch.randn(1, rows, pitch + 200, dtype=dtype, device=DEV)[:, :, :pitch] for _ in range(3)]
        for w, t in zip(wide, (x, g, dy)):
            w[:, :, offset:offset + 66] = t
        xs, gs, ds = (w[:, :, offset:offset + 66] for w in wide)
        y2, final2 = kda.gated_scan(xs, gs, cu, initial_state=state, **c.form)
        assert torch.equal(y2, y) and torch.equal(final2, final), (offset, pitch)
        got = kda.gated_scan_backward(ds, xs, gs, f32(chunks), cu, initial_state=state, dfinal_state=dfinal, **c.form)
        want = kda.gated_scan_backward(dy, x, g, f32(chunks), cu, initial_state=state, dfinal_state=dfinal, **c.form)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (offset, pitch)
        step = kda.gated_step(xs[0, :3], gs[0, :3], state.clone(), **c.form)
        assert torch.equal(step, kda.gated_step(x[0, :3], g[0, :3], state.clone(), **c.form))
    # transposed, expanded and reversed layouts are copied
    odd = x.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(kda.gated_scan(odd, g, cu, initial_state=state, **c.form)[0], y)
    one = x[:, :1].expand(-1, rows, -1)
    assert torch.equal(kda.gated_scan(one, g, cu, **c.form)[0], kda.gated_scan(one.contiguous(), g, cu, **c.form)[0])
    assert grads[0].shape == x.shape
    dense = torch.randn(4, 30, 140, dtype=dtype, device=DEV)[:, :, 3:69]
    a = -dense.float().abs().to(dtype)
    assert torch.equal(kda.gated_scan(dense, a)[0], kda.gated_scan(dense.contiguous(), a)[0])


def f32(t):
    return t.to(F32)


@pytest.mark.parametrize("cu", [[0, 500, 100, 300], [-7, 50, 90, 100], [0, 40, 1 << 30, 130], [90, 60, 30, 0],
                                [5, 5, 5, 5], [200, 300, 400, 500], [0] * 40 + [10] + [0] * 40 + [130], [-5, -4, -3, -2]], ids=str)
def test_malformed_cu_seqlens_stay_inside_the_buffers(kda, cu):
    """Every index is clamped whatever the list holds; the results of such calls mean nothing."""
    rows, D, n = 130, 66, len(cu) - 1
    guard = 4096

    def boxed(rows, dtype=F32):
        t = torch.full((guard * 2 + rows * D,), 5.0, dtype=dtype, device=DEV)
        return t, t[guard:guard + rows * D].view(1, rows, D)

    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    x, g = torch.randn(1, rows, D, device=DEV), -torch.rand(1, rows, D, device=DEV)
    state = torch.randn(n, D, device=DEV)
    (yb, y), (cb, chunks), (sb, final) = boxed(rows), boxed(3), boxed(n)
    kda.gated_scan(x, g, cu, initial_state=state, final_state=final[0], chunk_states=chunks[0], out=y)
    (xb, dx), (gb, dg), (ib, ds) = boxed(rows), boxed(rows), boxed(n)
    kda.gated_scan_backward(x, x, g, torch.randn(3, D, device=DEV), cu, initial_state=state, dfinal_state=state, dx=dx,
                            dg=dg, dinitial_state=ds[0])
    torch.cuda.synchronize()
    for whole in (yb, cb, sb, xb, gb, ib):
        assert (whole[:guard] == 5.0).all() and (whole[-guard:] == 5.0).all()


@pytest.mark.parametrize("dtype, gdtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16)])
@pytest.mark.parametrize("N, D", [(1, 1), (1, 64), (3, 33), (7, 2305), (40, 512)])
def test_step(kda, dtype, gdtype, N, D):
    for gate, complement in (("log", False), ("log", True), ("sigmoid", False), ("sigmoid", True)):
        c = Case([1] * N, D, dtype, gdtype, gate, complement, seed=N)
        pool = torch.from_numpy(np.random.default_rng(N).standard_normal((N + 3, D))).to(F32)
        slots = torch.from_numpy(np.random.default_rng(D).permutation(N + 3)[:N].astype(np.int32))
        if N > 2:
            slots[1], slots[2] = -1, N + 3
        for n, s in enumerate(slots.tolist()):
            c.start[n] = f64(pool[s]) if 0 <= s < N + 3 else 0.0
        wy, wf, _, by, bf, _ = c.want()
        mine = pool.to(DEV)
        y = kda.gated_step(c.gpu(c.x)[0], c.gpu(c.g)[0], mine, slots=slots.to(DEV), gate=gate, complement=complement)
        near(y, wy, by, "step")
        used = [s for s in slots.tolist() if 0 <= s < N + 3]
        for n, s in enumerate(slots.tolist()):
            if s in used:
                near(mine[s], wf[n], bf[n], "state")
        others = [i for i in range(N + 3) if i not in used]
        assert torch.equal(mine[others].cpu(), pool[others])


@pytest.mark.parametrize("dtype, gdtype", [(F32, F32), (BF16, F32), (F16, F16)])
@pytest.mark.parametrize("N, D", [(2, 127), (2, 254), (3, 258), (2, 512), (3, 516), (2, 1020), (5, 1028), (3, 2306), (2, 4100)])
def test_step_widths(kda, dtype, gdtype, N, D):
    """Widths at which a request's last block has one vector to a thread, part of one, or none for most; the same bits
    from rows at other addresses, which go by smaller vectors."""
    c = Case([1] * N, D, dtype, gdtype, "sigmoid" if D % 4 else "log", D % 4 == 2, seed=D)
    wy, wf, _, by, bf, _ = c.want()
    pool = torch.full((N + 1, D), 3.0, device=DEV)
    pool[:N] = torch.from_numpy(c.start).to(F32)
    x, g = c.gpu(c.x)[0], c.gpu(c.g)[0]
    first = pool.clone()
    y = kda.gated_step(x, g, first, **c.form)
    near(y, wy, by, "step")
    near(first[:N], wf, bf, "states")
    assert (first[N] == 3.0).all()
    for offset in (1, 2, 4):
        wide = torch.zeros(N, D + 12, dtype=dtype, device=DEV)
        wide[:, offset:offset + D] = x
        again = pool.clone()
        assert torch.equal(kda.gated_step(wide[:, offset:offset + D], g, again, **c.form), y) and torch.equal(again, first)


def test_steps_go_on_from_a_scan(kda):
    """Prompts, then tokens one by one, as the same tokens in one scan."""
    lens, more, D = [70, 1, 33], 5, 66
    whole = Case([n + more for n in lens], D, BF16, F32, "log", False, initial=False, seed=11)
    wy, wf, _, by, bf, _ = whole.want()
    head = torch.cat([whole.x[0, a:b - more] for a, b in whole.spans])[None]
    gates = torch.cat([whole.g[0, a:b - more] for a, b in whole.spans])[None]
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    pool = torch.zeros(5, D, device=DEV)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    kda.gated_scan(head.to(DEV), gates.to(DEV), cu.to(DEV), initial_state=pool, slots=slots)
    for k in range(more):
        at = [b - more + k for _, b in whole.spans]
        y = kda.gated_step(whole.x[0, at].to(DEV), whole.g[0, at].to(DEV), pool, slots=slots)
        near(y, wy[at], by[at], f"token {k}")
    near(pool[slots.long()], wf, bf, "states")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows, dim", [(1, 1), (3, 31), (5, 32), (7, 33), (2, 64), (9, 128), (4, 2305), (3, 4096)])
def test_checkpoints_are_exact(kda, dtype, rows, dim):
    rng = np.random.default_rng(rows)
    x = rng.standard_normal((rows, dim)) * 10.0 ** rng.uniform(-3, 3, (rows, dim))
    x[rng.uniform(size=x.shape) < 0.1] = 0.0
    x[-1, : dim // 2] = 0.0
    x = torch.from_numpy(x).to(dtype)
    codes, exps, values = ref.checkpoint(f64(x))
    saved = kda.checkpoint_save(x.to(DEV))
    assert (f64(saved.codes) == codes).all() and (f64(saved.exponents) == exps).all()
    for to in DTYPES:
        got = kda.checkpoint_load(saved, to)
        assert got.dtype == to and torch.equal(got.cpu(), torch.from_numpy(values).to(to))
    assert torch.equal(kda.checkpoint_load(saved, dtype).cpu().double(), torch.from_numpy(values))
    wide = torch.randn(rows, 2 * dim + 3, device=DEV).to(dtype)
    wide[:, 1:dim + 1] = x.to(DEV)
    again = kda.checkpoint_save(wide[:, 1:dim + 1])
    assert torch.equal(again.codes, saved.codes) and torch.equal(again.exponents, saved.exponents)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows, dim", [(3, 255), (2, 256), (5, 257), (4, 289), (300, 515), (3, 1000), (2, 4100), (9000, 40)])
def test_checkpoints_of_unaligned_rows(kda, dtype, rows, dim):
    """Rows at odd addresses and of odd widths, into buffers whose neighbours stay as they are."""
    rng = np.random.default_rng(dim)
    x = torch.from_numpy(rng.standard_normal((rows, dim)) * 10.0 ** rng.uniform(-3, 3, (rows, dim))).to(dtype)
    codes, exps, values = ref.checkpoint(f64(x))
    wide = torch.zeros(rows, dim + 2, dtype=dtype, device=DEV)
    wide[:, 1:dim + 1] = x.to(DEV)
    blocks = -(-dim // 32)
    cbox = torch.full((rows * dim + 2,), 99, dtype=torch.int8, device=DEV)
    ebox = torch.full((rows * blocks + 2,), 99, dtype=torch.uint8, device=DEV)
    saved = kda.Checkpoint(cbox[1:-1].view(rows, dim), ebox[1:-1].view(rows, blocks))
    kda.checkpoint_save(wide[:, 1:dim + 1], out=saved)
    assert (f64(saved.codes) == codes).all() and (f64(saved.exponents) == exps).all()
    box = torch.full((rows * dim + 2,), 5.0, dtype=dtype, device=DEV)
    kda.checkpoint_load(saved, dtype, out=box[1:-1].view(rows, dim))
    assert (f64(box[1:-1]) == values.reshape(-1)).all()
    assert all(b[0] == v and b[-1] == v for b, v in ((cbox, 99), (ebox, 99), (box, 5.0)))


def test_checkpoints_of_special_values(kda):
    tiny = [2.0 ** -149, -(2.0 ** -140), 2.0 ** -127, 127 * 2.0 ** -127, 127.5 * 2.0 ** -127, 2.0 ** -126, 1e-38, 3e-36]
    large = [3.4e38, 2.0 ** 127, -3.4028235e38, 127 * 2.0 ** 120, 127.5 * 2.0 ** 120]
    edges = [127.0, 127.00001, 126.5, 125.5, 63.5, 254.0, 253.0, 1.9843750, 1.9843751]
    rows = []
    for v in tiny + large + edges:
        rows.append([v, v / 2, -v / 3, 0.0, v / 127, v * 0.996] + [0.0] * 26)
    x = torch.tensor(rows, dtype=torch.float64).to(F32)
    codes, exps, values = ref.checkpoint(f64(x))
    saved = kda.checkpoint_save(x.to(DEV))
    assert (f64(saved.codes) == codes).all() and (f64(saved.exponents) == exps).all()
    assert (f64(kda.checkpoint_load(saved, F32)) == values).all()
    for dtype in DTYPES:
        x = torch.randn(3, 70, device=DEV).to(dtype)
        x[0, 3], x[1, 40], x[2, 69] = float("nan"), float("inf"), -float("inf")
        got = kda.checkpoint_load(kda.checkpoint_save(x), dtype)
        bad = torch.zeros(3, 70, dtype=torch.bool, device=DEV)
        bad[0, :32] = bad[1, 32:64] = bad[2, 64:] = True
        assert torch.isnan(got[bad]).all() and torch.isfinite(got[~bad]).all()
    for dtype in DTYPES:                                    # the type's largest values stay finite
        top = torch.finfo(dtype).max
        x = torch.tensor([[top, -top, top / 2, top / 128], [top * 0.99, -top * 0.995, 1.0, 0.0]]).to(dtype)
        got = kda.checkpoint_load(kda.checkpoint_save(x.to(DEV)), dtype)
        assert (f64(got) == ref.checkpoint(f64(x), top)[2]).all() and torch.isfinite(got).all()
    x = (torch.arange(1, 65, device=DEV).reshape(2, 32) * 2.0 ** -24).to(F16)       # subnormals
    assert torch.equal(kda.checkpoint_load(kda.checkpoint_save(x), F16), x)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows, dim", [(1, 1), (5, 7), (3, 32), (700, 64), (33, 96), (2000, 128), (9, 200), (40, 512), (3, 513),
                                       (5, 520), (70, 2305), (3, 4096), (2, 16384), (1, 16383)])
def test_norm_gradients(kda, dtype, rows, dim):
    rng = np.random.default_rng(dim)
    x, z, dy = (torch.from_numpy(s * rng.standard_normal((rows, dim))).to(dtype) for s in (0.3, 2.0, 1.0))
    w = torch.from_numpy(1 + 0.1 * rng.standard_normal(dim)).to(dtype)
    for act, save in (("sigmoid", (0, 0)), ("silu", (0, 0)), ("silu", (1, 1)), ("sigmoid", (1, 0)), ("silu", (0, 1))):
        gx, gz, wx, wz = x.to(DEV), z.to(DEV), f64(x), f64(z)
        if save[0]:
            gx, wx = kda.checkpoint_save(gx), ref.checkpoint(wx)[2]
        if save[1]:
            gz, wz = kda.checkpoint_save(gz), ref.checkpoint(wz)[2]
        got = kda.gated_norm_backward(dy.to(DEV), gx, gz, w.to(DEV), eps=1e-5, activation=act)
        dx, dz, dw, sx, sz, sw = ref.gated_norm_backward(f64(dy), wx, wz, f64(w), 1e-5, act)
        assert got[0].dtype == dtype and got[1].dtype == dtype and got[2].dtype == F32
        near(got[0], dx, 2.0 ** -17 * sx, f"dx {act} {save}")
        near(got[1], dz, 2.0 ** -17 * sz, f"dgate {act} {save}")
        near(got[2], dw, 2.0 ** -14 * sw, f"dweight {act} {save}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows, dim", [(1300, 130), (1300, 264), (611, 257), (700, 768), (650, 1024), (620, 2048), (320, 2049),
                                       (610, 2056), (500, 2304), (330, 4096), (306, 4097), (310, 4104), (305, 8192), (4, 8200)])
def test_norm_gradients_of_rows_of_several_warps(kda, dtype, rows, dim):
    """Teams of threads of every size, with more rows than teams; a NaN stays in its row, but for dweight."""
    rng = np.random.default_rng(rows + dim)
    x, z, dy = (torch.from_numpy(s * rng.standard_normal((rows, dim), np.float32)).to(dtype) for s in (0.3, 2.0, 1.0))
    w = torch.from_numpy(1 + 0.1 * rng.standard_normal(dim)).to(dtype)
    for act, saved in (("sigmoid", False), ("silu", True)):
        gx, gz, wx, wz = x.to(DEV), z.to(DEV), f64(x), f64(z)
        if saved:
            gx, gz, wx, wz = kda.checkpoint_save(gx), kda.checkpoint_save(gz), ref.checkpoint(wx)[2], ref.checkpoint(wz)[2]
        got = kda.gated_norm_backward(dy.to(DEV), gx, gz, w.to(DEV), eps=1e-5, activation=act)
        dx, dz, dw, sx, sz, sw = ref.gated_norm_backward(f64(dy), wx, wz, f64(w), 1e-5, act)
        near(got[0], dx, 2.0 ** -17 * sx, f"dx {act}")
        near(got[1], dz, 2.0 ** -17 * sz, f"dgate {act}")
        near(got[2], dw, 2.0 ** -14 * sw, f"dweight {act}")
        bad = dy.to(DEV)
        bad[rows // 2, dim - 1] = float("nan")
        again = kda.gated_norm_backward(bad, gx, gz, w.to(DEV), eps=1e-5, activation=act)
        others = [r for r in range(rows) if r != rows // 2]
        assert all(torch.equal(a[others], b[others]) for a, b in zip(again[:2], got[:2]))
        assert again[0][rows // 2].isnan().all() and again[2][dim - 1].isnan() and not again[2][:dim - 1].isnan().any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [10240, 12161, 12200, 12288, 12320])
def test_norm_gradients_of_the_widest_rows(kda, dtype, dim):
    """Widths whose sums of dweight fill what shared memory a kernel has without asking for more."""
    rng = np.random.default_rng(dim)
    x, z, dy = (torch.from_numpy(s * rng.standard_normal((3, dim), np.float32)).to(dtype) for s in (0.3, 2.0, 1.0))
    w = torch.from_numpy(1 + 0.1 * rng.standard_normal(dim)).to(dtype)
    got = kda.gated_norm_backward(dy.to(DEV), x.to(DEV), z.to(DEV), w.to(DEV), eps=1e-5)
    dx, dz, dw, sx, sz, sw = ref.gated_norm_backward(f64(dy), f64(x), f64(z), f64(w), 1e-5, "sigmoid")
    near(got[0], dx, 2.0 ** -17 * sx, "dx")
    near(got[1], dz, 2.0 ** -17 * sz, "dgate")
    near(got[2], dw, 2.0 ** -14 * sw, "dweight")


def test_norm_gradients_of_many_rows_and_heads(kda):
    """Heads' rows whose checkpoints were taken of whole tokens; layouts that need copies; no rows."""
    gen = torch.Generator(device=DEV).manual_seed(0)
    x, z, dy = (torch.randn(300, 5, 64, generator=gen, device=DEV).to(BF16) for _ in range(3))
    w = torch.ones(64, dtype=BF16, device=DEV)
    cx, cz = kda.checkpoint_save(x.view(300, 320)), kda.checkpoint_save(z)
    a = kda.gated_norm_backward(dy, cx, cz, w)
    b = kda.gated_norm_backward(dy, kda.checkpoint_load(cx, BF16).view(300, 5, 64), kda.checkpoint_load(cz, BF16), w)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    plain = kda.gated_norm_backward(dy, x, z, w)
    odd = [torch.randn(300, 5, 67, device=DEV).to(BF16)[..., 1:65] for _ in range(3)]
    for o, t in zip(odd, (dy, x, z)):
        o.copy_(t)
    assert all(torch.equal(s, t) for s, t in zip(kda.gated_norm_backward(*odd, w), plain))
    e = torch.empty(0, 64, dtype=BF16, device=DEV)
    out = kda.gated_norm_backward(e, e, e, w, dweight=torch.ones(64, device=DEV))
    assert (out[2] == 0).all() and out[0].shape == e.shape


def test_repeats_streams_and_graphs_give_the_same_bits(kda):
    c = Case([300, 0, 1, 77, 130], 130, BF16, BF16, "sigmoid", True, seed=9)
    x, g, dy, cu, state, dfinal = (c.gpu(t) for t in (c.x, c.g, c.dy, c.cu, c.state, c.dfinal))
    w = torch.ones(130, dtype=BF16, device=DEV)
    chunks = torch.empty(kda.gated_scan_chunks(*x.shape[:2]), 130, device=DEV)
    pool, slots = torch.randn(4, 130, device=DEV), torch.tensor([3, 1], dtype=torch.int32, device=DEV)
    kept = pool.clone()

    def layer(stream=None):
        """All of the operators, as a training step and a decoding step would use them."""
        pool.copy_(kept) if stream is None else None
        y, final = kda.gated_scan(x, g, cu, initial_state=state, chunk_states=chunks, stream=stream, **c.form)
        sx, sg, sy = (kda.checkpoint_save(t, stream=stream) for t in (x, g, y))
        dh, dz, dw = kda.gated_norm_backward(dy, sy, sg, w, stream=stream)
        grads = kda.gated_scan_backward(dh, sx, sg, chunks, cu, initial_state=state, dfinal_state=dfinal, stream=stream,
                                        **c.form)
        step = kda.gated_step(x[0, :2], g[0, :2], pool, slots=slots, stream=stream, **c.form)
        return [y, final, dz, dw, *grads, step, kda.checkpoint_load(sy, BF16, stream=stream)]

    want = [t.clone() for t in layer()]
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(layer(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pool.copy_(kept)
    torch.cuda.synchronize()
    got = layer(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # two graphs of the same calls, replayed in turn
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer()
        graphs.append((graph, out))
    x0 = x.clone()
    for graph, out in graphs * 3:
        x.copy_(x0)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    x.mul_(2)
    graphs[0][0].replay()
    fresh = layer()
    assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], fresh))


def test_a_training_block_against_autograd(kda):
    """Scan, gated norm and a product with a weight, forwards and backwards, as a layer uses them: the
    gradients are those that automatic differentiation of the definitions gives in 64 bits."""
    N, T, H, W = 2, 70, 3, 32
    gen = torch.Generator().manual_seed(3)
    x, g, z = (torch.randn(N, T, H * W, generator=gen) for _ in range(3))
    w, dy = 1 + 0.1 * torch.randn(W, generator=gen), torch.randn(N, T, H, W, generator=gen)
    leaves = [t.double().requires_grad_() for t in (x, g, z, w)]
    a = torch.sigmoid(leaves[1])
    h, rows = torch.zeros(N, H * W, dtype=torch.float64), []
    for t in range(T):
        h = a[:, t] * h + (1 - a[:, t]) * leaves[0][:, t]
        rows.append(h)
    y = torch.stack(rows, 1).view(N, T, H, W)
    out = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * leaves[3] * torch.sigmoid(leaves[2]).view(N, T, H, W)
    want = torch.autograd.grad(out, leaves, dy.double())
    x, g, z, w, dy = (t.to(DEV) for t in (x, g, z, w, dy))
    chunks = torch.empty(kda.gated_scan_chunks(N, T), H * W, device=DEV)
    y, _ = kda.gated_scan(x, g, gate="sigmoid", complement=True, chunk_states=chunks)
    got = kda.gated_norm(y.view(N, T, H, W), z.view(N, T, H, W), w)
    dh, dz, dw = kda.gated_norm_backward(dy, y.view(N, T, H, W), z.view(N, T, H, W), w)
    dx, dg, _ = kda.gated_scan_backward(dh.view(N, T, -1), x, g, chunks, gate="sigmoid", complement=True)
    # a chain of some tens of FP32 roundings behind sums of 70 tokens and 32 elements: 2^-24 * 32 * 16
    for name, a, b in (("out", got, out), ("dx", dx, want[0]), ("dg", dg, want[1]), ("dz", dz, want[2]), ("dw", dw, want[3])):
        a, b = f64(a).ravel(), b.detach().numpy().ravel()
        assert np.linalg.norm(a - b) <= 2.0 ** -15 * np.linalg.norm(b), name


def test_python_refusals(kda):
    def t(*shape, dtype=BF16):
        return torch.zeros(*shape, dtype=dtype, device=DEV)

    x, g, st, ch = t(2, 5, 8), t(2, 5, 8), t(2, 8, dtype=F32), t(1, 8, dtype=F32)
    i32, w = torch.zeros(3, dtype=torch.int32, device=DEV), t(8)
    bad = [
        lambda: kda.gated_scan(x[0], g[0]), lambda: kda.gated_scan(x, g[:, :4]), lambda: kda.gated_scan(x, g.half()),
        lambda: kda.gated_scan(x.double(), g.double()), lambda: kda.gated_scan(x, g, gate="tanh"),
        lambda: kda.gated_scan(x, g, cu_seqlens=i32), lambda: kda.gated_scan(x[:1], g[:1], cu_seqlens=i32.long()),
        lambda: kda.gated_scan(x[:1], g[:1], cu_seqlens=i32[:1]), lambda: kda.gated_scan(x, g, slots=i32[:2]),
        lambda: kda.gated_scan(x, g, initial_state=st, slots=i32), lambda: kda.gated_scan(x, g, initial_state=st.half()),
        lambda: kda.gated_scan(x, g, initial_state=st[:1]), lambda: kda.gated_scan(x, g, final_state=st[:, :4]),
        lambda: kda.gated_scan(x, g, chunk_states=st), lambda: kda.gated_scan(x, g, out=x.float()),
        lambda: kda.gated_scan(x, g, out=t(2, 5, 16)[..., ::2]), lambda: kda.gated_scan(x, g.cpu()),
        lambda: kda.gated_scan(x.cpu(), g), lambda: kda.gated_scan(x, g, final_state=t(16, 2, dtype=F32).T[:2]),
        lambda: kda.gated_scan_backward(x, x, g, st), lambda: kda.gated_scan_backward(x, x[:, :3], g, ch),
        lambda: kda.gated_scan_backward(x, x.float(), g, ch), lambda: kda.gated_scan_backward(x, x, g.float(), ch, dg=g),
        lambda: kda.gated_scan_backward(x, x, g, ch, dg=g.float()), lambda: kda.gated_scan_backward(x, x, g, ch, dx=g.half()),
        lambda: kda.gated_scan_backward(x, kda.Checkpoint(t(2, 5, 8, dtype=torch.int8), t(2, 5, 2, dtype=torch.uint8)), g, ch),
        lambda: kda.gated_scan_backward(x, kda.Checkpoint(t(2, 5, 8, dtype=torch.uint8), t(2, 5, 1, dtype=torch.uint8)), g, ch),
        lambda: kda.gated_scan_backward(x, kda.Checkpoint(t(2, 5, 16, dtype=torch.int8)[..., :8], t(2, 5, 1, dtype=torch.uint8)), g, ch),
        lambda: kda.gated_scan_backward(x, kda.Checkpoint(t(2, 5, 8, dtype=torch.int8).cpu(), t(2, 5, 1, dtype=torch.uint8)), g, ch),
        lambda: kda.gated_scan_backward(x, x, g, ch, initial_state=st[:1]), lambda: kda.gated_scan_backward(x, x, g, ch, dfinal_state=st.half()),
        lambda: kda.gated_step(x, g, st), lambda: kda.gated_step(x[0], g[0], st), lambda: kda.gated_step(x[0, :2], g[0, :2], st.half()),
        lambda: kda.gated_step(x[0, :2], g[0, :2], st, slots=i32), lambda: kda.gated_step(x[0, :2], g[0, :3], st),
        lambda: kda.checkpoint_save(x.double()), lambda: kda.checkpoint_save(t(0, 0)),
        lambda: kda.checkpoint_save(x, out=kda.Checkpoint(t(2, 5, 8, dtype=torch.int8), t(2, 5, 2, dtype=torch.uint8))),
        lambda: kda.checkpoint_load(kda.checkpoint_save(x), torch.float64),
        lambda: kda.checkpoint_load(kda.checkpoint_save(x), BF16, out=x.float()),
        lambda: kda.checkpoint_load(kda.Checkpoint(t(3, 8, dtype=torch.int8), t(2, 1, dtype=torch.uint8)), BF16),
        lambda: kda.gated_norm_backward(x, x, g, w.float()), lambda: kda.gated_norm_backward(x, x, g, w[:4]),
        lambda: kda.gated_norm_backward(x, x.float(), g, w), lambda: kda.gated_norm_backward(x, x, g[:1], w),
        lambda: kda.gated_norm_backward(x, x, g, w, activation="tanh"), lambda: kda.gated_norm_backward(x, x, g, w, dweight=w),
        lambda: kda.gated_norm_backward(x, x, g, w, workspace=t(9, 9, dtype=torch.uint8).T[:5]),
        # a checkpoint of rows whose blocks are not those of the heads' rows
        lambda: kda.gated_norm_backward(x, kda.checkpoint_save(x.view(2, 40)), g, w),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {n} was not refused")
    for call in (lambda: kda.gated_scan(x, g, out=x), lambda: kda.gated_scan(x, g, final_state=st, chunk_states=st[:1]),
                 lambda: kda.gated_scan_backward(x, g, g, ch, dx=x), lambda: kda.gated_step(x[0, :2], g[0, :2], st, out=x[0, :2]),
                 lambda: kda.gated_norm_backward(x, x, g, w, dx=x),
                 lambda: kda.gated_norm_backward(x, x, g, w, workspace=t(4, dtype=torch.uint8))):
        with pytest.raises(kda.KdaError):
            call()
    torch.cuda.synchronize()


def test_two_streams_at_once(kda):
    """Calls of every operator on two streams, with workspaces of their own, do not meet."""
    cases = [Case([700, 33, 0, 250], 128, BF16, BF16, "sigmoid", True, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in cases]
    data = [[c.gpu(t) for t in (c.x, c.g, c.dy, c.cu, c.state, c.dfinal)] for c in cases]
    w = torch.ones(128, dtype=BF16, device=DEV)

    def layer(d):
        x, g, dy, cu, state, dfinal = d
        chunks = torch.empty(kda.gated_scan_chunks(*x.shape[:2]), 128, device=DEV)
        y, final = kda.gated_scan(x, g, cu, "sigmoid", True, initial_state=state, chunk_states=chunks)
        sy, sx = kda.checkpoint_save(y), kda.checkpoint_save(x)
        dh, dz, dw = kda.gated_norm_backward(dy, sy, g, w)
        return [y, final, dz, dw, *kda.gated_scan_backward(dh, sx, g, chunks, cu, "sigmoid", True, initial_state=state,
                                                           dfinal_state=dfinal)]

    want = [layer(d) for d in data]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [None, None]
        for n in (0, 1):
            with torch.cuda.stream(streams[n]):
                for _ in range(3):
                    got[n] = layer(data[n])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for m in (0, 1) for a, b in zip(got[m], want[m]))
