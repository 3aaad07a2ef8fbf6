"""The gated delta rule (prompts and single tokens) and the layer's norms against the
64-bit oracle on the same rounded inputs.

Tolerances, fixed before the first run.  FP32 results: the solver's parity bar, 2e-5,
on the scale of the result itself, |d| <= 2e-5 (M + |ref|) with M the largest |ref| of
the sequence's outputs (or state).  Where it comes from: a result is a chain of at most
five products whose operands and sums carry 2^-20 or better relative to the sums of
absolute values, and those sums are at most about 4 M for the inputs below; 5 * 4 * 2^-20
= 1.9e-5.  16-bit results: the reference is rounded to the type, and one unit in the last
place plus 1e-3 (M + |ref|) is allowed, the solver's bar for 16-bit input (bf16 products
that only reach the output keep 11 bits: 2^-11 of sums up to 2 M).  Norms: FP32 sums of up
to 16384 squares in a tree carry less than 32 * 2^-24 relative, the exponential and the
root a few units: 4e-6 |ref|, plus one unit in the last place of a 16-bit type.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.layer as ref

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


def ulp(ref_rounded, dtype):
    bits = {F32: 23, BF16: 7, F16: 10}[dtype]
    low = {F32: -126, BF16: -126, F16: -14}[dtype]
    e = np.maximum(np.frexp(np.abs(ref_rounded))[1] - 1, low)
    return np.ldexp(1.0, e - bits)


def close(got, want, dtype, label):
    """got (a tensor) against want (64 bits) with the tolerance of the docstring."""
    got = f64(got)
    assert got.shape == want.shape, (label, got.shape, want.shape)
    assert np.isfinite(got).all(), f"{label}: not finite"
    if want.size == 0:
        return
    M = np.max(np.abs(want))
    if dtype == F32:
        tol = 2e-5 * (M + np.abs(want))
    else:
        want = f64(torch.from_numpy(want).to(dtype))
        tol = 1e-3 * (M + np.abs(want)) + ulp(want, dtype)
    err = np.abs(got - want)
    worst = np.max(err / np.maximum(tol, 1e-300)) if M > 0 else np.max(err)
    assert (err <= tol).all(), f"{label}: {worst:.2f} of the tolerance"


class Rule:
    """Inputs of the gated delta rule, on the CPU in their types."""

    def __init__(self, lens, Hk=2, H=2, K=128, V=128, dtype=F32, gate="channel", packed=True, seed=0, rate=0.5,
                 vmag=1.0, initial=False, lead=None):
        rng = np.random.default_rng(seed)
        self.lens, self.packed, self.dtype = list(lens), packed, dtype
        self.H, self.K, self.V = H, K, V
        rows = sum(lens)
        lead = lead or ((1, rows) if packed else (len(lens), lens[0] if lens else 0))

        def unit(*s):
            x = rng.standard_normal(s)
            return x / np.linalg.norm(x, axis=-1, keepdims=True)

        def t(x, dt=dtype):
            return torch.from_numpy(np.ascontiguousarray(x)).to(dt)

        self.q, self.k = t(unit(*lead, Hk, K)), t(unit(*lead, Hk, K))
        self.v = t(vmag * rng.standard_normal((*lead, H, V)))
        self.beta = t(1 / (1 + np.exp(-rng.standard_normal((*lead, H)))))
        gs = (*lead, H, K) if gate == "channel" else (*lead, H)
        self.g = t(-rate * np.logaddexp(0, rng.standard_normal(gs)), F32)
        self.state = t(0.3 * vmag * rng.standard_normal((len(lens), H, K, V)), F32) if initial else None
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)) if packed else None
        self.scale = K ** -0.5

    def rows(self):
        a = 0
        for n in self.lens:
            yield a, a + n
            a += n

    def want(self, scale=None):
        o, S = [], []
        flat = [f64(x.reshape(-1, *x.shape[2:])) for x in (self.q, self.k, self.v, self.g, self.beta)]
        for n, (a, b) in enumerate(self.rows()):
            S0 = f64(self.state[n]) if self.state is not None else np.zeros((self.H, self.K, self.V))
            on, Sn = ref.delta_rule(*(x[a:b] for x in flat), S0, self.scale if scale is None else scale)
            o.append(on)
            S.append(Sn)
        return o, S

    def args(self):
        return [x.to(DEV) for x in (self.q, self.k, self.v, self.g, self.beta)]

    def run(self, kda, **kw):
        state = self.state.to(DEV) if self.state is not None else None
        cu = self.cu.to(DEV) if self.cu is not None else None
        o, S = kda.delta_prefill(*self.args(), cu_seqlens=cu, initial_state=state, **kw)
        torch.cuda.synchronize()
        return o.reshape(-1, self.H, self.V), S

    def check(self, kda, label="", **kw):
        o, S = self.run(kda, **kw)
        wo, wS = self.want(kw.get("scale"))
        for n, (a, b) in enumerate(self.rows()):
            close(o[a:b], wo[n], self.dtype, f"{label} o of sequence {n} ({b - a} tokens)")
            close(S[n], wS[n], F32, f"{label} state of sequence {n} ({b - a} tokens)")


LENS = (1, 2, 0, 63, 64, 65, 7, 130, 0, 200)


# ---------------------------------------------------------------- prompts
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("gate", ["channel", "head"])
@pytest.mark.parametrize("initial", [False, True])
def test_prefill_packed(kda, dtype, gate, initial):
    Rule(LENS, dtype=dtype, gate=gate, initial=initial, seed=1).check(kda)


@pytest.mark.parametrize("T", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("H", [1, 3])
def test_prefill_dense_lengths(kda, T, H):
    Rule([T, T], Hk=H, H=H, packed=False, seed=T, dtype=BF16 if T % 2 else F32, initial=T % 3 == 0).check(kda)


@pytest.mark.parametrize("K", [32, 64, 96, 128])
@pytest.mark.parametrize("V", [32, 64, 96, 128])
def test_prefill_widths(kda, K, V):
    Rule([70, 5, 64, 129], K=K, V=V, seed=K + V, dtype=F16, initial=True).check(kda)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("K,V", [(32, 64), (64, 32), (96, 32), (96, 128), (128, 96)])
def test_prefill_widths_many_chunks(kda, dtype, K, V):
    """Enough chunk-heads that every buffer of a persistent block goes round several times, with one to four
    slices of channels to a chunk."""
    Rule([170, 126, 276, 64], Hk=49, H=49, K=K, V=V, seed=K + V + 1, dtype=dtype).check(kda)


@pytest.mark.parametrize("Hk,H", [(1, 1), (1, 4), (2, 6), (5, 5), (3, 12)])
@pytest.mark.parametrize("gate", ["channel", "head"])
def test_prefill_shared_key_heads(kda, Hk, H, gate):
    Rule([100, 64, 3], Hk=Hk, H=H, gate=gate, seed=H, dtype=BF16).check(kda)


@pytest.mark.parametrize("rate", [0.0, 0.01, 0.1, 1.0, 1.45, 3.0, 20.0, 1e4])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_prefill_decays(kda, rate, dtype):
    """From no decay at all to one that clears the state with every token."""
    Rule([150, 64, 40], rate=rate, dtype=dtype, seed=7, initial=True).check(kda, f"rate {rate}")


def test_prefill_mixed_decays(kda):
    """Channels that keep everything beside channels that keep nothing, rows that clear all, and rows whose log
    decay is minus infinity."""
    for dtype in (F32, BF16):
        x = Rule([200, 70], dtype=dtype, seed=8, initial=True)
        x.g[..., ::3] = 0.0
        x.g[..., 1::7] *= 200.0
        x.g[0, 40] = -1e30
        x.g[0, 90, :, 5] = -float("inf")
        x.g[0, 210] = -float("inf")
        x.check(kda, "mixed")


@pytest.mark.parametrize("vmag", [1e-20, 1e-6, 1e-2, 1e3, 1e12])
def test_prefill_value_magnitudes(kda, vmag):
    for dtype in (F32, BF16):
        Rule([130, 64], dtype=dtype, vmag=vmag, seed=9, initial=True).check(kda, f"values of {vmag}")


def test_prefill_value_magnitudes_change(kda):
    """Values that jump by many orders of magnitude between chunks and between columns."""
    x = Rule([260], dtype=F32, seed=10, rate=0.1)
    x.v[0, 64:128] *= 1e8
    x.v[0, 128:] *= 1e-6
    x.v[..., 5] *= 1e10
    x.v[..., 6] = 0
    o, S = x.run(kda)
    wo, wS = x.want()
    for j in (0, 5, 6, 127):                              # columns are independent: each on its own scale
        close(o[..., j], wo[0][..., j], F32, f"column {j}")
        close(S[0][..., j], wS[0][..., j], F32, f"state column {j}")


@pytest.mark.parametrize("kmag", [1e-4, 1e-2, 4.0])
def test_prefill_key_magnitudes(kda, kmag):
    """Keys that are not of unit length (beta kept so that beta |k|^2 <= 1), queries of another size."""
    x = Rule([130, 40], dtype=F32, seed=11)
    x.k *= kmag
    x.q *= 50.0
    x.beta *= min(1.0, kmag ** -2)
    x.check(kda, f"keys of {kmag}")


def test_prefill_equal_keys(kda):
    """The same key in every token: the largest chunk matrix there is."""
    x = Rule([128, 64], dtype=F32, seed=12, rate=0.05)
    x.k[:] = x.k[:, :1]
    x.check(kda, "equal keys")


def test_prefill_zeros(kda):
    for what in ("beta", "k", "q", "v"):
        x = Rule([70, 64], dtype=BF16, seed=13, initial=True)
        getattr(x, what)[:] = 0
        x.check(kda, f"zero {what}")


def test_prefill_scale(kda):
    Rule([70], dtype=F32, seed=14).check(kda, scale=1.7)


def test_prefill_many_short_sequences(kda):
    rng = np.random.default_rng(3)
    Rule(rng.integers(0, 5, 600), Hk=1, H=1, K=32, V=32, dtype=F32, seed=15, initial=True).check(kda)


def test_prefill_long_sequence_few_heads(kda):
    """A long chain of chunks on one head."""
    Rule([4100], Hk=1, H=1, dtype=F32, seed=16, rate=0.02, initial=True).check(kda)
    Rule([3000, 20], Hk=1, H=2, dtype=BF16, seed=17, rate=0.3).check(kda)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("K,V,gate", [(128, 128, "channel"), (64, 128, "head"), (128, 32, "channel"), (32, 96, "channel")])
def test_prefill_split_sequences(kda, dtype, K, V, gate):
    """Few heads and long sequences, which are walked in segments; short and empty ones among them."""
    Rule([1500, 0, 700, 1, 64, 2111], Hk=1, H=2, K=K, V=V, gate=gate, dtype=dtype, seed=41, rate=0.03,
         initial=True).check(kda, "packed")
    Rule([1300, 1300], packed=False, Hk=1, H=1, K=K, V=V, gate=gate, dtype=dtype, seed=42, rate=0.5).check(kda, "dense")


def test_prefill_split_sequences_with_slots(kda):
    x = Rule([1200, 900, 0, 1000], dtype=F32, seed=43, rate=0.05)
    pool = torch.randn(5, 2, 128, 128, device=DEV)
    before = pool.clone()
    slots = [3, -1, 1, 0]
    x.state = torch.stack([before[s].cpu() if s >= 0 else torch.zeros(2, 128, 128) for s in slots])
    wo, wS = x.want()
    o, _ = kda.delta_prefill(*x.args(), cu_seqlens=x.cu.to(DEV), initial_state=pool,
                             slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    for n, (a, b) in enumerate(x.rows()):
        close(o[0, a:b], wo[n], F32, f"o {n}")
        if slots[n] >= 0:
            close(pool[slots[n]], wS[n], F32, f"state {n}")
    assert torch.equal(pool[2], before[2]) and torch.equal(pool[4], before[4])


def test_prefill_many_sequences_of_any_order(kda):
    """More sequences than are sorted by length, and fewer; long, short and empty ones mixed."""
    rng = np.random.default_rng(5)
    for n in (300, 90):
        lens = rng.integers(0, 3, n) * rng.integers(0, 90, n)
        Rule(lens, Hk=1, H=1, K=64, V=64, dtype=BF16, seed=44, initial=True).check(kda, f"{n} sequences")


def test_prefill_continues(kda):
    """A prompt given in two calls, its state passed on, is the prompt given at once."""
    x = Rule([200], dtype=F32, seed=18)
    o, S = x.run(kda)
    q, k, v, g, beta = x.args()
    for cut in (1, 64, 100, 199):
        parts, state = [], None
        for s in (slice(0, cut), slice(cut, 200)):
            p, state = kda.delta_prefill(q[:, s], k[:, s], v[:, s], g[:, s], beta[:, s], initial_state=state)
            parts.append(p)
        close(torch.cat(parts, 1)[0], f64(o), F32, f"cut at {cut}")
        close(state, f64(S), F32, f"state, cut at {cut}")


def test_prefill_slots(kda):
    """Pool entries by slot, updated in place; sequences without a slot; entries nobody uses stay as they are."""
    x = Rule([70, 0, 64, 3, 130], dtype=F32, seed=19)
    pool = torch.randn(9, 2, 128, 128, device=DEV)
    before = pool.clone()
    slots = [7, 2, -1, 99, 0]
    x.state = torch.stack([before[s].cpu() if 0 <= s < 9 else torch.zeros(2, 128, 128) for s in slots])
    wo, wS = x.want()
    o, out = kda.delta_prefill(*x.args(), cu_seqlens=x.cu.to(DEV), initial_state=pool,
                               slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert out is pool
    for n, (a, b) in enumerate(x.rows()):
        close(o[0, a:b], wo[n], F32, f"o {n}")
        if 0 <= slots[n] < 9:
            close(pool[slots[n]], wS[n], F32, f"state {n}")
    for e in set(range(9)) - set(slots):
        assert torch.equal(pool[e], before[e]), e
    assert torch.equal(pool[2], before[2])                # an empty sequence keeps its state
    # a pool to read and another to write
    dst = torch.full_like(pool, 5.0)
    kda.delta_prefill(*x.args(), cu_seqlens=x.cu.to(DEV), initial_state=before, final_state=dst,
                      slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    for n, s in enumerate(slots):
        if 0 <= s < 9:
            assert torch.equal(dst[s], pool[s])
    assert all(torch.all(dst[e] == 5.0) for e in set(range(9)) - set(slots))


def test_prefill_sequences_do_not_mix(kda):
    """A sequence full of NaN beside sound ones, whose partial chunks end where it begins."""
    x = Rule([70, 66, 3, 64], dtype=BF16, seed=20)
    wo, wS = x.want()
    for t in (x.q, x.k, x.v, x.g, x.beta):
        t[0, 70:136] = float("nan")
    o, S = x.run(kda)
    for n, (a, b) in enumerate(x.rows()):
        if n != 1:
            close(o[a:b], wo[n], BF16, f"o {n}")
            close(S[n], wS[n], F32, f"state {n}")
    assert torch.isnan(o[70:136]).any() and torch.isnan(S[1]).any()


def test_prefill_value_columns_do_not_mix(kda):
    """NaN or infinite values stay in their column."""
    x = Rule([130], dtype=F32, seed=21)
    wo, wS = x.want()
    x.v[0, 3, :, 7] = float("nan")
    x.v[0, 70, :, 40] = float("inf")
    o, S = x.run(kda)
    keep = [j for j in range(128) if j not in (7, 40)]
    close(o[..., keep], wo[0][..., keep], F32, "o")
    close(S[0][..., keep], wS[0][..., keep], F32, "state")


def test_prefill_writes_only_its_rows(kda):
    """out and states between guard values."""
    x = Rule([70, 64, 5], dtype=BF16, seed=22)
    big = torch.full((139 + 64 + 64, 2, 128), 3.0, dtype=BF16, device=DEV)
    out = big[64:64 + 139].unsqueeze(0)
    S = torch.full((5, 2, 128, 128), 3.0, device=DEV)
    kda.delta_prefill(*x.args(), cu_seqlens=x.cu.to(DEV), out=out, final_state=S[1:4])
    torch.cuda.synchronize()
    assert torch.all(big[:64] == 3) and torch.all(big[64 + 139:] == 3)
    assert torch.all(S[0] == 3) and torch.all(S[4] == 3)
    o, S2 = x.run(kda)
    assert torch.equal(out[0], o) and torch.equal(S[1:4], S2)


def test_prefill_strided_and_offset_inputs(kda):
    """Views into a fused projection, and tensors that do not start on a vector."""
    x = Rule([100], dtype=F32, seed=23)
    o, S = x.run(kda)
    q, k, v, g, beta = x.args()
    fused = torch.cat([q, k, v], dim=-1)
    qs, ks, vs = fused.split([128, 128, 128], dim=-1)
    flat = torch.empty(g.numel() + 1, device=DEV)
    go = flat[1:].view(g.shape)
    go.copy_(g)
    o2, S2 = kda.delta_prefill(qs, ks, vs, go, beta.transpose(1, 2).contiguous().transpose(1, 2))
    torch.cuda.synchronize()
    assert torch.equal(o2.reshape(-1, 2, 128), o) and torch.equal(S2, S)


def test_prefill_repeats_bit_for_bit(kda):
    x = Rule([300, 64, 5], Hk=4, H=4, dtype=BF16, seed=24, initial=True)
    o, S = x.run(kda)
    for _ in range(3):
        o2, S2 = x.run(kda)
        assert torch.equal(o, o2) and torch.equal(S, S2)


def test_prefill_workspace_of_the_caller(kda):
    x = Rule([130, 64], dtype=BF16, seed=25)
    o, S = x.run(kda)
    need = kda.delta_prefill_workspace_size(1, 194, 2, 2, 128, 128)
    ws = torch.full((max(need, 16) + 256,), 255, dtype=torch.uint8, device=DEV)
    o2, S2 = x.run(kda, workspace=ws[:max(need, 16)])
    assert torch.equal(o, o2) and torch.equal(S, S2)
    assert torch.all(ws[max(need, 16):] == 255)


def test_prefill_on_another_stream(kda):
    x = Rule([200, 64], dtype=BF16, seed=26, initial=True)
    o, S = x.run(kda)
    s = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device=DEV)
    for _ in range(3):
        args = x.args()
        state, cu = x.state.to(DEV), x.cu.to(DEV)
        big @ big                                         # keeps the default stream busy
        s.wait_stream(torch.cuda.current_stream())
        o2, S2 = kda.delta_prefill(*args, cu_seqlens=cu, initial_state=state, stream=s)
        s.synchronize()
        assert torch.equal(o2.reshape(-1, 2, 128), o) and torch.equal(S2, S)


def test_prefill_and_step_in_a_graph(kda):
    x = Rule([70, 64], dtype=BF16, seed=27)
    y = Rule([1, 1], dtype=BF16, seed=28, lead=(2,))
    o, S = x.run(kda)
    args, cu, step = x.args(), x.cu.to(DEV), y.args()
    state = S.clone()
    want = kda.delta_step(*step, state)
    out, S1 = torch.zeros_like(args[2]), torch.zeros_like(S)
    o1 = torch.zeros_like(want)
    ws = torch.empty(max(16, kda.delta_prefill_workspace_size(1, 134, 2, 2, 128, 128)), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.delta_prefill(*args, cu_seqlens=cu, out=out, final_state=S1, workspace=ws)
        kda.delta_step(*step, S1, out=o1)
    for _ in range(2):
        out.zero_()
        S1.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.reshape(-1, 2, 128), o) and torch.equal(S1, state) and torch.equal(o1, want)


def test_prefill_empty(kda):
    e = torch.empty(0, 64, 2, 128, device=DEV)
    o, S = kda.delta_prefill(e, e, e, e, e[..., 0])
    assert o.shape == e.shape and S.shape == (0, 2, 128, 128)
    e = torch.empty(2, 0, 2, 128, device=DEV)
    init = torch.randn(2, 2, 128, 128, device=DEV)
    o, S = kda.delta_prefill(e, e, e, e, e[..., 0], initial_state=init)
    assert o.shape == e.shape and torch.equal(S, init)
    o, S = kda.delta_prefill(e, e, e, e, e[..., 0])
    assert torch.all(S == 0)


# ---------------------------------------------------------- single tokens
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("gate", ["channel", "head"])
@pytest.mark.parametrize("N", [1, 3])
@pytest.mark.parametrize("K,V", [(128, 128), (64, 128), (128, 64), (96, 32), (32, 96)])
def test_step(kda, dtype, gate, N, K, V):
    x = Rule([1] * N, Hk=2, H=4, K=K, V=V, dtype=dtype, gate=gate, seed=30, initial=True, lead=(N,))
    pool = x.state.to(DEV)
    o = kda.delta_step(*x.args(), pool)
    torch.cuda.synchronize()
    for n in range(N):
        wo, wS = ref.delta_rule(*(f64(t[n:n + 1]) for t in (x.q, x.k, x.v, x.g, x.beta)), f64(x.state[n]), x.scale)
        close(o[n:n + 1], wo, dtype, f"o {n}")
        close(pool[n], wS, F32, f"state {n}")


@pytest.mark.parametrize("N,H", [(40, 16), (400, 2)])
def test_step_batches_and_slots(kda, N, H):
    x = Rule([1] * N, Hk=H, H=H, dtype=BF16, seed=31, lead=(N,))
    pool = torch.randn(N + 5, H, 128, 128, device=DEV)
    before = pool.clone()
    slots = np.random.default_rng(0).permutation(N + 5)[:N].astype(np.int32)
    slots[3], slots[7] = -1, N + 5
    o = kda.delta_step(*x.args(), pool, slots=torch.from_numpy(slots).to(DEV))
    torch.cuda.synchronize()
    used = set()
    for n in range(N):
        s = int(slots[n])
        has = 0 <= s < N + 5
        used |= {s} if has else set()
        S0 = f64(before[s]) if has else np.zeros((H, 128, 128))
        wo, wS = ref.delta_rule(*(f64(t[n:n + 1]) for t in (x.q, x.k, x.v, x.g, x.beta)), S0, x.scale)
        close(o[n:n + 1], wo, BF16, f"o {n}")
        if has:
            close(pool[s], wS, F32, f"state {n}")
    for e in set(range(N + 5)) - used:
        assert torch.equal(pool[e], before[e]), e


def test_steps_are_the_prompt(kda):
    """Token by token from zero states is the prompt at once."""
    x = Rule([100, 100], packed=False, dtype=F32, seed=32, rate=0.1)
    o, S = x.run(kda)
    q, k, v, g, beta = x.args()
    pool = torch.zeros(2, 2, 128, 128, device=DEV)
    steps = [kda.delta_step(q[:, t], k[:, t], v[:, t], g[:, t], beta[:, t], pool) for t in range(100)]
    close(torch.stack(steps, 1).reshape(-1, 2, 128), f64(o), F32, "o")
    close(pool, f64(S), F32, "state")


def test_step_extreme_decays(kda):
    x = Rule([1, 1, 1], dtype=F32, seed=33, initial=True, lead=(3,))
    x.g[0], x.g[1], x.g[2] = 0.0, -1e30, -float("inf")
    pool = x.state.to(DEV)
    o = kda.delta_step(*x.args(), pool)
    for n in range(3):
        wo, wS = ref.delta_rule(*(f64(t[n:n + 1]) for t in (x.q, x.k, x.v, x.g, x.beta)), f64(x.state[n]), x.scale)
        close(o[n:n + 1], wo, F32, f"o {n}")
        close(pool[n], wS, F32, f"state {n}")


def test_step_far_into_the_pool(kda):
    """Entries whose offset passes 32 bits."""
    H, entries = 64, 2100                                 # 64 heads of 64 KiB: entry 2048 starts at 2^31 values
    pool = torch.zeros(entries, H, 128, 128, device=DEV)
    x = Rule([1, 1], Hk=H, H=H, dtype=BF16, seed=34, initial=True, lead=(2,))
    slots = [2099, 1]
    for n, s in enumerate(slots):
        pool[s] = x.state[n].to(DEV)
    o = kda.delta_step(*x.args(), pool, slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    for n, s in enumerate(slots):
        wo, wS = ref.delta_rule(*(f64(t[n:n + 1]) for t in (x.q, x.k, x.v, x.g, x.beta)), f64(x.state[n]), x.scale)
        close(o[n:n + 1], wo, BF16, f"o {n}")
        close(pool[s], wS, F32, f"state {n}")
    assert int(torch.count_nonzero(pool[2:2099])) == 0 and int(torch.count_nonzero(pool[0])) == 0


# ----------------------------------------------------------------- norms
def norm_close(got, want, dtype, label):
    got = f64(got)
    assert np.isfinite(got).all(), label
    rounded = f64(torch.from_numpy(want).to(dtype))
    tol = 4e-6 * np.abs(want) + (ulp(rounded, dtype) if dtype != F32 else 0) + 1e-37
    assert (np.abs(got - rounded) <= tol).all(), (label, np.max(np.abs(got - rounded) / tol))


DIMS = [1, 2, 7, 8, 31, 33, 64, 96, 128, 255, 256, 300, 512, 520, 1000, 2049, 2304, 4096, 8192, 8200, 16383, 16384]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("dim", DIMS)
def test_add_norm(kda, dtype, dim):
    rng = np.random.default_rng(dim)
    rows = 5 if dim > 600 else 37
    x, r = (torch.from_numpy(rng.standard_normal((rows, dim))).to(dtype) for _ in range(2))
    w = torch.from_numpy(1 + 0.1 * rng.standard_normal(dim)).to(dtype)
    y, out = kda.add_norm(x.to(DEV), r.to(DEV), w.to(DEV), alpha=0.75, eps=1e-5)
    wy, wr = ref.add_norm(f64(x), f64(r), f64(w), 0.75, 1e-5)
    # r itself can cancel: its error is that of its terms
    assert (np.abs(f64(out) - wr) <= 2.0 ** -22 * (np.abs(f64(x)) + np.abs(f64(r))) + ulp(wr, dtype)).all()
    scale = np.abs(f64(w)) / np.sqrt(np.mean(wr * wr, -1, keepdims=True) + 1e-5)
    tol = 4e-6 * np.abs(wy) + 2.0 ** -22 * (np.abs(f64(x)) + np.abs(f64(r))) * scale + ulp(wy, dtype)
    assert (np.abs(f64(y) - wy) <= tol).all()
    # no residual: the plain norm of alpha x; outputs in the inputs' buffers
    xb = x.to(DEV)
    y2, out2 = kda.add_norm(xb, None, w.to(DEV), alpha=0.75, eps=1e-5, out=xb)
    wy, _ = ref.add_norm(f64(x), None, f64(w), 0.75, 1e-5)
    norm_close(y2, wy, dtype, "no residual")
    assert y2 is xb
    rb = r.to(DEV)
    y3, out3 = kda.add_norm(x.to(DEV), rb, w.to(DEV), alpha=0.75, eps=1e-5, residual_out=rb)
    assert out3 is rb and torch.equal(y3, y) and torch.equal(rb, out)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gated_norm(kda, dtype, dim, act):
    rng = np.random.default_rng(dim)
    lead = (3,) if dim > 600 else (7, 5)
    x, z = (torch.from_numpy(rng.standard_normal((*lead, dim))).to(dtype) for _ in range(2))
    w = torch.from_numpy(1 + 0.1 * rng.standard_normal(dim)).to(dtype)
    want = ref.gated_norm(f64(x), f64(z), f64(w), 1e-6, act)
    y = kda.gated_norm(x.to(DEV), z.to(DEV), w.to(DEV), activation=act)
    norm_close(y, want, dtype, f"{dim}")
    for into in (0, 1):
        bufs = [x.to(DEV), z.to(DEV)]
        y2 = kda.gated_norm(bufs[0], bufs[1], w.to(DEV), activation=act, out=bufs[into])
        assert torch.equal(y2, y)


@pytest.mark.parametrize("dim", [128, 129, 4096])
def test_norms_edge_rows(kda, dim):
    """Rows of zeros, of very large and very small values, and gates far out; a NaN row stays alone."""
    x = torch.randn(6, dim)
    x[0] = 0
    x[1] *= 1e15
    x[2] *= 1e-25
    w = torch.ones(dim)
    z = torch.randn(6, dim)
    z[3] = 300.0
    z[4] = -300.0
    y = kda.gated_norm(x.to(DEV), z.to(DEV), w.to(DEV))
    want = ref.gated_norm(f64(x), np.maximum(f64(z), -300), f64(w), 1e-6, "sigmoid")
    got = f64(y)
    assert np.isfinite(got).all() and (got[0] == 0).all()
    rows = [1, 2, 3, 5]
    assert (np.abs(got[rows] - want[rows]) <= 4e-6 * np.abs(want[rows]) + 1e-37).all()
    assert (np.abs(got[4]) <= 1e-37).all()
    a, _ = kda.add_norm(x.to(DEV), None, w.to(DEV))
    x[5] = float("nan")
    b, _ = kda.add_norm(x.to(DEV), None, w.to(DEV))
    assert torch.equal(a[:5], b[:5]) and torch.isnan(b[5]).all()


def test_norms_views_and_offsets(kda):
    """Strided views, rows that do not start on a vector, guard values around the outputs."""
    base = torch.randn(10, 3, 256, device=DEV, dtype=BF16)
    x, z = base[:, 0, :128], base[:, 1, 128:]
    w = torch.randn(128, device=DEV, dtype=BF16)
    y = kda.gated_norm(x, z, w)
    assert torch.equal(y, kda.gated_norm(x.contiguous(), z.contiguous(), w))
    flat = torch.full((10 * 128 + 3,), 9.0, device=DEV, dtype=BF16)
    out = flat[1:1 + 1280].view(10, 128)
    kda.gated_norm(x, z, w, out=out)
    assert torch.equal(out, y) and flat[0] == 9 and torch.all(flat[1281:] == 9)
    many = torch.randn(100003, 64, device=DEV, dtype=F16)
    r, _ = kda.add_norm(many, None, torch.ones(64, device=DEV, dtype=F16))
    want = f64(many) / np.sqrt(np.mean(f64(many) ** 2, -1, keepdims=True) + 1e-6)
    norm_close(r, want, F16, "many rows")
    assert kda.add_norm(many[:0], None, torch.ones(64, device=DEV, dtype=F16))[0].shape == (0, 64)


def test_norms_on_another_stream(kda):
    s = torch.cuda.Stream()
    x, z = (torch.randn(4096, 1000, device=DEV) for _ in range(2))
    w = torch.ones(1000, device=DEV)
    want = kda.gated_norm(x, z, w)
    s.wait_stream(torch.cuda.current_stream())
    got = kda.gated_norm(x.t().contiguous().t(), z, w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


# -------------------------------------------------------------- refusals
def test_refusals(kda):
    x = Rule([70, 64], dtype=BF16, seed=40)
    q, k, v, g, beta = x.args()
    cu = x.cu.to(DEV)
    S = torch.zeros(2, 2, 128, 128, device=DEV)
    for bad in (
        lambda: kda.delta_prefill(q.cpu(), k, v, g, beta),
        lambda: kda.delta_prefill(q, k[..., :64], v, g, beta),
        lambda: kda.delta_prefill(q[..., :48], k[..., :48], v, g[..., :48], beta),
        lambda: kda.delta_prefill(q, k, v[..., :100], g, beta),
        lambda: kda.delta_prefill(q, k, v, g.to(BF16), beta),
        lambda: kda.delta_prefill(q, k, v, g[..., :64], beta),
        lambda: kda.delta_prefill(q, k, v, g, beta.float()),
        lambda: kda.delta_prefill(q, k, v, g, beta[..., 0]),
        lambda: kda.delta_prefill(q.double(), k.double(), v.double(), g, beta.double()),
        lambda: kda.delta_prefill(q, k, v, g, beta, cu_seqlens=cu.long()),
        lambda: kda.delta_prefill(q, k, v, g, beta, cu_seqlens=cu[:1]),
        lambda: kda.delta_prefill(q, k, v, g, beta, cu_seqlens=cu, initial_state=S[:1]),
        lambda: kda.delta_prefill(q, k, v, g, beta, cu_seqlens=cu, initial_state=S.to(BF16)),
        lambda: kda.delta_prefill(q, k, v, g, beta, cu_seqlens=cu, initial_state=S.transpose(2, 3)),
        lambda: kda.delta_prefill(q, k, v, g, beta, cu_seqlens=cu, slots=cu[:2]),
        lambda: kda.delta_prefill(q, k, v, g, beta, cu_seqlens=cu, initial_state=S, slots=cu),
        lambda: kda.delta_prefill(q, k, v, g, beta, out=v[..., :64]),
        lambda: kda.delta_step(q[0], k[0], v[0], g[0], beta[0], S),
        lambda: kda.delta_step(q[0, :2], k[0, :2], v[0, :2], g[0, :2], beta[0, :2], S[:, :1]),
        lambda: kda.delta_step(q[0, :2], k[0, :2], v[0, :2], g[0, :2], beta[0, :2], S, slots=cu),
        lambda: kda.add_norm(q, k[..., :64], q[0, 0, 0]),
        lambda: kda.add_norm(q, k, q[0, 0, 0].float()),
        lambda: kda.add_norm(q, k.float(), q[0, 0, 0]),
        lambda: kda.add_norm(q, k, q[0, 0]),
        lambda: kda.gated_norm(q, k, q[0, 0, 0], activation="tanh"),
        lambda: kda.gated_norm(q, k[:, :3], q[0, 0, 0]),
    ):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(kda.KdaError):
        kda.delta_prefill(q, k, v, g, beta, out=v)        # o on top of v
    with pytest.raises(kda.KdaError):
        kda.gated_norm(q, k, q[0, 0, 0], eps=-1.0)
    wide = torch.zeros(1, 16385, device=DEV)
    with pytest.raises(kda.KdaError):
        kda.add_norm(wide, None, wide[0])


@pytest.mark.parametrize("dtype, K", [(F32, 64), (F32, 128), (F16, 128), (BF16, 96)], ids=str)
def test_prefill_batch_rows_do_not_mix(kda, dtype, K):
    """A dense batch whose middle row is NaN: its neighbours' last chunks are partial."""
    x = Rule([70, 70, 70], K=K, dtype=dtype, packed=False, seed=41)
    wo, wS = x.want()
    for t in (x.q, x.k, x.v, x.g, x.beta):
        t[1] = float("nan")
    o, S = x.run(kda)
    for n, (a, b) in enumerate(x.rows()):
        if n != 1:
            close(o[a:b], wo[n], dtype, f"o {n}")
            close(S[n], wS[n], F32, f"state {n}")


@pytest.mark.parametrize("batch, tokens", [(1, 1500), (2, 1500), (3, 1030), (5, 2048)])
def test_prefill_split_batches(kda, batch, tokens):
    """Dense batches of few heads, whose rows are split into segments."""
    x = Rule([tokens] * batch, H=1, Hk=1, dtype=F32, packed=False, seed=42, rate=0.02, initial=True)
    x.check(kda)


@pytest.mark.parametrize("lens", [(70, 33), (5, 3)], ids=["chunks", "tokens"])
def test_prefill_rows_past_the_last_sequence(kda, lens):
    """Rows of the packed tensors that belong to no sequence are neither read nor written."""
    x = Rule([*lens, 20], dtype=BF16, seed=44)
    used = sum(lens)
    wo, wS = x.want()
    for t in (x.q, x.k, x.v, x.g, x.beta):
        t[0, used:] = float("nan")
    out = torch.full((1, used + 20, 2, 128), 3.0, dtype=BF16, device=DEV)
    o, S = kda.delta_prefill(*x.args(), cu_seqlens=x.cu[:-1].to(DEV), out=out)
    torch.cuda.synchronize()
    assert torch.all(out[0, used:] == 3)
    for n, (a, b) in enumerate(list(x.rows())[:-1]):
        close(o[0, a:b], wo[n], BF16, f"o {n}")
        close(S[n], wS[n], F32, f"state {n}")
