"""The layer operators' argument checks on a machine without a GPU: every refusal comes
before any CUDA call, which would give KDA_ERR_CUDA here."""
import numpy as np
import pytest

import linear_attention_chunked_02_gb300 as kda
import oracle.layer as ref
from linear_attention_chunked_02_gb300 import build as kbuild

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = [1 << (30 + i) for i in range(12)]                     # distinct, aligned, far apart


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kda.lib()


def prefill(L, q=P[0], k=P[1], v=P[2], g=P[3], beta=P[4], o=P[5], sin=None, sout=P[6], slots=None, nslots=0, cu=None,
            nseq=0, B=1, T=64, Hk=2, H=2, K=128, V=128, dt=1, gate=0, scale=1.0, ws=P[7], wsb=1 << 30):
    return L.kda_delta_prefill(q, k, v, g, beta, o, sin, sout, slots, nslots, cu, nseq, B, T, Hk, H, K, V, dt, gate,
                               scale, ws, wsb, None)


def test_prefill_refusals(L):
    for name in ("q", "k", "v", "g", "beta", "o"):
        assert prefill(L, **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "g", "o", "sin", "sout", "beta"):
        assert prefill(L, **{name: P[9] + (1 if name == "beta" else 8)}) == INVALID, name
    for K in (0, 16, 48, 160, 256, -32):
        assert prefill(L, K=K) == UNSUPPORTED and prefill(L, V=K) == UNSUPPORTED
    assert prefill(L, dt=3) == UNSUPPORTED and prefill(L, dt=-1) == UNSUPPORTED
    assert prefill(L, gate=2) == INVALID
    assert prefill(L, Hk=0) == INVALID and prefill(L, H=0) == INVALID and prefill(L, Hk=2, H=3) == INVALID
    assert prefill(L, Hk=4, H=2) == INVALID
    assert prefill(L, B=-1) == INVALID and prefill(L, T=-1) == INVALID and prefill(L, nseq=-1) == INVALID
    assert prefill(L, cu=P[8]) == INVALID and prefill(L, nseq=2) == INVALID
    assert prefill(L, cu=P[8], nseq=2, B=2) == INVALID
    assert prefill(L, slots=P[8], nslots=-1) == INVALID
    assert prefill(L, T=1 << 31) == UNSUPPORTED and prefill(L, B=1 << 20, T=1 << 12) == UNSUPPORTED
    assert prefill(L, Hk=1 << 17, H=1 << 17) == UNSUPPORTED
    assert prefill(L, o=P[2]) == INVALID                                   # on top of v
    assert prefill(L, o=P[0] + 64 * 2 * 128 * 2 - 16) == INVALID           # the last bytes of q
    assert prefill(L, sin=P[6], sout=P[6] + 64) == INVALID                 # neither the same nor apart
    assert prefill(L, o=P[6]) == INVALID
    need = kda.delta_prefill_workspace_size(1, 64, 2)
    if need:
        assert prefill(L, ws=None) == WORKSPACE and prefill(L, wsb=need - 1) == WORKSPACE
        assert prefill(L, ws=P[7] + 8) == INVALID
    assert prefill(L, B=0) == OK and prefill(L, T=0, sout=None) == OK


def test_prefill_workspace_size(L):
    size = kda.delta_prefill_workspace_size
    for bad in ((1, 64, 0), (1, 64, 2, -1), (2, 64, 2, 3), (1, 64, 2, 0, 48, 128), (1, 64, 2, 0, 128, 12)):
        assert size(*bad) == 0
    assert size(0, 64, 2) == 0 and size(1, 0, 2) == 0


def step(L, q=P[0], k=P[1], v=P[2], g=P[3], beta=P[4], o=P[5], state=P[6], slots=None, nslots=4, N=4, Hk=2, H=2,
         K=128, V=128, dt=1, gate=0, scale=1.0):
    return L.kda_delta_step(q, k, v, g, beta, o, state, slots, nslots, N, Hk, H, K, V, dt, gate, scale, None)


def test_step_refusals(L):
    for name in ("q", "k", "v", "g", "beta", "o", "state"):
        assert step(L, **{name: None}) == INVALID, name
        assert step(L, **{name: P[9] + (1 if name == "beta" else 8)}) == INVALID, name
    assert step(L, K=100) == UNSUPPORTED and step(L, V=8) == UNSUPPORTED and step(L, dt=9) == UNSUPPORTED
    assert step(L, gate=-1) == INVALID and step(L, Hk=3) == INVALID and step(L, N=-1) == INVALID
    assert step(L, nslots=3) == INVALID and step(L, slots=P[8], nslots=-1) == INVALID
    assert step(L, o=P[6] + 1024) == INVALID and step(L, o=P[1]) == INVALID
    assert step(L, N=0) == OK


def add(L, x=P[0], r=P[1], w=P[2], y=P[3], out=P[4], rows=4, dim=64, alpha=1.0, eps=1e-6, dt=0):
    return L.kda_add_norm(x, r, w, y, out, rows, dim, alpha, eps, dt, None)


def gated(L, x=P[0], z=P[1], w=P[2], y=P[3], rows=4, dim=64, eps=1e-6, act=0, dt=0):
    return L.kda_gated_norm(x, z, w, y, rows, dim, eps, act, dt, None)


def test_norm_refusals(L):
    for name in ("x", "w", "y"):
        assert add(L, **{name: None}) == INVALID and gated(L, **{name: None}) == INVALID, name
    assert gated(L, z=None) == INVALID
    for name in ("x", "r", "w", "y", "out"):
        assert add(L, **{name: P[9] + 2}) == INVALID, name
    for name in ("x", "z", "w", "y"):
        assert gated(L, **{name: P[9] + 1}, dt=1) == INVALID, name
    for f in (add, gated):
        assert f(L, dim=0) == INVALID and f(L, rows=-1) == INVALID and f(L, eps=-1.0) == INVALID
        assert f(L, eps=float("nan")) == INVALID
        assert f(L, dim=16385) == UNSUPPORTED and f(L, dt=4) == UNSUPPORTED and f(L, rows=1 << 31) == UNSUPPORTED
        assert f(L, rows=0) == OK
        assert f(L, y=P[2] + 4) == INVALID                                 # inside the weight
        assert f(L, y=P[0] + 4) == INVALID                                 # shifted against x
    assert add(L, y=P[1]) == INVALID and add(L, out=P[0]) == INVALID and add(L, out=P[3]) == INVALID
    assert add(L, out=P[1] + 4) == INVALID
    assert gated(L, act=2) == INVALID and gated(L, act=-1) == INVALID


def test_python_refuses_cpu_tensors():
    import torch
    x = torch.zeros(1, 4, 2, 128)
    with pytest.raises(ValueError, match="CUDA"):
        kda.delta_prefill(x, x, x, x, x[..., 0])
    with pytest.raises(ValueError, match="CUDA"):
        kda.delta_step(x[0], x[0], x[0], x[0], x[0, ..., 0], x)
    with pytest.raises(ValueError, match="CUDA"):
        kda.add_norm(x, x, x[0, 0, 0])
    with pytest.raises(ValueError, match="CUDA"):
        kda.gated_norm(x, x, x[0, 0, 0])


def test_oracle_by_hand():
    """Two tokens of one channel and one column, worked by hand; and the chunk form's closed formula."""
    one = np.ones((2, 1, 1))
    o, S = ref.delta_rule(one, one, np.array([[[2.0]], [[3.0]]]), np.log(np.array([[[0.5]], [[0.25]]])),
                          np.array([[0.5], [1.0]]), np.full((1, 1, 1), 4.0), 2.0)
    # S: 4 -> 2, u = .5 (2 - 2) = 0, S = 2; -> .5, u = 3 - .5, S = 3
    assert o.ravel().tolist() == [4.0, 6.0] and S.item() == 3.0
    rng = np.random.default_rng(0)
    n, K, V = 9, 5, 3
    q, k = rng.standard_normal((2, n, 1, K)) * 0.4
    v, g, b = rng.standard_normal((n, 1, V)), -rng.random((n, 1, K)), rng.random((n, 1))
    S0 = rng.standard_normal((1, K, V))
    o, S = ref.delta_rule(q, k, v, g, b, S0, 1.0)
    G = np.cumsum(g[:, 0], 0)
    D = np.exp(G[:, None] - G[None])
    A = np.tril(b * np.einsum("id,jd,ijd->ij", k[:, 0], k[:, 0], D), -1)
    Pm = np.tril(np.einsum("id,jd,ijd->ij", q[:, 0], k[:, 0], D))
    U = np.linalg.solve(np.eye(n) + A, b * (v[:, 0] - (k[:, 0] * np.exp(G)) @ S0[0]))
    assert np.allclose(o[:, 0], (q[:, 0] * np.exp(G)) @ S0[0] + Pm @ U, rtol=0, atol=1e-13)
    assert np.allclose(S[0], np.exp(G[-1])[:, None] * S0[0] + (k[:, 0] * np.exp(G[-1] - G)).T @ U, rtol=0, atol=1e-13)
    x, z, w = rng.standard_normal((2, 4)), rng.standard_normal((2, 4)), rng.standard_normal(4)
    y, r = ref.add_norm(x, z, w, 2.0, 0.0)
    assert np.allclose((y / w) ** 2 @ np.ones(4), 4) and np.allclose(r, z + 2 * x)
    assert np.allclose(ref.gated_norm(x, z, w, 0.0, "silu"), ref.gated_norm(x, z, w, 0.0, "sigmoid") * z)
