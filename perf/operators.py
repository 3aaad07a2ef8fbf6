"""The layer operators around the chunk solve, as cases that can be timed and compared.

Four operators make up a gated-delta-rule layer between its projections:

  prefill      the gated delta rule over whole prompts, chunk by chunk
  step         one token for each running request, its state updated in place
  add_norm     residual sum and the norm before the block
  gated_norm   the norm after the block, times its gate

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits.
With ``own`` true, it calls the package's operators.  ``exact`` follows the
definition token by token in 64 bits.

The gated delta rule of one head, state S [K, V], for each token:
    S <- diag(exp(g)) S;   u = beta (v - S^T k);   S <- S + k u^T;   o = scale S^T q.
"""
import math
import random

import torch

own = False

CHUNK = 64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # the smallest prompt: one chunk of four heads, where the launches count
        {"name": "prefill_1x64_h4_f32", "op": "prefill", "packed": False, "seqs": 1, "longest": 64, "ragged": 0,
         "hk": 4, "h": 4, "k": 128, "v": 128, "gate": "channel", "initial": False, "dtype": "f32"},
        # a full batch of equal prompts, packed
        {"name": "prefill_16x512_h64_bf16", "op": "prefill", "packed": True, "seqs": 16, "longest": 512, "ragged": 0,
         "hk": 64, "h": 64, "k": 128, "v": 128, "gate": "channel", "initial": False, "dtype": "bf16"},
        # continued prompts of mixed lengths, their states in a pool that is updated in place
        {"name": "prefill_ragged37_h32_f16", "op": "prefill", "packed": True, "seqs": 37, "longest": 2048, "ragged": 3,
         "hk": 32, "h": 32, "k": 128, "v": 128, "gate": "channel", "initial": True, "dtype": "f16"},
        # one long document: few rows, a long chain of chunks
        {"name": "prefill_1x16384_h32_bf16", "op": "prefill", "packed": False, "seqs": 1, "longest": 16384,
         "ragged": 0, "hk": 32, "h": 32, "k": 128, "v": 128, "gate": "channel", "initial": False, "dtype": "bf16"},
        # the largest: four long prompts at 64 heads
        {"name": "prefill_4x8192_h64_bf16", "op": "prefill", "packed": False, "seqs": 4, "longest": 8192, "ragged": 0,
         "hk": 64, "h": 64, "k": 128, "v": 128, "gate": "channel", "initial": False, "dtype": "bf16"},
        # one decay for a whole head, keys shared by four heads, lengths that end inside a chunk
        {"name": "prefill_2x1000_hk4_h16_f32", "op": "prefill", "packed": False, "seqs": 2, "longest": 1000,
         "ragged": 0, "hk": 4, "h": 16, "k": 64, "v": 128, "gate": "head", "initial": True, "dtype": "f32"},
        # one running request
        {"name": "step_1_h32_bf16", "op": "step", "seqs": 1, "hk": 32, "h": 32, "k": 128, "v": 128,
         "gate": "channel", "dtype": "bf16"},
        # a full decoding batch
        {"name": "step_256_h64_bf16", "op": "step", "seqs": 256, "hk": 64, "h": 64, "k": 128, "v": 128,
         "gate": "channel", "dtype": "bf16"},
        # residual sum and norm of a prompt batch's hidden rows
        {"name": "add_norm_8192x4096_bf16", "op": "add_norm", "rows": 8192, "dim": 4096, "alpha": 1.0, "dtype": "bf16"},
        # the same for a few decoding rows, of a width that is no multiple of a vector
        {"name": "add_norm_7x2305_f32", "op": "add_norm", "rows": 7, "dim": 2305, "alpha": 0.5, "dtype": "f32"},
        # the heads' outputs of a prompt batch, with their gates
        {"name": "gated_norm_8192x64x128_bf16", "op": "gated_norm", "rows": 8192, "h": 64, "dim": 128,
         "act": "sigmoid", "dtype": "bf16"},
        # the same for a small decoding batch
        {"name": "gated_norm_16x32x128_f16", "op": "gated_norm", "rows": 16, "h": 32, "dim": 128,
         "act": "silu", "dtype": "f16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "step", "step", "add_norm", "gated_norm"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("prefill", "step"):
        group = rng.choice([1, 1, 2, 4])
        hk = _log(rng, 1, 64 // group)
        case = {"op": op, "hk": hk, "h": hk * group, "k": rng.choice([32, 64, 96, 128, 128, 128]),
                "v": rng.choice([32, 64, 96, 128, 128, 128]), "gate": rng.choice(["channel", "channel", "head"]),
                "dtype": dtype}
        if op == "step":
            return dict(case, seqs=_log(rng, 1, 256))
        seqs = _log(rng, 1, 48)
        longest = _log(rng, 1, 16384)
        most = (1 << 20) // (seqs * case["h"])               # bounds the plain form's padded work
        return dict(case, seqs=seqs, longest=max(1, min(longest, most)), packed=rng.random() < 0.6,
                    ragged=rng.randrange(1, 1000), initial=rng.random() < 0.5)
    if op == "add_norm":
        return {"op": op, "rows": _log(rng, 1, 8192), "dim": _log(rng, 64, 8192), "alpha": rng.choice([1.0, 0.25]),
                "dtype": dtype}
    return {"op": op, "rows": _log(rng, 1, 8192), "h": _log(rng, 1, 64), "dim": rng.choice([64, 96, 128, 128, 256]),
            "act": rng.choice(["sigmoid", "silu"]), "dtype": dtype}


def _lengths(case):
    """Tokens of every sequence: equal ones, or (packed and ragged) uniform in [1, longest]."""
    if not case["packed"] or not case["ragged"]:
        return [case["longest"]] * case["seqs"]
    rng = random.Random(case["ragged"])
    return [rng.randint(1, case["longest"]) for _ in range(case["seqs"])]


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = {"case": case}
    if case["op"] == "add_norm":
        s["x"] = normal(case["rows"], case["dim"]).to(dt)
        s["residual"] = (4 * normal(case["rows"], case["dim"])).to(dt)
        s["weight"] = (1 + 0.1 * normal(case["dim"])).to(dt)
        return s
    if case["op"] == "gated_norm":
        s["x"] = (0.1 * normal(case["rows"], case["h"], case["dim"])).to(dt)
        s["gate"] = normal(case["rows"], case["h"], case["dim"]).to(dt)
        s["weight"] = (1 + 0.1 * normal(case["dim"])).to(dt)
        return s
    hk, h, K, V = case["hk"], case["h"], case["k"], case["v"]
    if case["op"] == "step":
        lead = (case["seqs"],)
    else:
        lens = _lengths(case)
        lead = (1, sum(lens)) if case["packed"] else (case["seqs"], case["longest"])
        if case["packed"]:
            ends = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)
            s["cu_seqlens"] = ends.to(dev)
    # unit keys and queries; decays exp(g) whose rate differs from head to head by a factor of a
    # hundred, from long memories to one that is gone in a few tokens
    s["q"] = _unit(normal(*lead, hk, K)).to(dt)
    s["k"] = _unit(normal(*lead, hk, K)).to(dt)
    s["v"] = normal(*lead, h, V).to(dt)
    s["beta"] = torch.sigmoid(normal(*lead, h)).to(dt)
    rate = 0.01 * 100 ** torch.rand(h, generator=gen, device=dev)
    if case["gate"] == "channel":
        s["g"] = -rate[:, None] * torch.nn.functional.softplus(normal(*lead, h, K))
    else:
        s["g"] = -rate * torch.nn.functional.softplus(normal(*lead, h))
    if case["op"] == "step":
        # a pool with room for more requests than are running
        pool = case["seqs"] + 1 + case["seqs"] // 8
        s["state"] = 0.3 * normal(pool, h, K, V)
        s["slots"] = torch.randperm(pool, generator=gen, device=dev)[: case["seqs"]].to(torch.int32)
    elif case["initial"]:
        s["state"] = 0.3 * normal(case["seqs"], h, K, V)
        if case["packed"]:
            s["slots"] = torch.randperm(case["seqs"], generator=gen, device=dev).to(torch.int32)
    return s


# ------------------------------------------------------------ the plain forms
def _prefill_plain(s):
    case = s["case"]
    h, K, V = case["h"], case["k"], case["v"]
    group = h // case["hk"]
    dev = s["q"].device
    N, L = case["seqs"], -(-case["longest"] // CHUNK) * CHUNK
    nc = L // CHUNK
    t = torch.arange(L, device=dev)
    if case["packed"]:
        cu = s["cu_seqlens"].long()
        start, length = cu[:-1], cu[1:] - cu[:-1]
    else:
        start = torch.arange(N, device=dev) * case["longest"]
        length = torch.full((N,), case["longest"], device=dev)
    live = t[None, :] < length[:, None]                                      # [N, L]
    row = torch.where(live, start[:, None] + t, 0)

    def chunks(x, heads):                                                    # -> [nc, N, heads, 64, width]
        x = x.reshape(-1, heads, x.numel() // max(1, x.shape[0] * x.shape[1] * heads)).float()
        x = torch.where(live[:, :, None, None], x[row], 0.0)
        return x.reshape(N, nc, CHUNK, heads, -1).permute(1, 0, 3, 2, 4)

    q = chunks(s["q"], case["hk"]).repeat_interleave(group, dim=2)
    k = chunks(s["k"], case["hk"]).repeat_interleave(group, dim=2)
    v, beta, g = chunks(s["v"], h), chunks(s["beta"], h), chunks(s["g"], h)
    G = g.expand(*g.shape[:-1], K).cumsum(dim=3)
    mid, end = G[..., CHUNK // 2 - 1: CHUNK // 2, :], G[..., -1:, :]
    q = q * K ** -0.5
    cols = (k * torch.exp(mid - G)).transpose(-1, -2)
    up = torch.exp(G - mid)
    A = torch.tril(beta * ((k * up) @ cols), -1)
    P = torch.tril((q * up) @ cols)
    # (I + A)^-1 = (I - A)(I + A^2)(I + A^4) ..., exact since A^64 = 0
    M, Y = torch.eye(CHUNK, device=dev) - A, A @ A
    for _ in range(5):
        M, Y = M + M @ Y, Y @ Y
    M = M * beta.transpose(-1, -2)
    decay = torch.exp(G)
    kd, qd, ke = k * decay, q * decay, (k * torch.exp(end - G)).transpose(-1, -2)
    keep = torch.exp(end).transpose(-1, -2)                                  # [nc, N, h, K, 1]
    if "state" not in s:
        S = torch.zeros(N, h, K, V, device=dev)
    else:
        S = s["state"][s["slots"].long()] if "slots" in s else s["state"]
    o = torch.empty_like(v)
    for c in range(nc):
        u = M[c] @ (v[c] - kd[c] @ S)
        o[c] = qd[c] @ S + P[c] @ u
        S = keep[c] * S + ke[c] @ u
    o = o.permute(1, 0, 3, 2, 4).reshape(N, L, h, V).to(s["q"].dtype)
    out = torch.empty_like(s["v"])
    if case["packed"]:
        seq = torch.searchsorted(cu[1:], torch.arange(out.shape[1], device=dev), right=True)
        out[0] = o[seq, torch.arange(out.shape[1], device=dev) - start[seq]]
    else:
        out.copy_(o[:, : case["longest"]])
    if "slots" in s:
        s["state"][s["slots"].long()] = S
        S = s["state"]
    return out, S


def _step_plain(s):
    case = s["case"]
    group = case["h"] // case["hk"]
    at = s["slots"].long()
    q = s["q"].float().repeat_interleave(group, dim=1) * case["k"] ** -0.5
    k = s["k"].float().repeat_interleave(group, dim=1)
    g = s["g"] if case["gate"] == "channel" else s["g"][..., None]
    S = s["state"][at] * torch.exp(g)[..., None]
    u = s["beta"].float()[..., None] * (s["v"].float() - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    s["state"][at] = S
    return (S * q[..., None]).sum(-2).to(s["q"].dtype), s["state"]


def _norm(x, weight, eps=1e-6):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.float()


def run(s):
    case = s["case"]
    if own:
        import linear_attention_chunked_02_gb300 as kda
        if case["op"] == "add_norm":
            return kda.add_norm(s["x"], s["residual"], s["weight"], alpha=case["alpha"])
        if case["op"] == "gated_norm":
            return kda.gated_norm(s["x"], s["gate"], s["weight"], activation=case["act"])
        if case["op"] == "step":
            return kda.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"]), s["state"]
        pool = s["state"] if "slots" in s else None
        return kda.delta_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], cu_seqlens=s.get("cu_seqlens"),
                                 initial_state=s.get("state"), final_state=pool, slots=s.get("slots"))
    if case["op"] == "add_norm":
        r = s["residual"].float() + case["alpha"] * s["x"].float()
        return _norm(r, s["weight"]).to(s["x"].dtype), r.to(s["x"].dtype)
    if case["op"] == "gated_norm":
        gate = s["gate"].float()
        act = 1 / (1 + torch.exp(-gate))
        if case["act"] == "silu":
            act = gate * act
        return (_norm(s["x"].float(), s["weight"]) * act).to(s["x"].dtype)
    return _step_plain(s) if case["op"] == "step" else _prefill_plain(s)


# ------------------------------------------------- the definition in 64 bits
def _rule(S, q, k, v, g, beta):
    """One token of every sequence and head: the new state and the output (unscaled)."""
    S = S * g.exp().unsqueeze(-1)
    u = beta.unsqueeze(-1) * (v - torch.einsum("nhkv,nhk->nhv", S, k))
    S = S + torch.einsum("nhk,nhv->nhkv", k, u)
    return S, torch.einsum("nhkv,nhk->nhv", S, q)


def exact(case, seed):
    if case["op"] == "prefill":
        cost = case["seqs"] * case["h"] * case["k"] * case["v"] * 8 * 8 / 3e12 + 1.2e-4
        if cost * case["longest"] > 15:
            return None
    s = prepare(case, seed)
    if case["op"] == "add_norm":
        r = s["residual"].double() + case["alpha"] * s["x"].double()
        return r / (r.square().mean(-1, keepdim=True) + 1e-6).sqrt() * s["weight"].double(), r
    if case["op"] == "gated_norm":
        x, gate = s["x"].double(), s["gate"].double()
        y = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * s["weight"].double() * torch.sigmoid(gate)
        return y * gate if case["act"] == "silu" else y
    h, K = case["h"], case["k"]
    of = torch.arange(h, device=s["q"].device) // (h // case["hk"])          # key head of each head
    state = s["state"].double() if "state" in s else None
    slots = s["slots"].long() if "slots" in s else None

    def token(sel):
        """q, k, v, g, beta of the selected tokens in 64 bits; the decays are one per channel."""
        g = sel(s["g"]).double()
        g = g if case["gate"] == "channel" else g.unsqueeze(-1).expand(*g.shape, K)
        return sel(s["q"]).double()[:, of], sel(s["k"]).double()[:, of], sel(s["v"]).double(), g, sel(s["beta"]).double()

    if case["op"] == "step":
        new, o = _rule(state[slots], *token(lambda x: x))
        state[slots] = new
        return o / math.sqrt(K), state
    lens = _lengths(case)
    N = case["seqs"]
    o = torch.zeros(s["v"].shape, dtype=torch.float64, device=s["v"].device)
    flat = o.reshape(-1, *o.shape[2:])
    order = sorted(range(N), key=lambda n: -lens[n])                         # longest first: live ones stay a prefix
    first = [0] * N
    for n in range(1, N):
        first[n] = first[n - 1] + lens[n - 1]
    first_t = torch.tensor([first[n] for n in order], device=o.device)
    S = torch.zeros(N, h, K, case["v"], dtype=torch.float64, device=o.device)
    if state is not None:
        S += (state if slots is None else state[slots])[torch.tensor(order, device=o.device)]
    for t in range(max(lens)):
        m = sum(lens[n] > t for n in order)
        rows = first_t[:m] + t
        S[:m], flat[rows] = _rule(S[:m], *token(lambda x: x.reshape(-1, *x.shape[2:])[rows]))
    final = torch.empty_like(S)
    final[torch.tensor(order, device=o.device)] = S
    if slots is not None:
        state[slots] = final
        final = state
    return o / math.sqrt(K), final


def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] == "add_norm":
        n = case["rows"] * case["dim"]
        return {"bytes": 4 * n * b + case["dim"] * b, "flops": 6 * n}
    if case["op"] == "gated_norm":
        n = case["rows"] * case["h"] * case["dim"]
        return {"bytes": 3 * n * b + case["dim"] * b, "flops": 8 * n}
    h, hk, K, V = case["h"], case["hk"], case["k"], case["v"]
    tokens = case["seqs"] if case["op"] == "step" else sum(_lengths(case))
    gate = h * K if case["gate"] == "channel" else h
    io = tokens * (2 * hk * K * b + 2 * h * V * b + 4 * gate + h * b)
    states = case["seqs"] * h * K * V * 4
    if case["op"] == "step":
        return {"bytes": io + 2 * states + 4 * case["seqs"], "flops": 7 * tokens * h * K * V}
    # a chunk of n tokens: A, P (n n K each), the inverse (n n n / 3), K S and Q S (2 n K V), the two products
    # with the n x V updates (2 n n V) and the state's (n K V), at two operations each; products with
    # triangular matrices count half
    flops = 0
    for length in _lengths(case):
        for n in [CHUNK] * (length // CHUNK) + [length % CHUNK]:
            flops += h * (2 * n * n * K + 2 * n * n * n / 3 + 6 * n * K * V + 2 * n * n * V)
    return {"bytes": io + states * (2 if case["initial"] else 1), "flops": flops}
