"""The gated delta rule and the norm of heads, as measured cases.

Three operators, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and, with ``own`` set, as the calls a user makes:

  delta  the gated delta rule over prompts, batched or packed, with carried
         states: a = exp(dt A), S <- a S + beta (x - a S k) k^T, y = scale S q
         (x the values, B = k the keys, C = q the queries)
  step   the same recurrence at one token, states in a pool of slots
  heads  root-mean-square or Euclidean norm of each head of the queries and
         keys, and the rotation of their channels by the token's position

Tokens, heads and head sizes are those of the layers in ``ssd_inputs.CONFIGS``
(8 x 2048 tokens, 32 heads, head dimensions of 64 and states of 64, 128 and
256) or generic.
"""

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
CHUNK = 64


def listed():
    return [
        # a short question to one user: latency of one prompt of 37 tokens
        dict(name="delta-short-bf16", op="delta", io="bf16", dt="fp32", batch=1, L=37, H=32, P=128, N=128, G=16,
             seqs=0, init=False),
        # a batch of prompts, keys and queries shared by two heads each
        dict(name="delta-batch-bf16", op="delta", io="bf16", dt="bf16", batch=8, L=2048, H=32, P=128, N=128, G=16,
             seqs=0, init=False),
        # one long document: heads and value rows are all the parallelism there is
        dict(name="delta-long-bf16", op="delta", io="bf16", dt="bf16", batch=1, L=16384, H=32, P=128, N=128, G=16,
             seqs=0, init=True),
        # prompts of 37 requests packed back to back, some empty, some continued from a state
        dict(name="delta-packed-bf16", op="delta", io="bf16", dt="bf16", batch=1, L=8197, H=32, P=64, N=128, G=32,
             seqs=37, init=True),
        # a small layer in full precision, prompts of odd length
        dict(name="delta-ragged-fp32", op="delta", io="fp32", dt="fp32", batch=3, L=1001, H=32, P=64, N=64, G=32,
             seqs=0, init=True),
        # one user's next token
        dict(name="step-1-bf16", op="step", io="bf16", dt="bf16", batch=1, H=32, P=128, N=128, G=16, slots=4),
        # the next tokens of 37 requests of the small layer
        dict(name="step-37-fp32", op="step", io="fp32", dt="fp32", batch=37, H=32, P=64, N=64, G=32, slots=64),
        # the next tokens of 256 requests, their states in a pool of 320 slots
        dict(name="step-256-bf16", op="step", io="bf16", dt="bf16", batch=256, H=32, P=128, N=128, G=16, slots=320),
        # keys and queries of length one before the batched delta rule
        dict(name="heads-unit-bf16", op="heads", io="bf16", batch=8, L=2048, Hq=16, Hk=16, D=128, R=0, pairs=False,
             l2=True, weight=False, first=0),
        # queries and keys of a layer that goes by position, far into a document: norm, weights and rotation
        dict(name="heads-far-bf16", op="heads", io="bf16", batch=1, L=16384, Hq=32, Hk=8, D=128, R=128, pairs=False,
             l2=False, weight=True, first=1000000),
        # the same at one user's next token
        dict(name="heads-token-bf16", op="heads", io="bf16", batch=1, L=1, Hq=32, Hk=8, D=128, R=128, pairs=False,
             l2=False, weight=True, first=4095),
        # a ragged batch, heads of 80 channels, 32 of them rotated as neighbouring pairs
        dict(name="heads-part-fp32", op="heads", io="fp32", batch=3, L=1001, Hq=24, Hk=24, D=80, R=32, pairs=True,
             l2=False, weight=True, first=0),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "step", "heads"])
    io = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("delta", "step"):
        G = rng.choice([1, 2, 4, 8, 16, 32])
        H = G * rng.choice([1, 1, 2, 3, 4])
        P = rng.choice([64, 64, 128, 128, 16, 32, 96, 256, rng.randrange(1, 257)])
        N = rng.choice([64, 128, 128, 128, 32, 96, 256, rng.randrange(1, 257)])
        case = dict(op=op, io=io, dt=rng.choice([io, "fp32"]))
        if op == "step":
            batch = _spread(rng, 1, max(1, min(256, (1 << 27) // (H * P * N))))
            return dict(case, batch=batch, H=H, P=P, N=N, G=G, slots=batch + rng.randrange(0, 64))
        packed = rng.random() < 0.4
        batch = 1 if packed else _spread(rng, 1, 16)
        # the largest listed case's state updates and tokens times heads, in fp32 at most a quarter of the updates
        most = max(1, min(16384, (1 << (31 if io == "fp32" else 33)) // (batch * H * P * N), (1 << 19) // (batch * H)))
        return dict(case, batch=batch, L=_spread(rng, 1, most), H=H, P=P, N=N, G=G,
                    seqs=_spread(rng, 1, 64) if packed else 0, init=rng.random() < 0.5)
    Hk = _spread(rng, 1, 32)
    Hq = Hk * rng.choice([1, 1, 2, 4])
    D = rng.choice([64, 128, 128, 80, 96, 192, 256, rng.randrange(1, 257)])
    R = rng.choice([0, D // 2 * 2, D // 4 * 2])
    batch = _spread(rng, 1, 16)
    L = _spread(rng, 1, max(1, min(16384, (1 << 26) // (batch * (Hq + Hk) * D))))
    return dict(op=op, io=io, batch=batch, L=L, Hq=Hq, Hk=Hk, D=D, R=R, pairs=rng.random() < 0.5, l2=rng.random() < 0.4,
                weight=rng.random() < 0.6, first=rng.choice([0, 0, 511, 100000, 4000000]))


def _lengths(case, seed):
    """Token counts of the packed requests: ragged, an empty and a one-token
    one among them where there is room, together all of the tokens."""
    r = random.Random(seed * 1009 + 7)
    cuts = sorted(r.randrange(0, case["L"] + 1) for _ in range(case["seqs"] - 1))
    if len(cuts) >= 4:
        cuts[1] = cuts[0]
        cuts[3] = min(cuts[2] + 1, case["L"])
    return sorted([0] + cuts + [case["L"]])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    io = TYPES[case["io"]]
    op = case["op"]

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    s = dict(case=dict(case))
    b = case["batch"]
    if op == "heads":
        L, Hq, Hk, D, R = (case[k] for k in ("L", "Hq", "Hk", "D", "R"))
        # queries and keys lie behind one another in a projection's output
        qk = normal(b, L, (Hq + Hk) * D, dtype=io)
        s.update(q=qk[..., :Hq * D].unflatten(-1, (Hq, D)), k=qk[..., Hq * D:].unflatten(-1, (Hk, D)),
                 wq=1.0 + normal(D, scale=0.2) if case["weight"] else None,
                 wk=1.0 + normal(D, scale=0.2) if case["weight"] else None, positions=None, freq=None)
        if R:
            # every row of the batch at a place of its own in its document
            start = (uniform(b, 1) * 64).to(torch.int32) + case["first"]
            s["positions"] = start + torch.arange(L, device=DEV, dtype=torch.int32)
            s["freq"] = torch.exp(torch.arange(R // 2, device=DEV) * (-2.0 * math.log(10000.0) / R))
        return s
    H, P, N, G = (case[k] for k in ("H", "P", "N", "G"))
    lead = (b, case["L"]) if op == "delta" else (b,)
    dtt = TYPES[case["dt"]]
    # keys and queries of length one, behind one another in a buffer
    bc = normal(*lead, 2 * G, N)
    bc = (bc / torch.sqrt((bc * bc).sum(-1, keepdim=True) + EPS)).to(io)
    s.update(x=normal(*lead, H, P, dtype=io), B=bc[..., :G, :], C=bc[..., G:, :],
             dt=normal(*lead, H, dtype=dtt, scale=0.5), beta=normal(*lead, H, dtype=dtt),
             A=-torch.exp(uniform(H) * math.log(16.0)), scale=N ** -0.5,
             # steps of 0.001 to 0.1 after the softplus, spread over their logarithm
             bias=torch.log(torch.expm1(torch.exp(uniform(H) * math.log(100.0) + math.log(1e-3)))))
    if op == "step":
        s["state"] = normal(case["slots"], H, P, N, scale=0.3)
        s["slots"] = torch.randperm(case["slots"], generator=g, device=DEV)[:b].to(torch.int32)
        return s
    cuts = _lengths(case, seed) if case["seqs"] else [i * case["L"] for i in range(b + 1)]
    s["init"] = normal(len(cuts) - 1, H, P, N, scale=0.3) if case["init"] else None
    s["cuts"] = cuts  # the scheduler's own list of where each request begins
    if case["seqs"]:
        s["cu"] = torch.tensor(cuts, dtype=torch.int32, device=DEV)
    return s


# ---- plain forms ---------------------------------------------------------------


def _steps(s):
    """log of the decay (64 bits: it is summed over tokens) and beta."""
    v = s["dt"].float() + s["bias"]
    dt = torch.where(v > 20.0, v, torch.log1p(torch.exp(v)))
    return dt.double() * s["A"].double(), 1.0 / (1.0 + torch.exp(-s["beta"].float()))


def _plain_delta(s):
    c = s["case"]
    H, P, N, G = (c[k] for k in ("H", "P", "N", "G"))
    cuts = s["cuts"]
    n = len(cuts) - 1
    logs, beta = _steps(s)
    # chunks of every sequence, the last one padded with tokens that do nothing
    chunks = [-(-(e - a) // CHUNK) for a, e in zip(cuts, cuts[1:])]
    first = [0]
    for k in chunks:
        first.append(first[-1] + k)
    cu = torch.tensor(cuts, device=DEV)
    base = torch.tensor(first, device=DEV)
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), torch.tensor(chunks, device=DEV))
    at = (cu[seq] + (torch.arange(first[-1], device=DEV) - base[seq]) * CHUNK).unsqueeze(1) + torch.arange(CHUNK, device=DEV)
    inside = at < cu[seq + 1].unsqueeze(1)
    at = at.clamp(max=cuts[-1] - 1)

    def take(t):
        v = t.flatten(0, 1)[at].transpose(1, 2)  # [chunks, heads, CHUNK, ..]
        m = inside.view(inside.shape[0], 1, CHUNK, *[1] * (v.dim() - 3))
        return torch.where(m, v, torch.zeros((), dtype=v.dtype, device=DEV))

    k, q = take(s["B"].float()), take(s["C"].float())
    g, beta = take(logs).cumsum(2), take(beta)
    lower = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=DEV).tril()
    decay = torch.exp(torch.where(lower, g.unsqueeze(3) - g.unsqueeze(2), -math.inf).float())
    per = H // G
    share = lambda t: t.repeat_interleave(per, 1)  # noqa: E731
    kt = k.transpose(2, 3)
    A = share(k @ kt) * decay * beta.unsqueeze(3)
    att = share(q @ kt) * decay
    k, q = share(k), share(q)
    # (1 + strictly lower part of A)^-1, row after row
    T = torch.eye(CHUNK, device=DEV).repeat(*A.shape[:2], 1, 1)
    for i in range(1, CHUNK):
        T[:, :, i, :i] = -(A[:, :, i:i + 1, :i] @ T[:, :, :i, :i]).squeeze(2)
    eg = torch.exp(g).float().unsqueeze(3)
    U = T @ (beta.unsqueeze(3) * take(s["x"].float()))
    W = T @ (beta.unsqueeze(3) * eg * k)
    q = q * eg
    kend = k * torch.exp(g[:, :, -1:] - g).float().unsqueeze(3)
    S = torch.zeros((n, H, P, N), device=DEV) if s["init"] is None else s["init"].clone()
    y = torch.zeros((cuts[-1], H, P), device=DEV)
    for step in range(max(chunks, default=0)):
        live = [i for i in range(n) if chunks[i] > step]
        rows = torch.tensor(live, device=DEV)
        j = base[rows] + step
        St = S[rows].transpose(2, 3)
        Uj = U[j] - W[j] @ St
        o = (q[j] @ St + att[j] @ Uj).transpose(1, 2)
        m = inside[j]
        y[at[j][m]] = o[m]
        S[rows] = S[rows] * eg[j][:, :, -1:] + Uj.transpose(2, 3) @ kend[j]
    return (y * s["scale"]).to(s["x"].dtype).view(s["x"].shape), S


def _plain_step(s):
    per = s["case"]["H"] // s["case"]["G"]
    logs, beta = _steps(s)
    k, q = (s[n].float().repeat_interleave(per, 1).unsqueeze(2) for n in "BC")
    slots = s["slots"].long()
    S = s["state"][slots] * torch.exp(logs).float()[..., None, None]
    u = beta.unsqueeze(2) * (s["x"].float() - (S * k).sum(-1))
    S = S + u.unsqueeze(3) * k
    s["state"][slots] = S
    return ((S * q).sum(-1) * s["scale"]).to(s["x"].dtype), s["state"]


def _plain_heads(s):
    c = s["case"]
    R = c["R"]
    if R:
        # 64 bits: positions in the millions leave 32 no digits of the angle
        angle = s["positions"].double().unsqueeze(-1) * s["freq"].double()
        cos, sin = torch.cos(angle).float().unsqueeze(2), torch.sin(angle).float().unsqueeze(2)
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        v = x.float()
        sq = v * v
        v = v / torch.sqrt((sq.sum(-1, keepdim=True) if c["l2"] else sq.mean(-1, keepdim=True)) + EPS)
        if w is not None:
            v = v * w
        if R:
            a, b = (v[..., 0:R:2], v[..., 1:R:2]) if c["pairs"] else (v[..., :R // 2], v[..., R // 2:R])
            turned = [a * cos - b * sin, b * cos + a * sin]
            turned = torch.stack(turned, -1).flatten(-2) if c["pairs"] else torch.cat(turned, -1)
            v = torch.cat([turned, v[..., R:]], -1)
        out.append(v.to(x.dtype))
    return out


# ---- the framework's calls -------------------------------------------------------


def _own(s):
    import mamba_ssd_scan_fwd_amd as ssd

    c = s["case"]
    if c["op"] == "heads":
        return ssd.head_norm(s["q"], s["k"], s["wq"], s["wk"], positions=s["positions"], inv_freq=s["freq"], eps=EPS,
                             l2=c["l2"], pairs=c["pairs"])
    more = dict(scale=s["scale"], beta_sigmoid=True, dt_pre=dict(bias=s["bias"], softplus=True))
    if c["op"] == "step":
        y = ssd.delta_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["beta"], s["state"], state_slots=s["slots"], **more)
        return y, s["state"]
    if c["seqs"]:
        return ssd.delta_rule_varlen(s["x"], s["dt"], s["A"], s["B"], s["C"], s["beta"], cu_seqlens=s["cu"],
                                     init_states=s["init"], **more)
    return ssd.delta_rule(s["x"], s["dt"], s["A"], s["B"], s["C"], s["beta"], s["init"], **more)


def run(state):
    if own:
        return _own(state)
    return dict(delta=_plain_delta, step=_plain_step, heads=_plain_heads)[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------


def work(case):
    io = 2 if case["io"] == "bf16" else 4
    if case["op"] == "heads":
        tokens = case["batch"] * case["L"]
        each = tokens * (case["Hq"] + case["Hk"]) * case["D"]
        return {"bytes": 2 * each * io + (tokens * 4 if case["R"] else 0), "flops": 8 * each}
    tokens = case["batch"] * case.get("L", 1)
    H, P, N, G = (case[k] for k in ("H", "P", "N", "G"))
    dt = 2 if case["dt"] == "bf16" else 4
    moved = tokens * ((2 * H * P + 2 * G * N) * io + 2 * H * dt) + H * 8
    states = case["batch"] * 2 if case["op"] == "step" else (case["seqs"] or case["batch"]) * (2 if case["init"] else 1)
    # S k, S q and the update, a product and a sum each for every entry of the state
    return {"bytes": moved + states * H * P * N * 4, "flops": 6 * tokens * H * P * N}


# ---- the definitions in 64 bits -----------------------------------------------------


def _exact_recurrence(s, x, a, beta, k, q, S):
    """x [n, L, H, P], a, beta [n, L, H], k, q [n, L, G, N], S [n, H, P, N]: token after token."""
    c = s["case"]
    n, L = x.shape[:2]
    G, N = c["G"], c["N"]
    S = S.reshape(n, G, -1, c["P"], N).clone()
    y = torch.empty((n, L, G, c["H"] // G, c["P"]), dtype=torch.float64, device=DEV)
    for t in range(L):
        kt, qt = k[:, t].view(n, G, 1, N, 1), q[:, t].view(n, G, 1, N, 1)
        S *= a[:, t].view(n, G, -1, 1, 1)
        u = beta[:, t].view(n, G, -1, 1) * (x[:, t].view(n, G, -1, c["P"]) - torch.matmul(S, kt).squeeze(-1))
        S += u.unsqueeze(-1) * kt.transpose(-1, -2)
        y[:, t] = torch.matmul(S, qt).squeeze(-1)
    return y.view(x.shape) * s["scale"], S.view(n, c["H"], c["P"], N)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "heads":
        out = []
        for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
            v = x.double()
            norm = torch.linalg.vector_norm(v, dim=-1, keepdim=True).square()
            v = v * torch.rsqrt((norm if case["l2"] else norm / case["D"]) + EPS)
            v = v if w is None else v * w.double()
            R = case["R"]
            if R:
                turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                                   s["positions"].double()[..., None] * s["freq"].double())[:, :, None]
                pairs = v[..., :R].unflatten(-1, (R // 2, 2) if case["pairs"] else (2, R // 2))
                if not case["pairs"]:
                    pairs = pairs.transpose(-1, -2)
                done = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
                if not case["pairs"]:
                    done = done.transpose(-1, -2)
                v = torch.cat([done.flatten(-2), v[..., R:]], -1)
            out.append(v)
        return out
    x, k, q = s["x"].double(), s["B"].double(), s["C"].double()
    # log(1 + e^v), without loss for small e^v
    dt = torch.logaddexp(s["dt"].double() + s["bias"].double(), torch.zeros((), dtype=torch.float64, device=DEV))
    a, beta = torch.exp(dt * s["A"].double()), torch.sigmoid(s["beta"].double())
    if case["op"] == "step":
        at = s["slots"].long()
        state = s["state"].double()
        y, S = _exact_recurrence(s, x[:, None], a[:, None], beta[:, None], k[:, None], q[:, None], state[at])
        state[at] = S
        return y[:, 0], state
    n = case["seqs"] or case["batch"]
    S0 = torch.zeros((n, case["H"], case["P"], case["N"]), dtype=torch.float64, device=DEV)
    if s["init"] is not None:
        S0 = s["init"].double()
    if not case["seqs"]:
        return _exact_recurrence(s, x, a, beta, k, q, S0)
    parts = [_exact_recurrence(s, *(t[:, f:e] for t in (x, a, beta, k, q)), S0[i:i + 1])
             for i, (f, e) in enumerate(zip(s["cuts"], s["cuts"][1:]))]
    return torch.cat([p[0] for p in parts], 1), torch.cat([p[1] for p in parts])
