"""The layer operators around the state-space scan, as measured cases.

Five operators, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and, with ``own`` set, as the calls a user makes:

  scan       selective scan over prompts: a decay per channel and state,
             batched or packed, with gate, skip term and carried states
  step       the same recurrence at one token, states in a pool of slots
  conv       short causal convolution over prompts, batched or packed
  conv_step  the same at one token, its state rolled in place
  norm       group norm over the channels of each token, gated by silu(z)

Channel counts are those of the layers in ``ssd_inputs.CONFIGS`` (32 x 64,
64 x 64 and 128 x 64 channels; 64 x 64 + 2 x 128 convolved channels) or
generic; 16 states per channel is the usual size of the selective scan.
"""

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # a short question to one user: latency of one prompt of 37 tokens
        dict(name="scan-short-fp32", op="scan", io="fp32", dt="fp32", batch=1, L=37, E=2048, N=16, G=1, seqs=0,
             gate=False, init=False),
        # a batch of prompts, the training-length layer of 64 x 64 channels
        dict(name="scan-batch-bf16", op="scan", io="bf16", dt="bf16", batch=8, L=2048, E=4096, N=16, G=1,
             seqs=0, gate=True, init=False),
        # one long document: the time axis is all the parallelism there is
        dict(name="scan-long-bf16", op="scan", io="bf16", dt="bf16", batch=1, L=16384, E=4096, N=16, G=1,
             seqs=0, gate=True, init=True),
        # prompts of 37 requests packed back to back, some empty, some continued from a state
        dict(name="scan-packed-bf16", op="scan", io="bf16", dt="bf16", batch=1, L=8197, E=2048, N=16, G=1,
             seqs=37, gate=True, init=True),
        # one user's next token
        dict(name="step-1-bf16", op="step", io="bf16", dt="bf16", batch=1, E=4096, N=16, G=1, slots=4, gate=True),
        # the next tokens of 256 requests, their states in a pool of 320 slots
        dict(name="step-256-bf16", op="step", io="bf16", dt="bf16", batch=256, E=8192, N=16, G=1, slots=320,
             gate=True),
        # the convolution before the batched scan: the x half of the input projection
        dict(name="conv-batch-bf16", op="conv", io="bf16", batch=8, L=2048, H=0, P=0, G=0, N=0, CH=4096, K=4,
             seqs=0, init=False),
        # the x | B | C channels of 37 packed requests, split for the packed scan
        dict(name="conv-packed-bf16", op="conv", io="bf16", batch=1, L=8197, H=64, P=64, G=1, N=128, CH=4352,
             K=4, seqs=37, init=True),
        # one user's next token, split into x, B and C
        dict(name="conv-step-1-bf16", op="conv_step", io="bf16", batch=1, H=64, P=64, G=1, N=128, CH=4352, K=4,
             slots=4),
        # the next tokens of 256 requests
        dict(name="conv-step-256-bf16", op="conv_step", io="bf16", batch=256, H=0, P=0, G=0, N=0, CH=8192, K=4,
             slots=320),
        # after the batched scan: root mean square over all channels, gate first
        dict(name="norm-batch-bf16", op="norm", io="bf16", rows=16384, C=4096, G=1, center=False, gate_first=True),
        # a ragged batch with one norm per head, centred, gate last
        dict(name="norm-heads-fp32", op="norm", io="fp32", rows=1001, C=8192, G=128, center=True, gate_first=False),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "step", "conv", "conv_step", "norm"])
    io = rng.choice(["bf16", "bf16", "fp32"])
    if op == "scan":
        G = rng.choice([1, 1, 2, 4])
        N = rng.choice([16, 16, 16, 8, 13, 32, 64, 128])
        E = G * _spread(rng, max(1, 64 // G), 8192 // G)
        packed = rng.random() < 0.4
        batch = 1 if packed else _spread(rng, 1, 16)
        # at most half the state updates of the largest listed case
        most = max(1, min(32768, (1 << 29) // (batch * E * N)))
        L = _spread(rng, 1, most)
        return dict(op=op, io=io, dt=rng.choice([io, "fp32"]), batch=batch, L=L, E=E, N=N, G=G, seqs=_spread(rng, 1, 64) if packed else 0,
                    gate=rng.random() < 0.7, init=rng.random() < 0.5)
    if op == "step":
        batch = _spread(rng, 1, 256)
        G = rng.choice([1, 1, 2, 4])
        return dict(op=op, io=io, dt=rng.choice([io, "fp32"]), batch=batch, E=G * _spread(rng, max(1, 64 // G), 8192 // G),
                    N=rng.choice([16, 16, 16, 8, 13]), G=G, slots=batch + rng.randrange(0, 64), gate=rng.random() < 0.7)
    if op in ("conv", "conv_step"):
        split = rng.random() < 0.5
        H, P, G, N = (rng.choice([4, 32, 64, 128]), rng.choice([32, 64]), rng.choice([1, 2, 4]),
                      rng.choice([16, 64, 128])) if split else (0, 0, 0, 0)
        CH = H * P + 2 * G * N if split else _spread(rng, 16, 8192)
        K = rng.choice([4, 4, 3, 2])
        if op == "conv_step":
            batch = _spread(rng, 1, 256)
            return dict(op=op, io=io, batch=batch, H=H, P=P, G=G, N=N, CH=CH, K=K, slots=batch + rng.randrange(0, 64))
        packed = split or rng.random() < 0.4
        batch = 1 if packed else _spread(rng, 1, 16)
        L = _spread(rng, 1, max(1, min(32768, (1 << 26) // (batch * CH * (2 if io == "fp32" else 1)))))
        return dict(op=op, io=io, batch=batch, L=L, H=H, P=P, G=G, N=N, CH=CH, K=K,
                    seqs=_spread(rng, 1, 64) if packed else 0, init=rng.random() < 0.5)
    G = rng.choice([1, 1, 2, 8, 32])
    C = G * _spread(rng, max(1, 64 // G), 8192 // G)
    return dict(op=op, io=io, rows=_spread(rng, 1, (1 << 25) // C), C=C, G=G, center=rng.random() < 0.5,
                gate_first=rng.random() < 0.5)


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
    if op in ("scan", "step"):
        b, E, N, G = case["batch"], case["E"], case["N"], case["G"]
        lead = (b, case["L"]) if op == "scan" else (b,)
        # x is the first half of a buffer that holds z as its second, B and C
        # lie behind one another in another: views, as projections leave them
        xz = normal(*lead, 2 * E, dtype=io)
        bc = normal(*lead, 2 * G * N, dtype=io, scale=N ** -0.5)
        s.update(x=xz[..., :E], z=xz[..., E:] if case["gate"] else None,
                 B=bc[..., :G * N].unflatten(-1, (G, N)), C=bc[..., G * N:].unflatten(-1, (G, N)),
                 dt=normal(*lead, E, dtype=TYPES[case["dt"]], scale=0.5),
                 A=-torch.exp(uniform(E, N) * math.log(16.0)), D=normal(E),
                 # steps of 0.001 to 0.1 after the softplus, spread over their logarithm
                 bias=torch.log(torch.expm1(torch.exp(uniform(E) * math.log(100.0) + math.log(1e-3)))))
        if op == "scan":
            n = case["seqs"] or b
            s["init"] = normal(n, E, N, scale=0.3) if case["init"] else None
        else:
            s["state"] = normal(case["slots"], E, N, scale=0.3)
            s["slots"] = torch.randperm(case["slots"], generator=g, device=DEV)[:b].to(torch.int32)
    elif op in ("conv", "conv_step"):
        b, CH, K = case["batch"], case["CH"], case["K"]
        lead = (b, case["L"]) if op == "conv" else (b,)
        # a plain input is half of a wider buffer; packed x | B | C rows stand alone
        s.update(x=normal(*lead, CH, dtype=io) if case["H"] else normal(*lead, 2 * CH, dtype=io)[..., :CH],
                 w=normal(CH, K, scale=K ** -0.5), bias=normal(CH, scale=0.1))
        if op == "conv":
            s["init"] = normal(case["seqs"] or b, CH, K - 1) if case["init"] else None
        else:
            s["state"] = normal(case["slots"], CH, K - 1)
            s["slots"] = torch.randperm(case["slots"], generator=g, device=DEV)[:b].to(torch.int32)
    else:
        R, C = case["rows"], case["C"]
        s.update(x=normal(R, C, dtype=io) + 0.5, z=normal(R, 2 * C, dtype=io)[:, C:], w=1.0 + normal(C, scale=0.2),
                 bias=normal(C, scale=0.2) if case["center"] else None)
    if case.get("seqs"):
        s["cu"] = torch.tensor(_lengths(case, seed), dtype=torch.int32, device=DEV)
    return s


# ---- plain forms ---------------------------------------------------------------


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(v)))


def _sequence_of(cu, T):
    """For each token of a packed stream its sequence and whether it starts it."""
    t = torch.arange(T, device=cu.device, dtype=cu.dtype)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq, cu[seq].eq(t)


def _plain_scan(s):
    c = s["case"]
    x, B, C = s["x"].float(), s["B"].float(), s["C"].float()
    b, L, E = x.shape
    per = E // c["G"]
    dt = _softplus(s["dt"].float() + s["bias"])
    B, C = B.repeat_interleave(per, 2), C.repeat_interleave(per, 2)
    decay = torch.exp(dt.unsqueeze(-1) * s["A"])
    h = (dt * x).unsqueeze(-1) * B
    init = s["init"]
    if c["seqs"]:
        seq, start = _sequence_of(s["cu"], L)
        if init is not None:
            h += torch.where(start.view(1, L, 1, 1), decay * init[seq].unsqueeze(0), torch.zeros((), device=DEV))
        decay = torch.where(start.view(1, L, 1, 1), torch.zeros((), device=DEV), decay)
    elif init is not None:
        h[:, 0] += decay[:, 0] * init
    # the recurrence in log2(L) doublings: after the step of offset k, every
    # h holds the last 2k tokens' sum and every decay their product
    k = 1
    while k < L:
        h = torch.cat([h[:, :k], torch.addcmul(h[:, k:], decay[:, k:], h[:, :-k])], 1)
        if 2 * k < L:
            decay = torch.cat([decay[:, :k], decay[:, k:] * decay[:, :-k]], 1)
        k *= 2
    if c["seqs"]:
        lens = s["cu"][1:] - s["cu"][:-1]
        last = h[0, (s["cu"][1:].long() - 1).clamp(min=0)]
        before = init if init is not None else torch.zeros_like(last)
        final = torch.where(lens.view(-1, 1, 1) > 0, last, before)
    else:
        final = h[:, -1].clone()
    y = (h * C).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(s["x"].dtype), final


def _plain_step(s):
    per = s["case"]["E"] // s["case"]["G"]
    x = s["x"].float()
    dt = _softplus(s["dt"].float() + s["bias"]).unsqueeze(-1)
    B, C = s["B"].float().repeat_interleave(per, 1), s["C"].float().repeat_interleave(per, 1)
    slots = s["slots"].long()
    h = s["state"][slots] * torch.exp(dt * s["A"]) + dt * x.unsqueeze(-1) * B
    s["state"][slots] = h
    y = (h * C).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(s["x"].dtype), s["state"]


def _split(s, y):
    c = s["case"]
    if not c["H"]:
        return [y]
    cut = c["H"] * c["P"]
    n = c["G"] * c["N"]
    return [y[..., :cut].unflatten(-1, (c["H"], c["P"])).contiguous(),
            y[..., cut:cut + n].unflatten(-1, (c["G"], c["N"])).contiguous(),
            y[..., cut + n:].unflatten(-1, (c["G"], c["N"])).contiguous()]


def _plain_conv(s):
    c = s["case"]
    K, L = c["K"], c["L"]
    x = s["x"].float()
    back = torch.arange(K, device=DEV) - (K - 1)
    at = torch.arange(L, device=DEV).unsqueeze(1) + back
    init = s["init"]
    if c["seqs"]:
        seq, _ = _sequence_of(s["cu"], L)
        first = s["cu"][seq].long().unsqueeze(1)
        ends = s["cu"][1:].long().unsqueeze(1)
        begins = s["cu"][:-1].long().unsqueeze(1)
    else:
        first = torch.zeros((1, 1), dtype=torch.long, device=DEV)
    inside = at >= first
    taps = torch.where(inside.unsqueeze(-1), x[:, at.clamp(min=0)], torch.zeros((), device=DEV))
    if init is not None:
        # position of each tap before the sequence's start in its carried state
        j = (at - first + K - 1).clamp(0, max(K - 2, 0))
        if c["seqs"]:
            old = init[seq].permute(0, 2, 1).gather(1, j.unsqueeze(-1).expand(-1, -1, c["CH"])).unsqueeze(0)
        else:
            old = init.permute(0, 2, 1)[:, j]
        taps = torch.where(inside.unsqueeze(-1), taps, old)
    y = _silu((taps * s["w"].t()).sum(2) + s["bias"])
    # the last K - 1 inputs of every sequence, older ones from its carried state
    tail = torch.arange(K - 1, device=DEV) - (K - 1)
    if c["seqs"]:
        p = ends + tail
        new = x[0, p.clamp(min=0)].permute(0, 2, 1)
        q = (p - begins + K - 1).clamp(0, max(K - 2, 0))
        keep = (p >= begins).unsqueeze(1)
        n = c["seqs"]
        old = torch.zeros((n, c["CH"], K - 1), device=DEV) if init is None else init.gather(2, q.unsqueeze(1).expand(-1, c["CH"], -1))
    else:
        p = (L + tail).unsqueeze(0)
        new = x[:, p[0].clamp(min=0)].permute(0, 2, 1)
        q = (p[0] + K - 1).clamp(0, max(K - 2, 0))
        keep = (p >= 0).unsqueeze(1)
        old = torch.zeros_like(new) if init is None else init[:, :, q]
    return _split(s, y.to(s["x"].dtype)) + [torch.where(keep, new, old)]


def _plain_conv_step(s):
    slots = s["slots"].long()
    window = torch.cat([s["state"][slots], s["x"].float().unsqueeze(-1)], -1)
    y = _silu((window * s["w"]).sum(-1) + s["bias"])
    s["state"][slots] = window[..., 1:]
    return _split(s, y.to(s["x"].dtype)) + [s["state"]]


def _plain_norm(s):
    c = s["case"]
    v = s["x"].float()
    gate = _silu(s["z"].float())
    if c["gate_first"]:
        v = v * gate
    v = v.unflatten(-1, (c["G"], c["C"] // c["G"]))
    if c["center"]:
        v = v - v.mean(-1, keepdim=True)
    v = (v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)).flatten(-2) * s["w"]
    if s["bias"] is not None:
        v = v + s["bias"]
    if not c["gate_first"]:
        v = v * gate
    return v.to(s["x"].dtype)


# ---- the framework's calls -------------------------------------------------------


def _own(s):
    import mamba_ssd_scan_fwd_amd as ssd

    c = s["case"]
    op = c["op"]
    if op == "scan":
        pre = dict(bias=s["bias"], softplus=True)
        if c["seqs"]:
            return ssd.selective_scan_varlen(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"],
                                             cu_seqlens=s["cu"], init_states=s["init"], dt_pre=pre)
        return ssd.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["init"], dt_pre=pre)
    if op == "step":
        y = ssd.selective_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["state"],
                               state_slots=s["slots"], dt_pre=dict(bias=s["bias"], softplus=True))
        return y, s["state"]
    if op == "conv":
        last = torch.empty((c["seqs"] or c["batch"], c["CH"], c["K"] - 1), device=DEV)
        heads = dict(nheads=c["H"], headdim=c["P"], ngroups=c["G"], dstate=c["N"])
        if c["H"]:
            out = ssd.conv1d_split_varlen(s["x"], s["w"], s["bias"], cu_seqlens=s["cu"], conv_states_in=s["init"],
                                          conv_states_out=last, **heads)
            return [*out, last]
        if c["seqs"]:
            y = ssd.conv1d_varlen(s["x"], s["w"], s["bias"], cu_seqlens=s["cu"], conv_states_in=s["init"],
                                  conv_states_out=last)
        else:
            y = ssd.conv1d(s["x"], s["w"], s["bias"], conv_state_in=s["init"], conv_state_out=last)
        return [y, last]
    if op == "conv_step":
        if c["H"]:
            out = ssd.conv1d_split_step(s["x"], s["w"], s["bias"], s["state"], state_slots=s["slots"], nheads=c["H"],
                                        headdim=c["P"], ngroups=c["G"], dstate=c["N"])
            return [*out, s["state"]]
        return [ssd.conv1d_step(s["x"], s["w"], s["bias"], s["state"], state_slots=s["slots"]), s["state"]]
    return ssd.group_norm(s["x"], s["w"], s["bias"], s["z"], ngroups=c["G"], eps=EPS, center=c["center"],
                          gate_first=c["gate_first"])


def run(state):
    if own:
        return _own(state)
    return dict(scan=_plain_scan, step=_plain_step, conv=_plain_conv, conv_step=_plain_conv_step,
                norm=_plain_norm)[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------


def work(case):
    io = 2 if case["io"] == "bf16" else 4
    op = case["op"]
    if op in ("scan", "step"):
        tokens = case["batch"] * case.get("L", 1)
        E, N, G = case["E"], case["N"], case["G"]
        dt = 2 if case["dt"] == "bf16" else 4
        moved = tokens * ((E * (3 if case["gate"] else 2) + 2 * G * N) * io + E * dt) + E * (N + 2) * 4
        states = case["batch"] * 2 if op == "step" else (case["seqs"] or case["batch"]) * (2 if case["init"] else 1)
        # exp, three products and two sums for each state of each token
        return {"bytes": moved + states * E * N * 4, "flops": 6 * tokens * E * N}
    if op in ("conv", "conv_step"):
        tokens = case["batch"] * case.get("L", 1)
        CH, K = case["CH"], case["K"]
        states = case["batch"] * 2 if op == "conv_step" else (case["seqs"] or case["batch"]) * (2 if case["init"] else 1)
        return {"bytes": tokens * CH * 2 * io + CH * (K + 1) * 4 + states * CH * (K - 1) * 4,
                "flops": tokens * CH * (2 * K + 4)}
    R, C = case["rows"], case["C"]
    return {"bytes": R * C * 3 * io + C * (8 if case["center"] else 4), "flops": R * C * 10}


# ---- the definitions in 64 bits -----------------------------------------------------


def _gate64(z):
    return z * torch.sigmoid(z)


def _exact_recurrence(s, x, dt, B, C, h):
    """x, dt [n, L, E], B, C [n, L, G, N], h [n, E, N]: token after token."""
    c = s["case"]
    n, L, E = x.shape
    A = s["A"].double().view(c["G"], -1, c["N"])
    h = h.view(n, c["G"], E // c["G"], c["N"]).clone()
    y = torch.empty((n, L, c["G"], E // c["G"]), dtype=torch.float64, device=DEV)
    for t in range(L):
        d = dt[:, t].view(n, c["G"], -1, 1)
        h = h * torch.exp(d * A) + d * x[:, t].view(n, c["G"], -1, 1) * B[:, t].unsqueeze(2)
        y[:, t] = (h * C[:, t].unsqueeze(2)).sum(-1)
    return y.view(n, L, E) + s["D"].double() * x, h.reshape(n, E, c["N"])


def _exact_conv(s, x, state):
    """x [n, L, CH] after state [n, CH, K - 1]: one tap at a time."""
    K = s["case"]["K"]
    L = x.shape[1]
    line = torch.cat([state.transpose(1, 2), x], 1)
    z = s["bias"].double().expand_as(x)
    for k in range(K):
        z = z + line[:, k:k + L] * s["w"][:, k].double()
    return _gate64(z), line[:, L:].transpose(1, 2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    x = s["x"].double()
    cu = s["cu"].tolist() if "cu" in s else None
    if op in ("scan", "step"):
        # log(1 + e^v), without loss for small e^v
        dt = torch.logaddexp(s["dt"].double() + s["bias"].double(), torch.zeros((), dtype=torch.float64, device=DEV))
        B, C = s["B"].double(), s["C"].double()
        if op == "step":
            at = s["slots"].long()
            y, h = _exact_recurrence(s, x[:, None], dt[:, None], B[:, None], C[:, None], s["state"][at].double())
            state = s["state"].double()
            state[at] = h
            y, h = y[:, 0], state
        else:
            n = case["seqs"] or case["batch"]
            h0 = torch.zeros((n, case["E"], case["N"]), dtype=torch.float64, device=DEV)
            if s["init"] is not None:
                h0 = s["init"].double()
            if cu is None:
                y, h = _exact_recurrence(s, x, dt, B, C, h0)
            else:
                parts = [_exact_recurrence(s, x[:, a:b], dt[:, a:b], B[:, a:b], C[:, a:b], h0[i:i + 1])
                         for i, (a, b) in enumerate(zip(cu, cu[1:]))]
                y, h = torch.cat([p[0] for p in parts], 1), torch.cat([p[1] for p in parts])
        return (y * _gate64(s["z"].double()) if s["z"] is not None else y), h
    if op in ("conv", "conv_step"):
        if op == "conv_step":
            at = s["slots"].long()
            y, last = _exact_conv(s, x[:, None], s["state"][at].double())
            y = y[:, 0]
            state = s["state"].double()
            state[at] = last
            last = state
        else:
            n = case["seqs"] or case["batch"]
            before = torch.zeros((n, case["CH"], case["K"] - 1), dtype=torch.float64, device=DEV)
            if s["init"] is not None:
                before = s["init"].double()
            if cu is None:
                y, last = _exact_conv(s, x, before)
            else:
                parts = [_exact_conv(s, x[:, a:b], before[i:i + 1]) for i, (a, b) in enumerate(zip(cu, cu[1:]))]
                y, last = torch.cat([p[0] for p in parts], 1), torch.cat([p[1] for p in parts])
        if not case["H"]:
            return [y, last]
        widths = [case["H"] * case["P"], case["G"] * case["N"], case["G"] * case["N"]]
        heads = [case["H"], case["G"], case["G"]]
        return [p.unflatten(-1, (k, -1)) for p, k in zip(y.split(widths, -1), heads)] + [last]
    gate = _gate64(s["z"].double())
    v = (x * gate if case["gate_first"] else x).view(case["rows"], case["G"], -1)
    var = v.var(-1, unbiased=False, keepdim=True) if case["center"] else v.pow(2).mean(-1, keepdim=True)
    mean = v.mean(-1, keepdim=True) if case["center"] else 0.0
    o = ((v - mean) * torch.rsqrt(var + EPS)).view(case["rows"], -1) * s["w"].double()
    if s["bias"] is not None:
        o = o + s["bias"].double()
    return o if case["gate_first"] else o * gate
