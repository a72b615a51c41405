"""The operators added beside the mixer's, as cases of real sizes: the per-channel selective scan
(prompts, its gradient, single tokens), the gradient of the short causal convolution, and the copying
and compacting of state-pool slots.

`own` false computes each operator from elementary torch operations in 32 bits, rounded once at the
end; `own` true calls the library.  `exact` computes the same from the definition in 64 bits."""
import math

import torch

own = False
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a chat turn's prompt on a small layer: latency counts
        dict(name="scan-turn", op="scan", batch=1, seqlen=37, channels=1536, groups=1, d_state=16, dtype="bf16",
             gate=True, init=False),
        # two documents of 8192 tokens, a large layer, continued from a stored state
        dict(name="scan-documents", op="scan", batch=2, seqlen=8192, channels=4096, groups=1, d_state=16,
             dtype="bf16", gate=True, init=True),
        # fine-tuning in fp32 on ragged texts, wider states in two groups, truncated back-propagation
        dict(name="scan-grad-ragged", op="scan_bwd", batch=3, seqlen=333, channels=768, groups=2, d_state=32,
             dtype="f32", gate=False, init=True),
        # a training step's layer: 4 sequences of 2048 tokens
        dict(name="scan-grad-train", op="scan_bwd", batch=4, seqlen=2048, channels=4096, groups=1, d_state=16,
             dtype="bf16", gate=True, init=False),
        # one user's next token
        dict(name="token-one", op="update", batch=1, channels=4096, groups=1, d_state=16, dtype="bf16", slots=0),
        # a full serving batch on a state pool
        dict(name="token-batch", op="update", batch=256, channels=8192, groups=1, d_state=16, dtype="bf16",
             slots=320),
        # the convolution's gradient on one short text, fp32
        dict(name="conv-grad-short", op="conv_bwd", batch=1, seqlen=77, channels=1792, dtype="f32", state=True),
        # the same on a training batch of the x|B|C channels of the 256-head layer
        dict(name="conv-grad-train", op="conv_bwd", batch=2, seqlen=8192, channels=18432, dtype="bf16", state=False),
        # one request forked into three samples: its conv windows in four layers
        dict(name="fork-windows", op="copy", layers=4, slots=16, slot=73728, dtype="bf16", pairs=3, snapshots=0),
        # 48 prefixes restored from a snapshot pool into the 256-head layer's states
        dict(name="restore-states", op="copy", layers=1, slots=64, slot=2097152, dtype="f32", pairs=48, snapshots=80),
        # a small pool's compaction after a few requests have ended
        dict(name="compact-small", op="compact", layers=2, slots=24, slot=32768, dtype="f32", live=11),
        # a serving pool's compaction: four layers' states of the 128-head layer
        dict(name="compact-pool", op="compact", layers=4, slots=96, slot=1048576, dtype="f32", live=56),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan_bwd", "update", "conv_bwd", "copy", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("scan", "scan_bwd"):
        most = (2 * 8192 * 4096 if op == "scan" else 4 * 2048 * 4096) * 16   # states x tokens
        N = rng.choice([16, 16, 16, 32, 64, 128])
        G = rng.choice([1, 1, 1, 2])
        D = 16 * _spread(rng, 8, 512)
        B = _spread(rng, 1, 16)
        L = _spread(rng, 1, 16384)
        L = max(1, min(L, most // (2 * B * D * N)))
        return dict(op=op, batch=B, seqlen=L, channels=D, groups=G, d_state=N, dtype=dtype,
                    gate=rng.random() < 0.7, init=rng.random() < 0.5)
    if op == "update":
        N = rng.choice([16, 16, 32, 64, 128])
        D = 16 * _spread(rng, 8, 512)
        B = max(1, min(_spread(rng, 1, 400), 256 * 8192 * 16 // (D * N)))
        return dict(op=op, batch=B, channels=D, groups=rng.choice([1, 1, 2]), d_state=N, dtype=dtype,
                    slots=rng.choice([0, B + _spread(rng, 1, 64)]))
    if op == "conv_bwd":
        CD = 8 * _spread(rng, 16, 2304)
        B = _spread(rng, 1, 8)
        L = max(1, min(_spread(rng, 1, 8192), 8192 * 18432 // (B * CD)))
        return dict(op=op, batch=B, seqlen=L, channels=CD, dtype=dtype, state=rng.random() < 0.5)
    layers = _spread(rng, 1, 8)
    slot = 8 * _spread(rng, 64, 262144)
    slots = max(8, min(_spread(rng, 8, 512), 100_000_000 // (layers * slot)))
    if op == "copy":
        return dict(op=op, layers=layers, slots=slots, slot=slot, dtype=dtype, pairs=rng.randint(1, slots // 2),
                    snapshots=rng.choice([0, slots // 2 + 3]))
    return dict(op=op, layers=layers, slots=slots, slot=slot, dtype=dtype, live=rng.randint(1, slots))


# ----------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=DEV) * std

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device=DEV) * (hi - lo) + lo

    s = dict(case)
    if case["op"] in ("scan", "scan_bwd", "update"):
        Bt, D, G, N = case["batch"], case["channels"], case["groups"], case["d_state"]
        rows = (Bt, case["seqlen"]) if "seqlen" in case else (Bt,)
        R = 8 * max(1, D // 128)                              # the rank of dt's projection
        u = normal(*rows, D)
        s["x"] = (u * torch.sigmoid(u)).to(t)                 # what the convolution and its SiLU leave
        s["dt"] = normal(*rows, D, std=0.5).to(t)
        dt0 = torch.exp(uniform(math.log(1e-3), math.log(1e-1), D))
        s["dt_bias"] = dt0 + torch.log(-torch.expm1(-dt0))    # softplus(dt_bias) = dt0
        s["A"] = -torch.arange(1, N + 1, device=DEV, dtype=torch.float32) * uniform(0.8, 1.25, D, N)
        proj = normal(*rows, R + 2 * G * N).to(t)             # dt's factor | B | C of one projection
        s["B"] = proj[..., R:R + G * N].unflatten(-1, (G, N))
        s["C"] = proj[..., R + G * N:].unflatten(-1, (G, N))
        s["D"] = normal(D)
        xz = normal(*rows, 2 * D).to(t) if case.get("gate", True) else None
        s["z"] = None if xz is None else xz[..., D:]
        if case["op"] == "update":
            n = case["slots"]
            s["state"] = normal(n or Bt, D, N, std=0.1)
            s["state_out"] = torch.zeros_like(s["state"])
            s["slot_idx"] = torch.randperm(n, generator=g, device=DEV)[:Bt].to(torch.int32) if n else None
        else:
            s["init"] = normal(Bt, D, N, std=0.1) if case["init"] else None
        if case["op"] == "scan_bwd":
            s["dy"] = normal(*rows, D).to(t)
            s["dfinal"] = normal(Bt, D, N, std=0.1) if case["init"] else None
        return s
    if case["op"] == "conv_bwd":
        Bt, L, CD = case["batch"], case["seqlen"], case["channels"]
        s["xbc"] = normal(Bt, L, CD).to(t)
        s["w"] = uniform(-0.5, 0.5, CD, 4).to(t)
        s["bias"] = uniform(-0.5, 0.5, CD).to(t)
        s["dout"] = normal(Bt, L, CD).to(t)
        s["conv_state"] = normal(Bt, CD, 4).to(t) if case["state"] else None
        return s
    s["pool"] = normal(case["layers"], case["slots"], case["slot"]).to(t)
    order = torch.randperm(case["slots"], generator=g, device=DEV).to(torch.int32)
    if case["op"] == "copy":
        n = case["pairs"]
        if case["snapshots"]:
            s["from"] = normal(case["layers"], case["snapshots"], case["slot"]).to(t)
            s["src"] = torch.randint(case["snapshots"], (n,), generator=g, device=DEV, dtype=torch.int32)
            s["dst"] = order[:n].contiguous()
        else:                                                 # forks: few sources, distinct destinations
            s["from"] = s["pool"]
            k = max(1, (case["slots"] - n) // 2)
            s["src"] = order[n:][torch.randint(k, (n,), generator=g, device=DEV)].contiguous()
            s["dst"] = order[:n].contiguous()
    else:
        s["slot_idx"] = order[:case["live"]].contiguous()
    return s


# ------------------------------------------------------------------------------------------- runs
def run(s):
    return {"scan": _scan, "scan_bwd": _scan_bwd, "update": _update, "conv_bwd": _conv_bwd, "copy": _copy,
            "compact": _compact}[s["op"]](s)


def _lib():
    from selective_state_space_conv1d_amd import ssd
    return ssd


def _per_channel(m, D):
    """[..., G, N] -> [..., D, N] in fp32."""
    return m.float().repeat_interleave(D // m.shape[-2], -2)


def _dt(s):
    v = s["dt"].float() + s["dt_bias"]
    return torch.where(v > 20, v, torch.log1p(torch.exp(v)))


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1 from zero, by doubling the span that each step joins."""
    k, L = 1, a.shape[1]
    while k < L:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        if 2 * k < L:
            a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _states(s, dt, x):
    """Decays a [B, L, D, N] and states h after each token."""
    a = torch.exp(dt[..., None] * s["A"])
    b = (dt * x)[..., None] * _per_channel(s["B"], x.shape[-1])
    if s["init"] is not None:
        b[:, 0] += a[:, 0] * s["init"]
    return a, _linear_scan(a, b)


def _gate(y, z):
    return y if z is None else y * (z.float() * torch.sigmoid(z.float()))


def _scan(s):
    if own:
        final = torch.empty((s["batch"], s["channels"], s["d_state"]), device=DEV)
        y = _lib().ssd_selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], z=s["z"], init_state=s["init"],
                                      final_state=final, dt_bias=s["dt_bias"], dt_softplus=True)
        return {"y": y, "final": final}
    x, dt = s["x"].float(), _dt(s)
    _, h = _states(s, dt, x)
    y = (h * _per_channel(s["C"], x.shape[-1])).sum(-1) + s["D"] * x
    return {"y": _gate(y, s["z"]).to(s["x"].dtype), "final": h[:, -1].contiguous()}


def _scan_bwd(s):
    if own:
        return _lib().ssd_selective_scan_bwd(s["dy"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], z=s["z"],
                                             init_state=s["init"], dfinal_state=s["dfinal"], dt_bias=s["dt_bias"],
                                             dt_softplus=True)
    t, x, dt, dout = s["x"].dtype, s["x"].float(), _dt(s), s["dy"].float()
    D, G = x.shape[-1], s["B"].shape[-2]
    a, h = _states(s, dt, x)
    B, C = _per_channel(s["B"], D), _per_channel(s["C"], D)
    dz, dy = None, dout
    if s["z"] is not None:
        z = s["z"].float()
        sig = torch.sigmoid(z)
        y = (h * C).sum(-1) + s["D"] * x
        dz = (dout * y * sig * (1 + z * (1 - sig))).to(t)
        dy = dout * z * sig
    b = dy[..., None] * C
    if s["dfinal"] is not None:
        b[:, -1] += s["dfinal"]
    later = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g = _linear_scan(later.flip(1), b.flip(1)).flip(1)
    before = h - (dt * x)[..., None] * B                      # a_t h_{t-1}
    gb = (g * B).sum(-1)
    ddt = ((g * before * s["A"]).sum(-1) + gb * x) * torch.sigmoid(s["dt"].float() + s["dt_bias"])
    per_group = lambda m: m.unflatten(2, (G, D // G)).sum(3).to(t)  # noqa: E731
    return {"dx": (s["D"] * dy + dt * gb).to(t), "ddt": ddt.to(t), "dA": (g * before * dt[..., None]).sum((0, 1)),
            "dB": per_group(g * (dt * x)[..., None]), "dC": per_group(h * dy[..., None]), "dD": (dy * x).sum((0, 1)),
            "dz": dz, "ddt_bias": ddt.sum((0, 1)),
            "dinit_state": None if s["init"] is None else a[:, 0] * g[:, 0]}


def _update(s):
    if own:
        y = _lib().ssd_selective_state_update(s["state"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], z=s["z"],
                                              slot_idx=s["slot_idx"], state_out=s["state_out"], dt_bias=s["dt_bias"],
                                              dt_softplus=True)
        return {"y": y, "state": s["state_out"]}
    x, dt, at = s["x"].float(), _dt(s), s["slot_idx"]
    old = s["state"] if at is None else s["state"][at.long()]
    h = torch.exp(dt[..., None] * s["A"]) * old + (dt * x)[..., None] * _per_channel(s["B"], x.shape[-1])
    y = (h * _per_channel(s["C"], x.shape[-1])).sum(-1) + s["D"] * x
    if at is None:
        s["state_out"].copy_(h)
    else:
        s["state_out"][at.long()] = h
    return {"y": _gate(y, s["z"]).to(s["x"].dtype), "state": s["state_out"]}


def _conv_bwd(s):
    if own:
        return _lib().ssd_conv1d_bwd(s["dout"], s["xbc"], s["w"], s["bias"], conv_state_in=s["conv_state"])
    t, L, w = s["xbc"].dtype, s["seqlen"], s["w"].float()
    if s["conv_state"] is None:
        head = torch.zeros((s["batch"], 3, s["channels"]), device=DEV)
    else:
        head = s["conv_state"][..., 1:].float().transpose(1, 2)
    u = torch.cat([head, s["xbc"].float()], 1)                # u[:, 3 + t] is token t
    p = s["bias"].float() + w[:, 0] * u[:, :L] + w[:, 1] * u[:, 1:L + 1] + w[:, 2] * u[:, 2:L + 2] + w[:, 3] * u[:, 3:]
    sig = torch.sigmoid(p)
    q = s["dout"].float() * sig * (1 + p * (1 - sig))
    q = torch.nn.functional.pad(q, (0, 0, 3, 3))              # q[:, 3 + t] is token t
    du = w[:, 3] * q[:, :L + 3] + w[:, 2] * q[:, 1:L + 4] + w[:, 1] * q[:, 2:L + 5] + w[:, 0] * q[:, 3:]
    q = q[:, 3:L + 3]
    dw = torch.stack([(q * u[:, :L]).sum((0, 1)), (q * u[:, 1:L + 1]).sum((0, 1)), (q * u[:, 2:L + 2]).sum((0, 1)),
                      (q * u[:, 3:]).sum((0, 1))], -1)
    dstate = None
    if s["conv_state"] is not None:
        dstate = torch.cat([torch.zeros_like(du[:, :1]), du[:, :3]], 1).transpose(1, 2).to(t)
    return {"dxbc": du[:, 3:].to(t), "dw": dw, "dbias": q.sum((0, 1)), "dconv_state_in": dstate}


def _copy(s):
    if own:
        _lib().ssd_pool_copy(s["pool"], s["dst"], s["from"], s["src"], stacked=True)
    else:
        s["pool"][:, s["dst"].long()] = s["from"][:, s["src"].long()]
    return s["pool"]


def _compact(s):
    if own:
        ssd = _lib()
        src, dst, new, count = ssd.ssd_pool_compact(s["slot_idx"], s["slots"])
        ssd.ssd_pool_copy(s["pool"], dst, s["pool"], src, stacked=True)
        return {"pool": s["pool"], "slot_idx": new, "count": count}
    at = torch.arange(s["slots"], device=DEV)
    live = torch.zeros(s["slots"], dtype=torch.bool, device=DEV)
    live[s["slot_idx"].long()] = True
    count = live.sum()
    holes, movers = (~live & (at < count)).nonzero()[:, 0], (live & (at >= count)).nonzero()[:, 0]
    s["pool"][:, holes] = s["pool"][:, movers]
    at[movers] = holes
    return {"pool": s["pool"], "slot_idx": at[s["slot_idx"].long()].to(torch.int32), "count": count.to(torch.int32)}


# ------------------------------------------------------------------------------------------- work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("scan", "scan_bwd", "update"):
        D, G, N = case["channels"], case["groups"], case["d_state"]
        rows = case["batch"] * case.get("seqlen", 1)
        z = 1 if case.get("gate", True) else 0
        params = 4 * D * (N + 2)
        state = 4 * case["batch"] * D * N
        if case["op"] == "scan":
            return {"bytes": e * rows * (D * (3 + z) + 2 * G * N) + params + state * (2 if case["init"] else 1),
                    "flops": rows * D * (8 * N + 8)}
        if case["op"] == "update":
            return {"bytes": e * rows * (D * (3 + z) + 2 * G * N) + params + 2 * state, "flops": rows * D * (8 * N + 8)}
        return {"bytes": e * rows * (D * (5 + 2 * z) + 4 * G * N) + 2 * params + (3 * state if case["init"] else 0),
                "flops": rows * D * (26 * N + 20)}
    if case["op"] == "conv_bwd":
        n, CD = case["batch"] * case["seqlen"] * case["channels"], case["channels"]
        return {"bytes": e * (3 * n + 5 * CD) + 20 * CD + (8 * e * case["batch"] * CD if case["state"] else 0),
                "flops": 32 * n}
    if case["op"] == "copy":
        moved = case["pairs"]
    else:                                                     # live slots above the live count, on average
        moved = max(1, round(case["live"] * (case["slots"] - case["live"]) / case["slots"]))
    return {"bytes": 2 * e * case["layers"] * case["slot"] * moved, "flops": 0}


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    if case["op"] in ("copy", "compact"):
        return None
    s = prepare(case, seed)
    f = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    return {"scan": _exact_scan, "scan_bwd": _exact_bwd, "update": _exact_update, "conv_bwd": _exact_conv}[case["op"]](f)


def _exact_dt(f):
    return torch.logaddexp(f["dt"] + f["dt_bias"], torch.zeros((), dtype=torch.float64, device=DEV))


def _exact_silu(z):
    return z / (1 + torch.exp(-z))


def _exact_token(f, h, t, dt, r):
    h = torch.exp(dt[:, t, :, None] * f["A"]) * h + (dt[:, t] * f["x"][:, t])[..., None] * f["B"][:, t].repeat_interleave(r, 1)
    return h


def _exact_scan(f):
    Bt, L, D = f["x"].shape
    r, dt = D // f["groups"], _exact_dt(f)
    h = f["init"] if f["init"] is not None else torch.zeros((Bt, D, f["d_state"]), dtype=torch.float64, device=DEV)
    y = torch.empty_like(f["x"])
    for t in range(L):
        h = _exact_token(f, h, t, dt, r)
        y[:, t] = (h * f["C"][:, t].repeat_interleave(r, 1)).sum(-1)
    y += f["D"] * f["x"]
    return {"y": y if f["z"] is None else y * _exact_silu(f["z"]), "final": h}


def _exact_bwd(f):
    Bt, L, D = f["x"].shape
    N, G = f["d_state"], f["groups"]
    r, dt, x = D // G, _exact_dt(f), f["x"]
    zero = torch.zeros((Bt, D, N), dtype=torch.float64, device=DEV)
    h = [f["init"] if f["init"] is not None else zero]
    for t in range(L):
        h.append(_exact_token(f, h[-1], t, dt, r))
    o = {k: torch.empty_like(x) for k in ("dx", "ddt")}
    o["dz"] = None if f["z"] is None else torch.empty_like(x)
    o["dB"], o["dC"] = torch.empty_like(f["B"]), torch.empty_like(f["C"])
    o["dA"] = torch.zeros_like(f["A"])
    o["dD"], o["ddt_bias"] = torch.zeros_like(f["D"]), torch.zeros_like(f["D"])
    g = f["dfinal"] if f["dfinal"] is not None else zero
    for t in range(L - 1, -1, -1):
        B, C = f["B"][:, t].repeat_interleave(r, 1), f["C"][:, t].repeat_interleave(r, 1)
        dy = f["dy"][:, t]
        if f["z"] is not None:
            z = f["z"][:, t]
            e = torch.exp(-z)
            o["dz"][:, t] = dy * ((h[t + 1] * C).sum(-1) + f["D"] * x[:, t]) * (1 + e + z * e) / (1 + e) ** 2
            dy = dy * _exact_silu(z)
        g = g + dy[..., None] * C
        a = torch.exp(dt[:, t, :, None] * f["A"])
        o["dC"][:, t] = (dy[..., None] * h[t + 1]).view(Bt, G, r, N).sum(2)
        o["dB"][:, t] = ((dt[:, t] * x[:, t])[..., None] * g).view(Bt, G, r, N).sum(2)
        o["dx"][:, t] = f["D"] * dy + dt[:, t] * (g * B).sum(-1)
        da = g * h[t] * a
        o["ddt"][:, t] = ((da * f["A"]).sum(-1) + x[:, t] * (g * B).sum(-1)) / (1 + torch.exp(-f["dt"][:, t] - f["dt_bias"]))
        o["dA"] += (da * dt[:, t, :, None]).sum(0)
        o["dD"] += (dy * x[:, t]).sum(0)
        o["ddt_bias"] += o["ddt"][:, t].sum(0)
        g = a * g
        h.pop()
    o["dinit_state"] = None if f["init"] is None else g
    return o


def _exact_update(f):
    at = f["slot_idx"]
    h = f["state"] if at is None else f["state"][at.long()]
    r, dt, x = f["channels"] // f["groups"], _exact_dt(f), f["x"]
    h = torch.exp(dt[..., None] * f["A"]) * h + (dt * x)[..., None] * f["B"].repeat_interleave(r, 1)
    y = (h * f["C"].repeat_interleave(r, 1)).sum(-1) + f["D"] * x
    if at is not None:
        f["state_out"][at.long()] = h
        h = f["state_out"]
    return {"y": y * _exact_silu(f["z"]), "state": h}


def _exact_conv(f):
    Bt, L, CD = f["xbc"].shape
    st = f["conv_state"] if f["conv_state"] is not None else torch.zeros((Bt, CD, 4), dtype=torch.float64, device=DEV)
    u = torch.cat([st.transpose(1, 2), f["xbc"]], 1)          # u[:, 4 + t] is token t
    p = f["bias"] + torch.zeros_like(f["xbc"])
    for k in range(4):
        p += f["w"][:, k] * u[:, 1 + k:1 + k + L]
    e = torch.exp(-p)
    q = f["dout"] * (1 + e + p * e) / (1 + e) ** 2
    du, dw = torch.zeros_like(u), torch.empty_like(f["w"])
    for k in range(4):
        du[:, 1 + k:1 + k + L] += f["w"][:, k] * q
        dw[:, k] = (q * u[:, 1 + k:1 + k + L]).sum((0, 1))
    return {"dxbc": du[:, 4:].contiguous(), "dw": dw, "dbias": q.sum((0, 1)),
            "dconv_state_in": None if f["conv_state"] is None else du[:, :4].transpose(1, 2).contiguous()}
