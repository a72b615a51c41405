"""The per-channel selective scan, its gradient, its single tokens and the conv's gradient on the GPU,
against the float64 definitions in selective_ref (which derives the bounds)."""
import pytest
import torch

import selective_ref as ref
from selective_state_space_conv1d_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def make(Bt, L, D, G, N, dtype, seed, gate=True, init=True, pad=8, tokens=True):
    """Inputs as a layer has them: x, z and B/C views into wider rows (pad extra elements), dt raw."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    rows = (Bt, L) if tokens else (Bt,)
    s = dict(x=n(*rows, D + pad).to(dtype).to(DEV)[..., pad:], dt=n(*rows, D).mul(0.7).sub(2.0).to(dtype).to(DEV),
             A=-torch.exp(n(D, N).mul(0.7)).to(DEV), D=n(D).to(DEV))
    bc = n(*rows, pad + 2 * G * N).to(dtype).to(DEV)
    s["B"] = bc[..., pad:pad + G * N].unflatten(-1, (G, N))
    s["C"] = bc[..., pad + G * N:].unflatten(-1, (G, N))
    s["z"] = n(*rows, 2 * D).to(dtype).to(DEV)[..., D:] if gate else None
    s["dt_bias"] = n(D).mul(0.3).to(DEV)
    if tokens:
        s["init"] = n(Bt, D, N).mul(0.5).to(DEV) if init else None
        s["dy"] = n(Bt, L, D).to(dtype).to(DEV)
        s["dfinal"] = n(Bt, D, N).mul(0.5).to(DEV) if init else None
    else:
        s["state"] = n(Bt, D, N).to(DEV)
    return s


def k_of(L, N):
    return 16 * L + N + 64


ARGS = ("x", "dt", "A", "B", "C", "D", "z")
# batch, tokens, channels, groups, states: one token; a tile's border; channels that end inside a
# workgroup, groups that do; every state count; several tiles; more than one batch entry
# (sequences of 64 tokens and more are cut into chunks at these sizes, save where the batch fills the chip)
SIZES = [(1, 140, 72, 1, 32), (1, 130, 40, 2, 64), (2, 133, 66, 1, 128), (512, 130, 8, 1, 16),
         (1, 1, 8, 1, 16), (2, 16, 64, 1, 16), (1, 17, 72, 1, 16), (2, 37, 200, 2, 16), (3, 100, 40, 1, 32),
         (1, 65, 96, 2, 64), (2, 33, 130, 1, 128), (1, 300, 64, 1, 16), (1, 5, 1, 1, 32), (1, 15, 66, 3, 64),
         (1, 1500, 24, 1, 16)]                      # more chunks of 32 tokens than the root of the length


def forward(s, **kw):
    final = torch.full((s["x"].shape[0], s["x"].shape[2], s["A"].shape[1]), 7.0, device=DEV)
    y = ssd.ssd_selective_scan(*[s[k] for k in ARGS], init_state=s["init"], final_state=final, dt_bias=s["dt_bias"],
                               dt_softplus=True, **kw)
    return y, final


@pytest.mark.parametrize("dtype,ydt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("size", SIZES)
def test_scan(size, dtype, ydt):
    s = make(*size, dtype, 1000 + size[1], gate=size[2] % 16 != 8, init=size[0] != 2)
    y, final = forward(s, y_dtype=ydt)
    args = [s[k] for k in ARGS] + [s["init"], s["dt_bias"], True]
    ry, rf, _, _ = ref.scan(*args)
    my, mf, _, _ = ref.scan(*args, absolute=True)
    k = k_of(size[1], size[4])
    ref.check(y, ry, my, k, "y")
    ref.check(final, rf, mf, k, "final")
    assert y.dtype == ydt


@pytest.mark.parametrize("dtype,ydt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("size", SIZES)
def test_gradient(size, dtype, ydt):
    Bt, L, D, G, N = size
    s = make(*size, dtype, 2000 + L, gate=D % 16 != 8, init=Bt != 2)
    dy = s["dy"].to(ydt)
    got = ssd.ssd_selective_scan_bwd(dy, *[s[k] for k in ARGS], init_state=s["init"], dfinal_state=s["dfinal"],
                                     dt_bias=s["dt_bias"], dt_softplus=True)
    args = [dy] + [s[k] for k in ARGS] + [s["init"], s["dfinal"], s["dt_bias"], True]
    r, m = ref.scan_grad(*args), ref.scan_grad(*args, absolute=True)
    assert set(got) == set(r)
    k = 2 * k_of(L, N) + D // G + Bt * L      # states on the way out and gradients on the way back, then sums
    for name in r:
        assert (got[name] is None) == (r[name] is None), name
        if r[name] is not None:
            ref.check(got[name], r[name], m[name], k, name)


def test_offsets_past_32_bits():
    """Token rows 2^23 elements apart: the last ones lie past 4 GiB, on their own and in the whole call."""
    L, D, N, rs = 300, 72, 16, 1 << 23
    s = make(1, L, D, 1, N, BF, 23)
    wide = {k: torch.empty((L, rs), dtype=BF, device=DEV) for k in ("x", "z")}
    t = dict(s)
    for k, v in wide.items():
        v[:, 8:8 + D] = s[k][0]
        t[k] = v[None, :, 8:8 + D]
    y, final = forward(t)
    yc, finalc = forward(s)
    assert torch.equal(y, yc) and torch.equal(final, finalc)
    a, b = (ssd.ssd_selective_scan_bwd(q["dy"], *[q[k] for k in ARGS], init_state=q["init"], dt_bias=q["dt_bias"], dt_softplus=True) for q in (t, s))
    assert all(v is None or torch.equal(v, b[k]) for k, v in a.items())
    w = torch.rand(128, 4, device=DEV).to(BF)
    x = wide["x"][None, :, :128]
    wide["x"][:, :128] = torch.randn(L, 128, device=DEV).to(BF)
    dout = torch.randn(1, L, 128, device=DEV).to(BF)
    a, b = ssd.ssd_conv1d_bwd(dout, x, w), ssd.ssd_conv1d_bwd(dout, x.contiguous(), w)
    assert all(v is None or torch.equal(v, b[k]) for k, v in a.items())


@pytest.mark.parametrize("softplus,limit,bias", [(False, None, False), (True, (0.05, 0.4), True), (False, (-0.2, 0.3), True)])
def test_dt_prologue_and_its_gradient(softplus, limit, bias):
    """dt as given, clamped after the softplus, clamped without it (dt may then be negative)."""
    s = make(2, 40, 48, 1, 16, F32, 31)
    if not softplus:
        s["dt"] = (s["dt"] + 2.0).mul(0.2).contiguous()
    b = s["dt_bias"].mul(0.2) if bias else None
    kw = dict(dt_bias=b, dt_softplus=softplus, dt_limit=limit)
    y = ssd.ssd_selective_scan(*[s[k] for k in ARGS], init_state=s["init"], **kw)
    got = ssd.ssd_selective_scan_bwd(s["dy"], *[s[k] for k in ARGS], init_state=s["init"], **kw)
    a = [s[k] for k in ARGS] + [s["init"]]
    ry = ref.scan(*a, b, softplus, limit)[0]
    # dt changes sign without the softplus: decays above 1 are in the sums of absolute values as they are
    my = ref.scan(*a, b, softplus, limit, absolute=True)[0] if softplus else None
    k = k_of(40, 16)
    if softplus:
        ref.check(y, ry, my, k, "y")
    else:
        assert float((ref.f64(y) - ry).abs().max()) <= k * ref.U * 8 * float(ry.abs().max())
    r = ref.scan_grad(s["dy"], *a, None, b, softplus, limit)
    for name in r:
        if r[name] is not None:
            e = float((ref.f64(got[name]) - r[name]).abs().max())
            assert e <= 2 * k * ref.U * 8 * float(r[name].abs().max()), (name, e)


def test_reference_gradient_is_autograds():
    """The formulas of the reference against automatic differentiation of its forward (float64, CPU)."""
    s = make(2, 9, 12, 2, 16, F32, 5)
    names = ["x", "dt", "A", "B", "C", "D", "z", "init", "dt_bias"]
    leaves = {n: ref.f64(s[n]).clone().requires_grad_() for n in names}
    keep = ref.f64
    try:
        ref.f64 = lambda t: t if t is None or t.requires_grad else keep(t)
        y, final, _, _ = ref.scan(*[leaves[n] for n in ARGS], leaves["init"], leaves["dt_bias"], True)
    finally:
        ref.f64 = keep
    ((y * ref.f64(s["dy"])).sum() + (final * ref.f64(s["dfinal"])).sum()).backward()
    r = ref.scan_grad(s["dy"], *[s[k] for k in ARGS], s["init"], s["dfinal"], s["dt_bias"], True)
    for n, k in zip(names, ["dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dinit_state", "ddt_bias"]):
        assert float((leaves[n].grad - r[k]).abs().max()) <= 1e-12 * (1 + float(r[k].abs().max())), n


def test_gradient_against_differences():
    """A step along a random direction changes the loss as the gradients say (fp32 kernel, float64 sums):
    central differences of step e are off by e^2 times the third derivative and 2^-24 |terms| / e."""
    s = make(1, 24, 32, 1, 16, F32, 77)
    got = ssd.ssd_selective_scan_bwd(s["dy"], *[s[k] for k in ARGS], init_state=s["init"], dfinal_state=s["dfinal"],
                                     dt_bias=s["dt_bias"], dt_softplus=True)
    g = torch.Generator().manual_seed(3)
    for name, key in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("z", "dz"), ("init", "dinit_state")):
        v = torch.randn(s[name].shape, generator=g).to(DEV)
        e = 2.0 ** -8
        loss = []
        for sign in (1, -1):
            t = dict(s)
            t[name] = (s[name] + sign * e * v).contiguous()
            y, final, _, _ = ref.scan(*[t[k] for k in ARGS], t["init"], t["dt_bias"], True)
            loss.append(float((y * ref.f64(s["dy"])).sum() + (final * ref.f64(s["dfinal"])).sum()))
        want = (loss[0] - loss[1]) / (2 * e)
        have = float((ref.f64(got[key]) * ref.f64(v)).sum())
        scale = float((ref.f64(got[key]) * ref.f64(v)).abs().sum())
        assert abs(want - have) <= 2e-3 * scale, (name, want, have)


@pytest.mark.parametrize("L", [0, 1])
def test_empty_and_single(L):
    """No tokens: the state passes through, parameters' gradients are zero; no batch entries at all."""
    s = make(2, 1, 24, 1, 16, F32, 9)
    t = {k: (v[:, :L] if k in ("x", "dt", "B", "C", "z", "dy") else v) for k, v in s.items()}
    t["dt"], t["dy"] = t["dt"].contiguous(), t["dy"].contiguous()
    y, final = forward(t)
    assert y.shape == (2, L, 24)
    got = ssd.ssd_selective_scan_bwd(t["dy"], *[t[k] for k in ARGS], init_state=t["init"], dfinal_state=t["dfinal"],
                                     dt_bias=t["dt_bias"], dt_softplus=True)
    if L == 0:
        assert torch.equal(final, t["init"]) and torch.equal(got["dinit_state"], t["dfinal"])
        assert all(float(got[k].abs().sum()) == 0 for k in ("dA", "dD", "ddt_bias"))
    none = {k: (v[:0] if k not in ("A", "D", "dt_bias") else v) for k, v in s.items()}
    assert forward(none)[0].shape == (0, 1, 24)
    got = ssd.ssd_selective_scan_bwd(none["dy"], *[none[k] for k in ARGS], dt_bias=none["dt_bias"])
    assert float(got["dA"].abs().sum()) == 0 and float(got["dD"].abs().sum()) == 0


def test_scan_split_in_two_continues():
    """A prompt in two parts through the state, the state updated in place, against the whole."""
    s = make(2, 90, 136, 1, 32, F32, 41)
    y, final = forward(s)
    state = s["init"].clone()
    ys = []
    for a, b in ((0, 41), (41, 90)):
        p = {k: (s[k][:, a:b] if k in ("x", "B", "C", "z") else s[k]) for k in ARGS}
        for i in range(2):      # one batch entry at a time: views of one entry have any batch stride
            q = {k: (v[i:i + 1] if k in ("x", "B", "C", "z") else v) for k, v in p.items()}
            st = state[i:i + 1]
            ys.append((a, i, ssd.ssd_selective_scan(q["x"], s["dt"][i:i + 1, a:b].contiguous(), s["A"], q["B"], q["C"], s["D"],
                                                    q["z"], init_state=st, final_state=st, dt_bias=s["dt_bias"], dt_softplus=True)))
    k = 2 * k_of(90, 32)
    args = [s[n] for n in ARGS] + [s["init"], s["dt_bias"], True]
    _, mf, _, _ = ref.scan(*args, absolute=True)
    my = ref.scan(*args, absolute=True)[0]
    ref.check(state, ref.f64(final), mf, k, "final")
    for a, i, part in ys:
        ref.check(part, ref.f64(y[i:i + 1, a:a + part.shape[1]]), my[i:i + 1, a:a + part.shape[1]], k, "y")


def test_values_out_of_range_stay_in_their_place():
    """A reset (dt A far below the range of exp) and an infinite input: nothing before the token or in
    another channel changes, the channel itself has what the definition has."""
    s = make(1, 48, 64, 1, 16, F32, 13, gate=False)
    base, _ = forward(s)
    x = s["x"].clone()
    x[0, 20, 3] = float("inf")
    y, final = forward({**s, "x": x})
    others = [c for c in range(64) if c != 3]
    assert torch.equal(y[:, :, others], base[:, :, others]) and torch.equal(y[:, :20], base[:, :20])
    assert not torch.isfinite(y[0, 20:, 3]).any()
    A = s["A"].clone()
    A[5] = -1e30
    t = {**s, "A": A}
    y, final = forward(t)
    ry, rf, _, _ = ref.scan(*[t[k] for k in ARGS], t["init"], t["dt_bias"], True)
    assert torch.isfinite(y).all() and float((ref.f64(y) - ry).abs().max()) <= k_of(48, 16) * ref.U * 64 * float(ry.abs().max())
    got = ssd.ssd_selective_scan_bwd(t["dy"], *[t[k] for k in ARGS], init_state=t["init"], dt_bias=t["dt_bias"], dt_softplus=True)
    assert all(torch.isfinite(v).all() for v in got.values() if v is not None)


@pytest.mark.parametrize("L", [5, 48, 141])
def test_channel_that_forgets_everything(L):
    """A of minus infinity: the state is what the last token brought, also where the last tile is not full."""
    s = make(1, L, 64, 1, 16, F32, 14, gate=False)
    s["A"][5] = float("-inf")
    y, final = forward(s)
    args = [s[k] for k in ARGS] + [s["init"], s["dt_bias"], True]
    ry, rf, _, _ = ref.scan(*args)
    my, mf, _, _ = ref.scan(*args, absolute=True)
    ref.check(y, ry, my, k_of(L, 16), "y")
    ref.check(final, rf, mf, k_of(L, 16), "final")
    got = ssd.ssd_selective_scan_bwd(s["dy"], *[s[k] for k in ARGS], init_state=s["init"], dfinal_state=s["dfinal"], dt_bias=s["dt_bias"],
                                     dt_softplus=True)
    assert all(torch.isfinite(v).all() for v in got.values() if v is not None)


@pytest.mark.parametrize("size", [(2, 700, 136, 1, 16), (1, 400, 72, 1, 64), (40, 130, 64, 1, 16)])
def test_chunked_scan_in_place(size):
    """The final state written over the initial one, which the first chunk needs."""
    s = make(*size, BF, 15)
    y, final = forward(s)
    state = s["init"].clone()
    for _ in range(3):
        state.copy_(s["init"])
        y2 = ssd.ssd_selective_scan(*[s[k] for k in ARGS], init_state=state, final_state=state, dt_bias=s["dt_bias"], dt_softplus=True)
        assert torch.equal(y, y2) and torch.equal(state, final)


def test_gradient_is_the_same_every_time_and_on_another_stream():
    s = make(2, 150, 192, 1, 16, BF, 17)
    call = lambda **kw: ssd.ssd_selective_scan_bwd(s["dy"], *[s[k] for k in ARGS], init_state=s["init"], dfinal_state=s["dfinal"],  # noqa: E731
                                                   dt_bias=s["dt_bias"], dt_softplus=True, **kw)
    a = call()
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [call(stream=st) for st in side]
    fy = [forward(s, stream=st)[0] for st in side]
    torch.cuda.synchronize()
    y = forward(s)[0]
    for o, f in zip(outs, fy):
        assert all(v is None or torch.equal(v, o[k]) for k, v in a.items()) and torch.equal(f, y)


# ------------------------------------------------------------------------------------- single tokens
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [(1, 8, 1, 16), (5, 200, 2, 16), (3, 40, 1, 32), (9, 96, 2, 64), (2, 131, 1, 128), (70, 24, 1, 16)])
@pytest.mark.parametrize("slots", [False, True])
def test_update(size, dtype, slots):
    Bt, D, G, N = size
    s = make(Bt, 1, D, G, N, dtype, 50 + Bt, tokens=False)
    state = s["state"] if not slots else torch.randn(Bt + 4, D, N, generator=torch.Generator().manual_seed(1)).to(DEV)
    idx = torch.randperm(Bt + 4, generator=torch.Generator().manual_seed(2))[:Bt].to(torch.int32) if slots else None
    if slots and Bt > 2:
        idx[1], idx[2] = -1, Bt + 4          # padding
    at = torch.arange(Bt) if idx is None else idx.long()
    pad = (at < 0) | (at >= state.shape[0])
    first = state.cpu()[at.clamp(0, state.shape[0] - 1)] * (~pad)[:, None, None]
    one = [s[k].unsqueeze(1) if k in ("x", "dt", "B", "C", "z") else s[k] for k in ARGS]
    ry, rf, _, _ = ref.scan(*one, first, s["dt_bias"], True)
    my, mf, _, _ = ref.scan(*one, first, s["dt_bias"], True, absolute=True)
    want = state.cpu().double()
    want[at[~pad]] = rf[~pad]
    mag = state.cpu().double().abs()
    mag[at[~pad]] = mf[~pad]
    dev_idx = None if idx is None else idx.to(DEV)
    out = torch.full_like(state, 3.0)
    before = state.clone()
    y = ssd.ssd_selective_state_update(state, *[s[k] for k in ARGS], slot_idx=dev_idx, state_out=out, dt_bias=s["dt_bias"], dt_softplus=True)
    assert torch.equal(state, before)
    ref.check(y, ry[:, 0], my[:, 0], k_of(1, N), "y")
    named = torch.zeros(state.shape[0], dtype=torch.bool)
    named[at[~pad]] = True
    assert bool((out[~named.to(DEV)] == 3.0).all())
    y2 = ssd.ssd_selective_state_update(state, *[s[k] for k in ARGS], slot_idx=dev_idx, dt_bias=s["dt_bias"], dt_softplus=True)
    assert torch.equal(y, y2) and torch.equal(state[named.to(DEV)], out[named.to(DEV)])
    assert torch.equal(state[~named.to(DEV)], before[~named.to(DEV)])
    ref.check(state, want, mag, k_of(1, N), "state")


def test_prompt_then_tokens_on_a_pool_under_a_graph():
    """A run as served: the conv and the scan of a prompt into pool slots, the prompt's slots forked, then
    single tokens from a captured graph replayed with new inputs -- against the scan of the whole text."""
    D, N, L, steps = 128, 16, 40, 4
    s = make(1, L + steps, D, 1, N, F32, 71, init=False)
    g = torch.Generator().manual_seed(8)
    w, bias = (torch.rand(D, 4, generator=g) - 0.5).to(DEV), (torch.rand(D, generator=g) - 0.5).to(DEV)
    pool, conv_pool = torch.zeros(6, D, N, device=DEV), torch.zeros(6, D, 4, device=DEV)
    par = dict(dt_bias=s["dt_bias"], dt_softplus=True)
    u = s["x"].contiguous()
    xs = ssd.ssd_conv1d_fwd(u[:, :L], w, bias, None, conv_pool[2:3])
    y0 = ssd.ssd_selective_scan(xs, s["dt"][:, :L].contiguous(), s["A"], s["B"][:, :L], s["C"][:, :L], s["D"], s["z"][:, :L],
                                final_state=pool[2:3], **par)
    src, dst = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in ([2, 2], [0, 5]))
    for p in (pool, conv_pool):
        ssd.ssd_pool_copy(p, dst, p, src)
    slots = torch.tensor([0, 2, 5], dtype=torch.int32, device=DEV)
    buf = {k: torch.zeros_like(s[k][:, 0].expand(3, *s[k].shape[2:]).contiguous()) for k in ("x", "dt", "B", "C", "z")}

    def step():
        xt = ssd.ssd_conv1d_update_slots(buf["x"], w, bias, conv_pool, slots)
        return ssd.ssd_selective_state_update(pool, xt, buf["dt"], s["A"], buf["B"], buf["C"], s["D"], buf["z"], slot_idx=slots, **par)

    kept = [pool.clone(), conv_pool.clone()]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    pool.copy_(kept[0])
    conv_pool.copy_(kept[1])
    ys = [y0]
    for t in range(L, L + steps):
        for k in buf:
            buf[k].copy_(s[k][:, t].expand_as(buf[k]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
        ys.append(out[:1, None].clone())
    y = torch.cat(ys, 1)
    xs = ssd.ssd_conv1d_fwd(u, w, bias)
    args = [xs, s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], None, s["dt_bias"], True]
    ry, rf, _, _ = ref.scan(*args)
    my, mf, _, _ = ref.scan(*args, absolute=True)
    ref.check(y, ry, my, k_of(L + steps, N), "y")
    for sl in (0, 2, 5):
        ref.check(pool[sl:sl + 1], rf, mf, k_of(L + steps, N), "state")
    assert float(pool[[1, 3, 4]].abs().sum()) == 0


def test_training_step_under_a_graph():
    """Forward and gradient of conv and scan captured together and replayed with new inputs, with eager work
    between the replays: every replay equals the eager calls."""
    D, N, L = 96, 16, 50
    w, bias = torch.rand(D, 4, device=DEV) - 0.5, torch.rand(D, device=DEV) - 0.5
    sets = [make(2, L, D, 1, N, BF, 90 + i, init=False) for i in range(3)]
    w, bias = w.to(BF), bias.to(BF)
    keys = ("x", "dt", "B", "C", "z", "dy")
    hold = {k: sets[0][k].clone(memory_format=torch.contiguous_format) for k in keys}
    A, Dv, bd = sets[0]["A"], sets[0]["D"], sets[0]["dt_bias"]

    def step(s):
        xs = ssd.ssd_conv1d_fwd(s["x"], w, bias)
        y = ssd.ssd_selective_scan(xs, s["dt"], A, s["B"], s["C"], Dv, s["z"], dt_bias=bd, dt_softplus=True)
        o = ssd.ssd_selective_scan_bwd(s["dy"], xs, s["dt"], A, s["B"], s["C"], Dv, s["z"], dt_bias=bd, dt_softplus=True)
        c = ssd.ssd_conv1d_bwd(o["dx"], s["x"], w, bias)
        return [y] + [v for v in list(o.values()) + list(c.values()) if v is not None]

    step(hold)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(hold)
    for i in (0, 1, 2, 0):
        for k in keys:
            hold[k].copy_(sets[i][k])
        graph.replay()
        torch.cuda.synchronize()
        eager = step({k: sets[i][k].contiguous() for k in keys})
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), i


# ------------------------------------------------------------------------------------ conv's gradient
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [(1, 1, 128), (2, 2, 136), (1, 3, 128), (1, 4, 200), (2, 64, 128), (1, 67, 520), (3, 261, 136), (1, 700, 1032)])
@pytest.mark.parametrize("state", [False, True])
def test_conv_gradient(size, dtype, state):
    Bt, L, CD = size
    g = torch.Generator().manual_seed(60 + L)
    n = lambda *s: torch.randn(*s, generator=g).to(dtype).to(DEV)  # noqa: E731
    xbc, w, dout = n(Bt, L, CD + 16)[..., :CD], n(CD, 4).mul(0.4), n(Bt, L, CD)
    bias = n(CD) if state else None
    st, dso = (n(Bt, CD, 4), n(Bt, CD, 4)) if state else (None, None)
    got = ssd.ssd_conv1d_bwd(dout, xbc, w, bias, st, dso)
    r, m = ref.conv_grad(dout, xbc, w, bias, st, dso), ref.conv_grad(dout, xbc, w, bias, st, dso, absolute=True)
    # per element: 5 roundings of p, 8 of silu' and the product, 5 of the taps; then the sum over tokens
    for name in r:
        assert (got[name] is None) == (r[name] is None), name
        if r[name] is not None:
            ref.check(got[name], r[name], m[name], 32 + (Bt * L if name in ("dw", "dbias") else 0), name)


def test_conv_gradient_without_tokens():
    dso = torch.randn(2, 128, 4, device=DEV)
    e = torch.empty(2, 0, 128, device=DEV)
    got = ssd.ssd_conv1d_bwd(e, e, torch.ones(128, 4, device=DEV), torch.ones(128, device=DEV), torch.ones(2, 128, 4, device=DEV), dso)
    assert torch.equal(got["dconv_state_in"], dso) and float(got["dw"].abs().sum()) == 0 and float(got["dbias"].abs().sum()) == 0


def test_reference_conv_gradient_is_autograds():
    g = torch.Generator().manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    Bt, L, CD = 2, 3, 8
    xbc, w, bias, st = (t.requires_grad_() for t in (n(Bt, L, CD), n(CD, 4), n(CD), n(Bt, CD, 4)))
    dout, dso = n(Bt, L, CD), n(Bt, CD, 4)
    u = torch.cat([st.transpose(1, 2), xbc], 1)
    p = bias + sum(w[:, k] * u[:, 1 + k:1 + k + L] for k in range(4))
    ((p * torch.sigmoid(p) * dout).sum() + (u[:, L:].transpose(1, 2) * dso).sum()).backward()
    r = ref.conv_grad(dout, xbc, w, bias, st, dso)
    for t, k in ((xbc, "dxbc"), (w, "dw"), (bias, "dbias"), (st, "dconv_state_in")):
        assert torch.allclose(t.grad, r[k], rtol=1e-12, atol=1e-12)
