"""Plain float64 definitions of the per-channel selective scan, its gradient and the conv's gradient (CPU),
with bounds on what fp32 arithmetic may be off by.

Bounds.  Every result is a sum of products of inputs and decays.  Its fp32 evaluation is off by at most
k u times the same sum over absolute values (u = 2^-24, k the roundings along the longest chain), so each
function also returns that sum over absolute values.  Per token a state passes through an exp (argument:
two roundings of at most 2 in magnitude; result: one unit, i.e. 2 u), dt's softplus (8 u) and two products:
16 u with room, hence k = 16 L + N + 64, plus the number of terms in sums over tokens or channels.  An
output stored in bf16 adds half a step, 2^-8 relative to the value."""
import torch

U = 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64)


def dt_of(dt, bias, softplus, limit):
    v = dt if bias is None else dt + bias
    d = torch.ones_like(v)
    if softplus:
        d = torch.sigmoid(v)
        v = torch.where(v > 20, v, torch.log1p(torch.exp(v)))
    if limit is not None:
        d = torch.where((v >= limit[0]) & (v <= limit[1]), d, torch.zeros_like(d))
        v = v.clamp(*limit)
    return v, d


def scan(x, dt, A, B, C, D=None, z=None, init=None, dt_bias=None, softplus=False, limit=None, absolute=False):
    """(y, final state, states after each token [L + 1 entries], dt after the prologue)."""
    x, dt, A, B, C, D, z, init, dt_bias = (f64(t) for t in (x, dt, A, B, C, D, z, init, dt_bias))
    v, _ = dt_of(dt, dt_bias, softplus, limit)
    gate = 1.0 if z is None else z * torch.sigmoid(z)
    if absolute:
        x, B, C = x.abs(), B.abs(), C.abs()
        D, init = (None if t is None else t.abs() for t in (D, init))
        gate = gate.abs() if z is not None else gate
    Bt, L, Dc = x.shape
    r = Dc // B.shape[2]
    h = torch.zeros(Bt, Dc, A.shape[1], dtype=torch.float64) if init is None else init
    hs, ys = [h], []
    for t in range(L):
        h = torch.exp(v[:, t, :, None] * A) * h + (v[:, t] * x[:, t])[..., None] * B[:, t].repeat_interleave(r, 1)
        hs.append(h)
        ys.append((h * C[:, t].repeat_interleave(r, 1)).sum(-1))
    y = torch.stack(ys, 1) if L else torch.zeros_like(x)
    if D is not None:
        y = y + D * x
    return y * gate, h, hs, v


def scan_grad(dy, x, dt, A, B, C, D=None, z=None, init=None, dfinal=None, dt_bias=None, softplus=False, limit=None,
              absolute=False):
    """The gradients by the recurrence's formulas, as a dict; absolute: every term by its absolute value."""
    _, _, hs, v = scan(x, dt, A, B, C, D, z, init, dt_bias, softplus, limit, absolute)
    y, _, _, _ = scan(x, dt, A, B, C, D, None, init, dt_bias, softplus, limit, absolute)
    dy, x, dt, A, B, C, D, z, dfinal, bias = (f64(t) for t in (dy, x, dt, A, B, C, D, z, dfinal, dt_bias))
    m = (lambda t: None if t is None else t.abs()) if absolute else (lambda t: t)
    dy, x, B, C, D, dfinal = m(dy), m(x), m(B), m(C), m(D), m(dfinal)
    Bt, L, Dc = x.shape
    G, N = B.shape[2:]
    r = Dc // G
    o = {"dz": None}
    if z is not None:
        sg = torch.sigmoid(z)
        o["dz"] = dy * y * (sg * (1 + z.abs()) if absolute else sg * (1 + z * (1 - sg)))
        dy = dy * m(z * sg)
    _, dv = dt_of(dt, bias, softplus, limit)
    g = torch.zeros(Bt, Dc, N, dtype=torch.float64) if dfinal is None else dfinal
    skip = 0.0 if D is None else D
    dx, ddt, dB, dC = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(B), torch.zeros_like(C)
    dA = torch.zeros_like(A)
    for t in reversed(range(L)):
        Bd, Cd = B[:, t].repeat_interleave(r, 1), C[:, t].repeat_interleave(r, 1)
        a = torch.exp(v[:, t, :, None] * A)
        g = g + dy[:, t, :, None] * Cd
        q = a * hs[t]
        dx[:, t] = skip * dy[:, t] + v[:, t] * (g * Bd).sum(-1)
        ddt[:, t] = ((g * q * m(A)).sum(-1) + x[:, t] * (g * Bd).sum(-1)) * dv[:, t]
        dB[:, t] = (g * (v[:, t] * x[:, t])[..., None]).reshape(Bt, G, r, N).sum(2)
        dC[:, t] = (hs[t + 1] * dy[:, t, :, None]).reshape(Bt, G, r, N).sum(2)
        dA += (g * q * v[:, t, :, None]).sum(0)
        g = a * g
    o.update(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=None if D is None else (dy * x).sum((0, 1)),
             ddt_bias=None if bias is None else ddt.sum((0, 1)), dinit_state=None if init is None else g)
    return o


def conv_grad(dout, xbc, w, bias=None, state=None, dstate_out=None, absolute=False):
    dout, xbc, w, bias, state, dso = (f64(t) for t in (dout, xbc, w, bias, state, dstate_out))
    Bt, L, CD = xbc.shape
    st = torch.zeros(Bt, CD, 4, dtype=torch.float64) if state is None else state
    u = torch.cat([st.transpose(1, 2), xbc], 1)              # u[:, 4 + t] is token t
    p = torch.zeros_like(xbc) if bias is None else bias + torch.zeros_like(xbc)
    pa = p.abs()
    for k in range(4):
        p = p + w[:, k] * u[:, 1 + k:1 + k + L]
        pa = pa + (w[:, k] * u[:, 1 + k:1 + k + L]).abs()
    sg = torch.sigmoid(p)
    q = dout * sg * (1 + p * (1 - sg))
    if absolute:       # |silu'| <= 1.1, |silu''| <= 1/2: what an error of p's terms makes of q
        q, u, w = dout.abs() * (1.1 + pa), u.abs(), w.abs()
        dso = None if dso is None else dso.abs()
    du, dw = torch.zeros_like(u), torch.zeros(CD, 4, dtype=torch.float64)
    for k in range(4):
        du[:, 1 + k:1 + k + L] += w[:, k] * q
        dw[:, k] = (q * u[:, 1 + k:1 + k + L]).sum((0, 1))
    if dso is not None:
        du[:, L:] += dso.transpose(1, 2)                     # the window holds the last four of (state, inputs)
    return dict(dxbc=du[:, 4:], dw=dw, dbias=None if bias is None else q.sum((0, 1)),
                dconv_state_in=None if state is None else du[:, :4].transpose(1, 2))


def check(got, ref, mag, k, what=""):
    """got within k u mag of ref, elementwise, plus half a step of got's type where it is narrower."""
    assert tuple(got.shape) == tuple(ref.shape), (what, got.shape, ref.shape)
    g = f64(got)
    tol = k * U * mag + (0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2 * (ref.abs() + k * U * mag))
    tol = tol + 2.0 ** -126      # results below the smallest normal number may be flushed to zero
    bad = ~((g - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst {float(((g - ref).abs() / tol).max()):.2f} x the bound"
