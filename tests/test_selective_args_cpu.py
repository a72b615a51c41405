"""What the per-channel scan, the conv's gradient and the pool calls refuse, on the host (CPU only).

Through the binding with its device check widened to CPU tensors and the library replaced by a recorder
(a well-formed call reaches it once, a malformed one raises ValueError and does not), and through the C
ABI with fake addresses in calls that all fail before anything is launched.
"""
import ctypes

import pytest
import torch

from selective_state_space_conv1d_amd import ssd

bf, f32 = torch.bfloat16, torch.float32
B_, L_, D_, G_, N_ = 2, 8, 48, 2, 32


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def f(*args):
            if name.endswith("_size"):       # size queries launch nothing
                return 64
            self.calls.append(name)
            return 0
        return f


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(ssd, "_DEVICE_TYPES", ("cpu",))
    monkeypatch.setattr(ssd, "_lib", lambda: r)
    monkeypatch.setattr(ssd, "_stream", lambda s: None)
    return r


def t(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


def meta(x):
    return torch.empty(x.shape, dtype=x.dtype, device="meta")


def inputs(*rows):
    bc = t(*rows, 16 + 2 * G_ * N_)
    return dict(x=t(*rows, D_ + 8)[..., 8:], dt=t(*rows, D_), A=t(D_, N_, dtype=f32), D=t(D_, dtype=f32), z=t(*rows, 2 * D_)[..., D_:],
                B=bc[..., 16:16 + G_ * N_].unflatten(-1, (G_, N_)), C=bc[..., 16 + G_ * N_:].unflatten(-1, (G_, N_)),
                dt_bias=t(D_, dtype=f32))


def scan_args():
    return dict(inputs(B_, L_), init_state=t(B_, D_, N_, dtype=f32), final_state=t(B_, D_, N_, dtype=f32), y=t(B_, L_, D_, dtype=f32))


def bwd_args():
    return dict(inputs(B_, L_), dy=t(B_, L_, D_), init_state=t(B_, D_, N_, dtype=f32), dfinal_state=t(B_, D_, N_, dtype=f32))


def update_args():
    return dict(inputs(B_), state=t(5, D_, N_, dtype=f32), slot_idx=torch.zeros(B_, dtype=torch.int32),
                state_out=t(5, D_, N_, dtype=f32), y=t(B_, D_))


def conv_args():
    return dict(dout=t(B_, L_, 200), xbc=t(B_, L_, 208)[..., :200], w=t(200, 4), bias=t(200), conv_state_in=t(B_, 200, 4),
                dconv_state_out=t(B_, 200, 4))


def copy_args():
    i = torch.zeros(3, dtype=torch.int32)
    return dict(dst_pool=t(4, 6, 8), dst_idx=i, src_pool=t(4, 9, 8), src_idx=i, stacked=True)


def clear_args():
    return dict(pool=t(6, 8), slot_idx=torch.zeros(3, dtype=torch.int32))


def wide(*shape):      # a view whose last axis is not packed
    return t(*shape, 2)[..., 0]


COMMON = [("x", lambda a: a["x"].half()), ("x", lambda a: a["x"].float()), ("dt", lambda a: a["dt"].float()),
          ("dt", lambda a: a["dt"][..., :-1]), ("dt", lambda a: meta(a["dt"])), ("A", lambda a: a["A"].to(bf)),
          ("A", lambda a: a["A"][:-1]), ("A", lambda a: t(N_, D_, dtype=f32).t()), ("B", lambda a: a["B"].float()),
          ("B", lambda a: a["B"][..., :1, :]), ("C", lambda a: meta(a["C"])), ("C", lambda a: a["C"].contiguous()),
          ("C", lambda a: a["C"].transpose(-1, -2).contiguous().transpose(-1, -2)), ("D", lambda a: t(D_ + 1, dtype=f32)),
          ("D", lambda a: a["D"].to(bf)), ("z", lambda a: a["z"][..., 1:]), ("z", lambda a: meta(a["z"])),
          ("dt_bias", lambda a: a["dt_bias"].to(bf)), ("dt_bias", lambda a: t(D_ - 1, dtype=f32)), ("x", lambda a: None),
          ("B", lambda a: None), ("A", lambda a: None), ("A", lambda a: a["A"][0]), ("z", lambda a: wide(*a["z"].shape)),
          ("x", lambda a: wide(*a["x"].shape)), ("dt_limit", lambda a: (0.5, 0.1))]
TOKENS = [("x", lambda a: t(B_, L_ + 1, D_)[:, 1:]), ("B", lambda a: t(L_, B_, G_, N_).transpose(0, 1)),
          ("init_state", lambda a: a["init_state"].to(bf)), ("init_state", lambda a: t(B_, N_, D_, dtype=f32).transpose(1, 2)),
          ("workspace", lambda a: torch.empty(64, dtype=torch.uint8, device="meta"))]
CASES = {
    "ssd_selective_scan": (scan_args, COMMON + TOKENS + [
        ("final_state", lambda a: t(B_ + 1, D_, N_, dtype=f32)), ("y", lambda a: t(B_, L_, D_ + 1)), ("y", lambda a: meta(a["y"])),
        ("y", lambda a: t(B_, L_, D_, dtype=torch.float16)), ("y_dtype", lambda a: bf)]),
    "ssd_selective_scan_bwd": (bwd_args, COMMON + TOKENS + [
        ("dy", lambda a: t(B_, L_, D_ + 8)[..., :D_]), ("dy", lambda a: a["dy"][:, :-1]), ("dy", lambda a: a["dy"].half()),
        ("dfinal_state", lambda a: t(B_, D_, N_)), ("dy", lambda a: None)]),
    "ssd_selective_state_update": (update_args, COMMON + [
        ("state", lambda a: a["state"].to(bf)), ("state", lambda a: a["state"][:, :, :-1]), ("slot_idx", lambda a: a["slot_idx"].long()),
        ("slot_idx", lambda a: torch.zeros(B_ + 1, dtype=torch.int32)), ("slot_idx", lambda a: None), ("slot_idx", lambda a: meta(a["slot_idx"])),
        ("state_out", lambda a: t(4, D_, N_, dtype=f32)), ("y", lambda a: t(B_, D_ - 1)), ("state", lambda a: None)]),
    "ssd_conv1d_bwd": (conv_args, [
        ("dout", lambda a: a["dout"].float()), ("dout", lambda a: t(B_, L_, 208)[..., :200]), ("w", lambda a: t(200, 3)),
        ("w", lambda a: t(200, 4, dtype=f32)), ("bias", lambda a: t(199)), ("conv_state_in", lambda a: t(B_, 200, 4, dtype=f32)),
        ("conv_state_in", lambda a: t(B_, 4, 200).transpose(1, 2)), ("dconv_state_out", lambda a: t(B_, 200, 3)),
        ("xbc", lambda a: wide(B_, L_, 200)), ("xbc", lambda a: a["xbc"][0]), ("xbc", lambda a: t(L_, B_, 200).transpose(0, 1)),
        ("dout", lambda a: meta(a["dout"])), ("w", lambda a: None), ("dout", lambda a: None)]),
    "ssd_pool_copy": (copy_args, [
        ("src_pool", lambda a: a["src_pool"].float()), ("src_pool", lambda a: t(4, 9, 16)), ("src_pool", lambda a: t(3, 9, 8)),
        ("dst_pool", lambda a: t(4, 6, 16)[..., :8]), ("dst_idx", lambda a: a["dst_idx"].long()), ("src_idx", lambda a: a["src_idx"][:2]),
        ("src_idx", lambda a: meta(a["src_idx"])), ("dst_pool", lambda a: t(8)), ("dst_idx", lambda a: None), ("dst_pool", lambda a: None),
        ("dst_idx", lambda a: torch.zeros(6, dtype=torch.int32)[::2]), ("dst_idx", lambda a: torch.zeros(3, 1, dtype=torch.int32))]),
    "ssd_pool_clear": (clear_args, [
        ("pool", lambda a: a["pool"].t()), ("slot_idx", lambda a: a["slot_idx"].float()), ("slot_idx", lambda a: meta(a["slot_idx"])),
        ("pool", lambda a: torch.tensor(1.0))]),
    "ssd_pool_compact": (lambda: dict(slot_idx=torch.zeros(3, dtype=torch.int32), nslots=7), [
        ("slot_idx", lambda a: a["slot_idx"].long()), ("slot_idx", lambda a: torch.zeros(6, dtype=torch.int32)[::2]),
        ("slot_idx", lambda a: None)]),
}


@pytest.mark.parametrize("fn", sorted(CASES))
def test_well_formed_call_reaches_the_library(rec, fn):
    getattr(ssd, fn)(**CASES[fn][0]())
    assert rec.calls == [fn]


@pytest.mark.parametrize("fn,i", [(fn, i) for fn in sorted(CASES) for i in range(len(CASES[fn][1]))])
def test_malformed_argument_is_rejected_before_the_library(rec, fn, i):
    make, bad = CASES[fn]
    args = make()
    name, mutate = bad[i]
    args[name] = mutate(args)
    with pytest.raises(ValueError):
        getattr(ssd, fn)(**args)
    assert rec.calls == []


def test_state_out_may_be_the_state_but_not_overlap_it(rec):
    a = update_args()
    both = t(6, D_, N_, dtype=f32)
    ssd.ssd_selective_state_update(**{**a, "state_out": a["state"]})
    with pytest.raises(ValueError):
        ssd.ssd_selective_state_update(**{**a, "state": both[:5], "state_out": both[1:]})
    assert rec.calls == ["ssd_selective_state_update"]


def test_views_whose_single_row_has_any_stride(rec):
    """One batch entry or one token: the strides that are never used do not matter."""
    for rows in ((1, L_), (B_, 1), (1, 1), (0, L_), (B_, 0)):
        a = inputs(rows[0] + 1, rows[1] + 3)
        a = {k: (v[:rows[0], :rows[1]] if v.dim() > 2 or k == "dt" else v) for k, v in a.items()}
        a["dt"] = a["dt"].contiguous()
        assert ssd.ssd_selective_scan(**a).shape == (*rows, D_)


# ----------------------------------------------------------------------------------------------- ABI
P0 = 0x10000      # fake aligned addresses, never dereferenced: every call below fails its checks


def p(i=1, off=0):
    return ctypes.c_void_p(P0 + 0x1000000 * i + off)


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(ssd.LIB_PATH):
        from selective_state_space_conv1d_amd import build_lib
        build_lib.build()
    return ssd.lib_handle()


def dims(**kw):
    d = dict(batch=2, seqlen=300, nheads=128, head_dim=1, ngroups=2, d_state=16, conv_width=4, act_dtype=1, y_dtype=1)
    d.update(kw)
    return ssd.SsdDims(**d)


BIG = 1 << 40
SEL_BAD = [(dict(batch=-1), "SHAPE"), (dict(seqlen=-1), "SHAPE"), (dict(head_dim=2), "SHAPE"), (dict(nheads=129), "SHAPE"),
           (dict(ngroups=0), "SHAPE"), (dict(d_state=8), "UNSUPPORTED"), (dict(d_state=24), "UNSUPPORTED"), (dict(d_state=256), "UNSUPPORTED"),
           (dict(act_dtype=2), "DTYPE"), (dict(y_dtype=5), "DTYPE"), (dict(seqlen=1 << 32), "UNSUPPORTED"),
           (dict(batch=1 << 20, seqlen=1 << 30), "UNSUPPORTED")]


def code(name):
    return ssd.STATUS.index("SSD_ERR_" + name)


def scan_call(lib, d, **kw):
    a = dict(x=p(1), xs=128, dt=p(2), A=p(3), B=p(4), C=p(5), bcs=32, D=None, z=p(6), zs=128, init=None, fin=None, y=p(7), ws=p(8), wsb=BIG)
    a.update(kw)
    return lib.ssd_selective_scan(ctypes.byref(d), a["x"], a["xs"], a["dt"], a["A"], a["B"], a["C"], a["bcs"], a["D"], a["z"], a["zs"],
                                  None, a["init"], a["fin"], a["y"], a["ws"], a["wsb"], None)


def bwd_call(lib, d, **kw):
    a = dict(dy=p(1), x=p(2), xs=128, dt=p(3), A=p(4), B=p(5), C=p(6), bcs=32, D=None, z=p(7), zs=128, init=None, dfin=None, dx=p(8),
             ddt=p(9), dA=p(10), dB=p(11), dC=p(12), dD=None, dz=p(13), dbias=None, dinit=None, ws=p(14), wsb=BIG)
    a.update(kw)
    return lib.ssd_selective_scan_bwd(ctypes.byref(d), a["dy"], a["x"], a["xs"], a["dt"], a["A"], a["B"], a["C"], a["bcs"], a["D"], a["z"],
                                      a["zs"], None, a["init"], a["dfin"], a["dx"], a["ddt"], a["dA"], a["dB"], a["dC"], a["dD"], a["dz"],
                                      a["dbias"], a["dinit"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("call", [scan_call, bwd_call])
def test_selective_scan_refusals(lib, call):
    for kw, want in SEL_BAD:
        assert call(lib, dims(**kw)) == code(want), kw
    for kw, want in [(dict(x=None), "NULL"), (dict(dt=None), "NULL"), (dict(A=None), "NULL"), (dict(B=None), "NULL"), (dict(C=None), "NULL"),
                     (dict(xs=127), "SHAPE"), (dict(zs=127), "SHAPE"), (dict(bcs=24), "SHAPE"), (dict(bcs=36), "ALIGN"),
                     (dict(B=p(4, 8)), "ALIGN"), (dict(C=p(4, 2)), "ALIGN"), (dict(x=p(1, 1)), "ALIGN"), (dict(z=p(1, 1)), "ALIGN"),
                     (dict(A=p(3, 2)), "ALIGN"), (dict(init=p(3, 2)), "ALIGN"), (dict(xs=(1 << 24) + 8), "UNSUPPORTED"),
                     (dict(bcs=(1 << 24) + 8), "UNSUPPORTED")]:
        assert call(lib, dims(), **kw) == code(want), kw
    need = (lib.ssd_selective_scan_workspace_size if call is scan_call else lib.ssd_selective_scan_bwd_workspace_size)(ctypes.byref(dims()))
    assert need > 0
    assert call(lib, dims(), wsb=need - 1) == code("WORKSPACE") and call(lib, dims(), ws=None) == code("WORKSPACE")
    assert call(lib, dims(), ws=p(8, 4)) == code("ALIGN")
    bias = ssd.SsdDtParams(P0 + 2, 0, 0.0, 0.0)
    assert lib.ssd_selective_scan(ctypes.byref(dims()), p(1), 128, p(2), p(3), p(4), p(5), 32, None, None, 0, ctypes.byref(bias), None, None,
                                  p(7), p(8), BIG, None) == code("ALIGN")


def test_selective_scan_own_refusals(lib):
    assert scan_call(lib, dims(), y=None) == code("NULL") and scan_call(lib, dims(), y=p(7, 1)) == code("ALIGN")
    for k in ("dy", "dx", "ddt", "dA", "dB", "dC", "dz"):
        assert bwd_call(lib, dims(), **{k: None}) == code("NULL"), k
        assert bwd_call(lib, dims(), **{k: p(9, 1)}) == code("ALIGN"), k
    for f in (lib.ssd_selective_scan_workspace_size, lib.ssd_selective_scan_bwd_workspace_size, lib.ssd_conv1d_bwd_workspace_size):
        assert f(None) == 0 and f(ctypes.byref(dims(batch=-1))) == 0


def test_update_refusals(lib):
    def call(d, state=p(1), out=p(1), idx=None, nslots=0, x=p(2), xs=128, dt=p(3), A=p(4), B=p(5), C=p(6), bcs=32, z=p(7), zs=128, y=p(8)):
        return lib.ssd_selective_state_update(ctypes.byref(d), state, out, idx, nslots, x, xs, dt, A, B, C, bcs, None, z, zs, None, y, None)
    for kw, want in SEL_BAD:
        if "seqlen" not in kw:
            assert call(dims(**kw)) == code(want), kw
    for kw, want in [(dict(state=None), "NULL"), (dict(out=None), "NULL"), (dict(x=None), "NULL"), (dict(y=None), "NULL"), (dict(dt=None), "NULL"),
                     (dict(A=None), "NULL"), (dict(idx=p(9), nslots=-1), "SHAPE"), (dict(xs=100), "SHAPE"), (dict(bcs=30), "SHAPE"),
                     (dict(zs=100), "SHAPE"), (dict(state=p(1, 4)), "ALIGN"), (dict(out=p(1, 8)), "ALIGN"), (dict(A=p(4, 4)), "ALIGN"),
                     (dict(x=p(2, 1)), "ALIGN"), (dict(B=p(2, 1)), "ALIGN"), (dict(y=p(2, 1)), "ALIGN"),
                     (dict(idx=p(9), nslots=4, state=None), "NULL")]:
        assert call(dims(), **kw) == code(want), kw


def test_conv_gradient_refusals(lib):
    def call(d, xbc=p(1), xs=192, w=p(2), bias=p(3), si=None, dout=p(4), dso=None, dx=p(5), dw=p(6), db=p(7), dsi=None, ws=p(8), wsb=BIG):
        return lib.ssd_conv1d_bwd(ctypes.byref(d), xbc, xs, w, bias, si, dout, dso, dx, dw, db, dsi, ws, wsb, None)
    d = dims(nheads=16, head_dim=8)           # 16 x 8 + 2 x 2 x 16 = 192 channels
    for kw, want in [(dict(xbc=None), "NULL"), (dict(w=None), "NULL"), (dict(dout=None), "NULL"), (dict(dx=None), "NULL"), (dict(dw=None), "NULL"),
                     (dict(xs=191), "SHAPE"), (dict(xs=196), "ALIGN"), (dict(xbc=p(1, 8)), "ALIGN"), (dict(dw=p(6, 4)), "ALIGN"),
                     (dict(dso=p(6, 2)), "ALIGN"), (dict(ws=None), "WORKSPACE"), (dict(wsb=16), "WORKSPACE"), (dict(ws=p(8, 4)), "ALIGN")]:
        assert call(d, **kw) == code(want), kw
    assert call(dims(nheads=18, head_dim=2)) == code("UNSUPPORTED")        # 100 channels
    assert call(dims(nheads=16, head_dim=8, seqlen=1 << 32)) == code("UNSUPPORTED")
    assert call(dims(nheads=16, head_dim=8, conv_width=3)) == code("UNSUPPORTED")


def test_pool_refusals(lib):
    def copy(dst=p(1), dn=8, dls=8 * 64, src=p(2), sn=8, sls=8 * 64, size=64, layers=2, di=p(3), si=p(4), n=3):
        return lib.ssd_pool_copy(dst, dn, dls, src, sn, sls, size, layers, di, si, n, None)
    for kw, want in [(dict(n=-1), "SHAPE"), (dict(dn=-1), "SHAPE"), (dict(size=-16), "SHAPE"), (dict(layers=-1), "SHAPE"), (dict(dls=8 * 64 - 16), "SHAPE"),
                     (dict(sls=0), "SHAPE"), (dict(dst=None), "NULL"), (dict(src=None), "NULL"), (dict(di=None), "NULL"), (dict(si=None), "NULL"),
                     (dict(size=56), "ALIGN"), (dict(dst=p(1, 8)), "ALIGN"), (dict(src=p(1, 4)), "ALIGN"), (dict(dls=8 * 64 + 8), "ALIGN"),
                     (dict(layers=65536), "UNSUPPORTED"), (dict(n=1 << 31), "UNSUPPORTED"), (dict(dn=1 << 31, dls=1 << 40), "UNSUPPORTED"),
                     (dict(n=1 << 20, size=1 << 28, dls=1 << 40, sls=1 << 40), "UNSUPPORTED"),
                     (dict(src=p(1, 64)), "SHAPE"), (dict(src=p(1, 1024 - 64)), "SHAPE"), (dict(src=p(1), sls=8 * 64 + 64), "SHAPE")]:
        assert copy(**kw) == code(want), kw
    for kw, want in [(dict(n=-1), "SHAPE"), (dict(slots=None), "NULL"), (dict(pool=None), "NULL"), (dict(pool=p(1, 8)), "ALIGN"), (dict(size=8), "ALIGN")]:
        a = dict(pool=p(1), nslots=8, ls=512, size=64, layers=2, slots=p(2), n=3)
        a.update(kw)
        assert lib.ssd_pool_clear(a["pool"], a["nslots"], a["ls"], a["size"], a["layers"], a["slots"], a["n"], None) == code(want), kw
    for kw, want in [(dict(n=-1), "SHAPE"), (dict(nslots=-1), "SHAPE"), (dict(nslots=131073), "UNSUPPORTED"), (dict(idx=None), "NULL"), (dict(src=None), "NULL"),
                     (dict(dst=None), "NULL"), (dict(new=None), "NULL"), (dict(count=None), "NULL"), (dict(n=1 << 31), "UNSUPPORTED")]:
        a = dict(idx=p(1), n=3, nslots=9, src=p(2), dst=p(3), new=p(4), count=p(5))
        a.update(kw)
        assert lib.ssd_pool_compact(a["idx"], a["n"], a["nslots"], a["src"], a["dst"], a["new"], a["count"], None) == code(want), kw
