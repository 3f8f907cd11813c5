"""CPU checks of the operators around the scan: the C entry points reject bad
arguments before any HIP call (host pointers that are never dereferenced), and
the binding checks every tensor's shape, type and layout first."""
import ctypes

import numpy as np
import pytest
import torch

import selective_state_space_09_amd as ssd

_buf = np.zeros(1 << 16, np.uint8)
_base = (_buf.ctypes.data + 255) // 256 * 256
_next = [0]


def ptr(off=0, k=None):
    """A 4 KB-apart host address: distinct arrays of a call do not overlap."""
    if k is None:
        _next[0] = (_next[0] + 1) % 15
        k = _next[0]
    return ctypes.c_void_p(_base + 4096 * k + off)


EINVAL, EUNSUP, EWS = ssd.SSD_EINVAL, ssd.SSD_EUNSUPPORTED, ssd.SSD_EWORKSPACE


def call(fn, spec, over):
    a = dict(spec)
    for k, v in over.items():
        assert k in a, k
        a[k] = v
    rc = getattr(ssd.lib(), fn)(*a.values())
    return rc, ssd.lib().ssd_last_error().decode()


def refuse(fn, spec, over, code, needle):
    rc, msg = call(fn, spec, over)
    assert rc == code and needle in msg, (rc, msg)


ADD = dict(x=ptr(), scale=None, residual=ptr(), w=ptr(), eps=1e-5, ro=ptr(), out=ptr(), M=4, D=16, xd=1, rd=0,
           od=1, st=None)


@pytest.mark.parametrize("over,code,needle", [
    (dict(x=None), EINVAL, "x is NULL"), (dict(w=None), EINVAL, "w is NULL"), (dict(out=None), EINVAL, "out is NULL"),
    (dict(M=-1), EINVAL, "M=-1"), (dict(D=0), EINVAL, "D=0"), (dict(D=16385), EUNSUP, "16384"),
    (dict(xd=2), EUNSUP, "x_dtype"), (dict(rd=-1), EUNSUP, "res_dtype"), (dict(od=5), EUNSUP, "out_dtype"),
    (dict(eps=-1.0), EINVAL, "eps"), (dict(eps=float("nan")), EINVAL, "eps"), (dict(eps=float("inf")), EINVAL, "eps"),
    (dict(x=ptr(1)), EINVAL, "x is not 2-byte aligned"), (dict(w=ptr(2)), EINVAL, "w is not 4-byte"),
    (dict(out=ADD["x"]), EINVAL, "overlap"), (dict(ro=ptr(4, k=ADD["residual"] and (ADD["residual"].value - _base) // 4096)), EINVAL, "overlap"),
    (dict(out=ADD["w"]), EINVAL, "out and w overlap"),
])
def test_add_norm_fwd_refuses(over, code, needle):
    refuse("ssd_add_norm_fwd", ADD, over, code, needle)


def test_no_rows_is_fine():
    assert call("ssd_add_norm_fwd", ADD, dict(M=0, x=None, out=None, residual=None, ro=None))[0] == ssd.SSD_OK
    assert call("ssd_gated_norm_fwd", GATED, dict(M=0, y=None, z=None, out=None))[0] == ssd.SSD_OK
    assert call("ssd_mixer_step", STEP, dict(B=0, xbc=None, dt=None, y=None))[0] == ssd.SSD_OK


ADDB = dict(dout=ptr(), dres=None, r=ptr(), x=ptr(), scale=None, w=ptr(), eps=1e-5, dr=ptr(), dx=ptr(), dw=ptr(),
            ds=ptr(), M=4, D=16, xd=1, rd=0, od=1, ws=ptr(), wsb=4096, st=None)


@pytest.mark.parametrize("over,code,needle", [
    (dict(dout=None), EINVAL, "dout is NULL"), (dict(r=None), EINVAL, "r is NULL"), (dict(dw=None), EINVAL, "dw is NULL"),
    (dict(x=None), EINVAL, "x is NULL"), (dict(ws=None), EWS, "workspace"), (dict(wsb=8), EWS, "workspace"),
    (dict(ws=ptr(16)), EINVAL, "256"), (dict(dx=ADDB["dr"]), EINVAL, "overlap"), (dict(dr=ADDB["r"]), EINVAL, "overlap"),
    (dict(dw=ADDB["ds"]), EINVAL, "dw and dscale overlap"), (dict(D=20000), EUNSUP, "16384"),
])
def test_add_norm_bwd_refuses(over, code, needle):
    refuse("ssd_add_norm_bwd", ADDB, over, code, needle)


GATED = dict(y=ptr(), z=ptr(), ldz=16, w=ptr(), eps=1e-5, before=0, out=ptr(), M=4, D=16, G=2, yd=0, zd=1, od=1, st=None)


@pytest.mark.parametrize("over,code,needle", [
    (dict(y=None), EINVAL, "y is NULL"), (dict(z=None), EINVAL, "z is NULL"), (dict(ldz=15), EINVAL, "ldz=15"),
    (dict(ldz=1 << 50), EINVAL, "ldz"), (dict(G=3), EINVAL, "multiple of groups"), (dict(G=0), EINVAL, "groups"),
    (dict(before=2), EINVAL, "norm_before_gate"), (dict(out=GATED["z"]), EINVAL, "overlap"), (dict(zd=9), EUNSUP, "z_dtype"),
    (dict(D=40000, G=2, ldz=40000), EUNSUP, "20000 channels"),
])
def test_gated_norm_fwd_refuses(over, code, needle):
    refuse("ssd_gated_norm_fwd", GATED, over, code, needle)


GATEDB = dict(dout=ptr(), y=ptr(), z=ptr(0, 3), ldz=64, w=ptr(), eps=1e-5, before=0, dy=ptr(), dz=ptr(0, 9), lddz=64,
              dw=ptr(), M=4, D=16, G=2, yd=0, zd=1, od=1, ws=ptr(), wsb=4096, st=None)


@pytest.mark.parametrize("over,code,needle", [
    (dict(dz=None), EINVAL, "dz is NULL"), (dict(lddz=8), EINVAL, "lddz=8"), (dict(wsb=0), EWS, "workspace"),
    (dict(dz=ptr(0, 3)), EINVAL, "dz and z overlap"),
    # 16 columns of 64-wide bf16 rows, 16 bytes into z's own: shared; in other columns of the same rows: fine
    (dict(dz=ptr(16, 3)), EINVAL, "dz and z overlap"), (dict(dz=ptr(128 - 16, 3)), EINVAL, "dz and z overlap"),
])
def test_gated_norm_bwd_refuses(over, code, needle):
    refuse("ssd_gated_norm_bwd", GATEDB, over, code, needle)


CONVB = dict(xbc=ptr(), ld=32, w=ptr(), bias=None, si=None, act=1, dx=ptr(), dB=ptr(), dC=ptr(), dso=None, dxbc=ptr(),
             lddx=32, dw=ptr(), dbias=ptr(), dsi=None, B=1, T=5, HP=16, GN=8, K=4, dtype=1, ws=ptr(), wsb=4096, st=None)


@pytest.mark.parametrize("over,code,needle", [
    (dict(xbc=None), EINVAL, "xbc is NULL"), (dict(dC=None), EINVAL, "dC is NULL"), (dict(K=3), EUNSUP, "K=3"),
    (dict(GN=4), EUNSUP, "GN=4"), (dict(lddx=24), EINVAL, "ld=24"), (dict(act=2), EINVAL, "act"),
    (dict(dtype=3), EUNSUP, "dtype"), (dict(T=-1), EINVAL, "T=-1"), (dict(dw=ptr(8)), EINVAL, "dw is not 16-byte"),
    (dict(wsb=64), EWS, "workspace"), (dict(dxbc=CONVB["xbc"]), EINVAL, "overlap"), (dict(dbias=CONVB["dw"]), EINVAL, "overlap"),
    (dict(B=0), EINVAL, "positive"), (dict(T=(1 << 30) + 1), EUNSUP, "T="),
])
def test_conv_bwd_refuses(over, code, needle):
    refuse("ssd_conv1d_bwd", CONVB, over, code, needle)


STEP = dict(conv=ptr(), h=ptr(), arr=ptr(), slots=None, nslots=2, xbc=ptr(), ldx=48, dt=ptr(), lddt=2, w=ptr(), bias=None,
            act=1, A=ptr(), D=None, dtb=None, lo=0.0, hi=1.0, y=ptr(), yd=0, B=2, H=2, P=8, G=1, N=16, K=4, dtype=0, st=None)


@pytest.mark.parametrize("over,code,needle", [
    (dict(conv=None), EINVAL, "conv_state is NULL"), (dict(h=None), EINVAL, "h is NULL"), (dict(arr=None), EINVAL, "arrivals is NULL"),
    (dict(B=3), EINVAL, "slot map"), (dict(B=-1), EINVAL, "positive"), (dict(nslots=0), EINVAL, "positive"),
    (dict(H=3, G=2), EINVAL, "multiple"), (dict(N=48), EUNSUP, "N=48"), (dict(P=1025), EUNSUP, "P=1025"), (dict(K=2), EUNSUP, "K=2"),
    (dict(ldx=47), EINVAL, "ldx=47"), (dict(lddt=1), EINVAL, "lddt=1"), (dict(lo=2.0), EINVAL, "dt_min"), (dict(yd=3), EUNSUP, "y_dtype"),
    (dict(w=ptr(4)), EINVAL, "w is not 16-byte"), (dict(y=STEP["xbc"]), EINVAL, "overlap"), (dict(h=STEP["conv"]), EINVAL, "overlap"),
])
def test_mixer_step_refuses(over, code, needle):
    refuse("ssd_mixer_step", STEP, over, code, needle)


def test_workspace_sizes_of_refused_shapes():
    assert ssd.ssd_add_norm_bwd_workspace_size(4, 0) == 0
    assert ssd.ssd_add_norm_bwd_workspace_size(-1, 8) == 0
    assert ssd.ssd_gated_norm_bwd_workspace_size(4, 9, 2) == 0
    assert ssd.ssd_conv1d_bwd_workspace_size(0, 4, 8, 8) == 0
    assert ssd.ssd_add_norm_bwd_workspace_size(0, 8) > 0  # no rows: the sums are still written


# ---- the binding, on CPU tensors: shapes and types come before the device ----

def z(*s, t=torch.float32):
    return torch.zeros(*s, dtype=t)


def add_args():
    return dict(x=z(3, 8), w=z(8), residual=z(3, 8), scale=z(8))


def gated_args():
    return dict(y=z(3, 8), z=z(3, 8), w=z(8))


def conv_args():
    return dict(xbc=z(2, 5, 16), w=z(16, 4), dx=z(2, 5, 8), dB=z(2, 5, 4), dC=z(2, 5, 4))


def step_args():
    return dict(conv_state=z(4, 3, 48), h=z(4, 2, 8, 16), arrivals=z(4, 1, t=torch.int32), xbc=z(3, 48), dt=z(3, 2),
                w=z(48, 4), A=z(2))


@pytest.mark.parametrize("fn,args,name,bad", [
    ("ssd_add_norm_fwd", add_args, "w", z(7)), ("ssd_add_norm_fwd", add_args, "residual", z(3, 7)),
    ("ssd_add_norm_fwd", add_args, "scale", z(3, 8)), ("ssd_gated_norm_fwd", gated_args, "z", z(3, 7)),
    ("ssd_gated_norm_fwd", gated_args, "w", z(9)), ("ssd_conv1d_bwd", conv_args, "dC", z(2, 5, 3)),
    ("ssd_conv1d_bwd", conv_args, "dx", z(2, 4, 8)),
    ("ssd_mixer_step", step_args, "conv_state", z(4, 3, 47)),
    ("ssd_mixer_step", step_args, "dt", z(3, 3)), ("ssd_mixer_step", step_args, "arrivals", z(4, 2, t=torch.int32)),
    ("ssd_mixer_step", step_args, "A", z(3)),
])
def test_binding_rejects_shapes(fn, args, name, bad):
    kw = args()
    kw[name] = bad
    with pytest.raises(ValueError, match=f"{name} has shape"):
        getattr(ssd, fn)(**kw)


@pytest.mark.parametrize("fn,args,name,bad", [
    ("ssd_add_norm_fwd", add_args, "x", z(3, 8, t=torch.float16)), ("ssd_add_norm_fwd", add_args, "residual", z(3, 8, t=torch.float64)),
    ("ssd_gated_norm_fwd", gated_args, "z", z(3, 8, t=torch.int32)), ("ssd_mixer_step", step_args, "dt", z(3, 2, t=torch.bfloat16)),
])
def test_binding_rejects_types(fn, args, name, bad):
    kw = args()
    kw[name] = bad
    with pytest.raises(TypeError):
        getattr(ssd, fn)(**kw)


@pytest.mark.parametrize("fn,args", [("ssd_add_norm_fwd", add_args), ("ssd_gated_norm_fwd", gated_args),
                                     ("ssd_conv1d_bwd", conv_args), ("ssd_mixer_step", step_args)])
def test_binding_has_no_cpu_path(fn, args):
    with pytest.raises(ValueError, match="GPU tensor"):
        getattr(ssd, fn)(**args())


@pytest.mark.parametrize("B,H", [((1 << 22) + 1, 2), (2, 1 << 23)])
def test_mixer_step_refuses_a_batch_past_one_grid(B, H):
    refuse("ssd_mixer_step", STEP, dict(B=B, H=H, P=1, ldx=H + 32, lddt=H, nslots=B), EUNSUP, "2^23")


def test_binding_passes_on_an_error_of_a_truth_value():
    with pytest.raises(RuntimeError, match="ambiguous"):
        ssd.ssd_conv1d_bwd(**conv_args(), want_dstate_in=z(2))


IN_PLACE = dict(residual=ADD["residual"], ro=ADD["residual"])  # allowed: residual_out is residual


@pytest.mark.parametrize("over,needle", [
    (dict(out=ADD["residual"], od=0), "out and residual_out overlap"),   # r would be lost
    (dict(x=ADD["residual"], xd=0), "residual_out and x overlap"),
    (dict(w=ADD["residual"]), "residual_out and w overlap"),
    (dict(w=ADD["residual"], M=1), "residual_out and w overlap"),
    (dict(scale=ADD["residual"], M=1), "residual_out and scale overlap"),
    (dict(out=ptr(128, (ADD["residual"].value - _base) // 4096), od=0), "out and residual_out overlap"),
])
def test_add_norm_fwd_in_place_shares_with_nothing_else(over, needle):
    """The update in place excuses residual_out and residual, no other pair of
    arrays at that address."""
    refuse("ssd_add_norm_fwd", ADD, {**IN_PLACE, **over}, EINVAL, needle)


def test_add_norm_fwd_in_place_is_accepted():
    assert call("ssd_add_norm_fwd", ADD, dict(M=0, **IN_PLACE))[0] == ssd.SSD_OK
    rc, msg = call("ssd_add_norm_fwd", ADD, dict(IN_PLACE, out=ADD["x"]))
    assert rc == EINVAL and "out and x overlap" in msg  # no fault found with residual and residual_out


def add_bwd_args():
    return dict(dout=z(3, 8), r=z(3, 8), w=z(8))


def gated_bwd_args():
    return dict(dout=z(3, 8), y=z(3, 8), z=z(3, 8), w=z(8))


@pytest.mark.parametrize("bad", [None, np.zeros((3, 8), np.float32), 1.0])
@pytest.mark.parametrize("fn,args", [
    ("ssd_add_norm_fwd", add_args), ("ssd_add_norm_bwd", add_bwd_args), ("ssd_gated_norm_fwd", gated_args),
    ("ssd_gated_norm_bwd", gated_bwd_args), ("ssd_conv1d_bwd", conv_args), ("ssd_mixer_step", step_args)])
def test_binding_names_what_is_no_tensor(fn, args, bad):
    """Every required tensor, the one whose device the call goes to among them."""
    for name in args():
        if bad is None and name in ("residual", "scale", "arrivals"):
            continue  # may be None
        with pytest.raises(TypeError, match=f"^{name} must be a tensor"):
            getattr(ssd, fn)(**{**args(), name: bad})
