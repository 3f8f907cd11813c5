"""Float64 oracle of the operators around the scan: the residual norm before a
block, the gated norm after the scan, the backward of the causal convolution
and the fused single-token step.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Everything is written
from the operators' definitions in numpy float64; the gradients are the
formulas of the reverse mode, pinned by central differences in the tests.
Inputs are float32 arrays or bfloat16 bit patterns (uint16); results float64.
"""
import numpy as np

from . import _widen, delta as _delta


def _opt(a, default):
    return default if a is None else _widen(a)


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def silu(v):
    return v * sigmoid(v)


def dsilu(v):
    s = sigmoid(v)
    return s * (1.0 + v * (1.0 - s))


def add_norm(x, w, residual=None, scale=None, eps=1e-5):
    """(out, r): r = residual + scale x, out = r / sqrt(mean(r^2) + eps) w."""
    r = _opt(residual, 0.0) + _opt(scale, 1.0) * _widen(x)
    return r / np.sqrt((r * r).mean(-1, keepdims=True) + eps) * _widen(w), r


def _norm_grad(u, dn, eps):
    """Gradient of sum(dn u / sqrt(mean(u^2) + eps)) and the normalised u."""
    rstd = 1.0 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    n = u * rstd
    return rstd * (dn - n * (dn * n).mean(-1, keepdims=True)), n


def add_norm_bwd(dout, r, w, dres=None, scale=None, x=None, eps=1e-5):
    r, dout = _widen(r), _widen(dout)
    g, n = _norm_grad(r, dout * _widen(w), eps)
    g = g + _opt(dres, 0.0)
    axes = tuple(range(r.ndim - 1))
    return dict(dresidual=g, dx=g * _opt(scale, 1.0), dw=(dout * n).sum(axes),
                dscale=None if x is None else (g * _widen(x)).sum(axes))


def _groups(a, groups):
    return a.reshape(a.shape[:-1] + (groups, a.shape[-1] // groups))


def gated_norm(y, z, w, groups=1, eps=1e-5, before=False):
    y, z, w = _widen(y), _widen(z), _widen(w)
    u = _groups(y if before else y * silu(z), groups)
    n = (u / np.sqrt((u * u).mean(-1, keepdims=True) + eps)).reshape(y.shape) * w
    return n * silu(z) if before else n


def gated_norm_bwd(dout, y, z, w, groups=1, eps=1e-5, before=False):
    dout, y, z, w = _widen(dout), _widen(y), _widen(z), _widen(w)
    gate = silu(z)
    u = y if before else y * gate
    dn = dout * w * (gate if before else 1.0)
    du, n = _norm_grad(_groups(u, groups), _groups(dn, groups), eps)
    du, n = du.reshape(y.shape), n.reshape(y.shape)
    dgate = dout * w * n if before else du * y
    axes = tuple(range(y.ndim - 1))
    return dict(dy=du if before else du * gate, dz=dgate * dsilu(z),
                dw=(dout * n * (gate if before else 1.0)).sum(axes))


def conv1d_bwd(xbc, w, dout, bias=None, state_in=None, dstate_out=None, act=1):
    """Gradient of <dout, out> + <dstate_out, state_out> of oracle.conv1d, one
    token at a time: xbc (Bsz,T,Ch), dout (Bsz,T,Ch)."""
    x, w, dout = _widen(xbc), _widen(w), _widen(dout)
    Bsz, T, Ch = x.shape
    seq = np.concatenate([np.zeros((Bsz, 3, Ch)) if state_in is None else _widen(state_in), x], 1)
    dseq = np.zeros_like(seq)
    dw, db = np.zeros((Ch, 4)), np.zeros(Ch)
    for t in range(T):
        v = _opt(bias, 0.0) + sum(w[:, j] * seq[:, t + j] for j in range(4))
        g = dout[:, t] * (dsilu(v) if act else 1.0)
        db += g.sum(0)
        for j in range(4):
            dw[:, j] += (g * seq[:, t + j]).sum(0)
            dseq[:, t + j] += g * w[:, j]
    if dstate_out is not None:
        dseq[:, T:] += _widen(dstate_out)
    return dict(dxbc=dseq[:, 3:], dw=dw, dbias=db, dstate_in=dseq[:, :3])


def mixer_step(conv_state, h, xbc, dt, w, A, G, bias=None, D=None, dt_bias=None, dt_min=0.0,
               dt_max=float("inf"), slots=None, act=1):
    """One token per row on the slots' states: (y, conv_state, h), float64.  A
    row whose slot is outside the pool or taken by an earlier row is padding."""
    conv, h = _widen(conv_state).copy(), _widen(h).copy()
    xbc, dt, w, A = _widen(xbc), _widen(dt), _widen(w), _widen(A)
    nslots, H, P, N = h.shape
    Bsz, HP, GN = xbc.shape[0], H * P, G * N
    y = np.zeros((Bsz, H, P))
    seen = set()
    for b in range(Bsz):
        s = b if slots is None else int(slots[b])
        if not 0 <= s < nslots or s in seen:
            continue
        seen.add(s)
        win = np.concatenate([conv[s], xbc[b][None]])
        v = _opt(bias, 0.0) + (win * w.T).sum(0)
        v = silu(v) if act else v
        conv[s] = win[1:]
        x, Bm, Cm = v[:HP].reshape(H, P), v[HP:HP + GN].reshape(G, N), v[HP + GN:].reshape(G, N)
        for hh in range(H):
            g = hh // (H // G)
            step = float(_delta(dt[b, hh], 0.0 if dt_bias is None else float(dt_bias[hh]), dt_min, dt_max))
            h[s, hh] = np.exp(A[hh] * step) * h[s, hh] + step * np.outer(x[hh], Bm[g])
            y[b, hh] = h[s, hh] @ Cm[g] + (0.0 if D is None else float(D[hh])) * x[hh]
    return y, conv, h
