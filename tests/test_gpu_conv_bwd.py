"""GPU parity of the causal convolution's backward against the float64 oracle.

Roundings (c of the bars, in units of 2^-24): v is 4 products and a bias (5),
the sigmoid of the hardware exponential and reciprocal at |v| < 12 (1.5 |v| + 6
= 24), the derivative and the product with dout (6), four products summed (5):
C = 40.  Since v's error moves the derivative by at most |v error| (|SiLU''| <=
1/2), v's own magnitude enters through it: the bars' magnitude takes
|dout| (1 + sum |w in| + |bias|).  A sum over n tokens adds at most n / 8 + 80
terms in sequence: a wave's tokens (one run of 8 to 32 and its first three; past
1024 runs in a call n / 1024 and at most a run more), 4 waves, then at most 256
parts in 16 chains and the chains."""
import numpy as np
import pytest
import torch

import selective_state_space_09_amd as ssd
from oracle import layer
from _layer import normal, rows_in, wide, within
import _gpu

pytestmark = pytest.mark.gpu
C = 40

CASES = [
    # Bsz, T, HP, GN, ld, col, type, act, state, bias
    (2, 44, 32, 8, 48, 0, "bf16", 1, True, True),
    (1, 1, 8, 8, 24, 0, "f32", 0, True, False),       # one token
    (3, 2, 16, 0, 16, 0, "f32", 1, True, True),       # no B and C, shorter than the kernel
    (1, 3, 16, 8, 40, 8, "bf16", 1, True, True),
    (2, 0, 16, 8, 32, 0, "f32", 1, True, True),       # no tokens: the state's gradient passes through
    (2, 31, 64, 16, 104, 8, "f32", 1, False, True),   # one token short of four runs of 8
    (1, 33, 64, 16, 96, 0, "bf16", 1, False, False),  # one past them
    (2, 200, 96, 16, 136, 8, "bf16", 1, False, True),
    (1, 70, 512, 64, 704, 64, "bf16", 1, True, True),
    (2, 129, 512, 64, 640, 0, "f32", 1, True, True),
    (1, 257, 64, 32, 128, 0, "f32", 0, True, True),
    (300, 5, 64, 8, 80, 0, "bf16", 1, True, True),    # many sequences shorter than a run: 75 parts of 4
]


def case(Bsz, T, HP, GN, t, state, bias):
    rng = np.random.default_rng(T + HP + Bsz)
    Ch = HP + 2 * GN
    return dict(xbc=normal(rng, (Bsz, T, Ch), t), w=normal(rng, (Ch, 4), mul=0.5),
                dx=normal(rng, (Bsz, T, HP), t), dB=normal(rng, (Bsz, T, GN)), dC=normal(rng, (Bsz, T, GN)),
                bias=normal(rng, Ch, mul=0.5) if bias else None,
                state_in=normal(rng, (Bsz, 3, Ch)) if state else None,
                dstate_out=normal(rng, (Bsz, 3, Ch)) if state else None)


@pytest.mark.parametrize("Bsz,T,HP,GN,ld,col,t,act,state,bias", CASES)
def test_conv_bwd(Bsz, T, HP, GN, ld, col, t, act, state, bias):
    print(f"conv_bwd Bsz={Bsz} T={T} HP={HP} GN={GN} ld={ld} {t} act={act}", flush=True)
    a = case(Bsz, T, HP, GN, t, state, bias)
    Ch = HP + 2 * GN
    dout = np.concatenate([wide(a["dx"]), wide(a["dB"]), wide(a["dC"])], 2)
    args = (a["xbc"], a["w"], dout, a["bias"], a["state_in"], a["dstate_out"], act)
    ref = layer.conv1d_bwd(*args)
    xv, _ = rows_in(a["xbc"], ld, col, fill=float("nan"))
    ov, buf = rows_in(np.zeros_like(a["xbc"]), ld, col, fill=7.0)
    d = {k: _gpu.to_dev(v) for k, v in a.items() if k != "xbc"}
    got = ssd.ssd_conv1d_bwd(xv, d["w"], d["dx"], d["dB"], d["dC"], bias=d["bias"], state_in=d["state_in"],
                             dstate_out=d["dstate_out"], act=act, dxbc=ov)
    # magnitudes: the same formulas on absolute values, without the activation
    ab = lambda v: None if v is None else np.abs(wide(v))  # noqa: E731
    seq = np.concatenate([np.zeros((Bsz, 3, Ch)) if not state else ab(a["state_in"]), ab(a["xbc"])], 1)
    v = 1.0 + (0.0 if not bias else ab(a["bias"])) + sum(ab(a["w"])[:, j] * seq[:, j:j + T] for j in range(4))
    mag = layer.conv1d_bwd(ab(a["xbc"]), ab(a["w"]), np.abs(dout) * v, None, ab(a["state_in"]), ab(a["dstate_out"]), 0)
    n = Bsz * T / 8 + 80
    within(got["dxbc"], ref["dxbc"], t, C, mag["dxbc"], "dxbc")
    within(got["dstate_in"], ref["dstate_in"], "f32", C, mag["dstate_in"], "dstate_in")
    within(got["dw"], ref["dw"], "f32", C + n, mag["dw"], "dw")
    within(got["dbias"], ref["dbias"], "f32", C + n, mag["dbias"], "dbias")
    keep = torch.ones(ld, dtype=torch.bool)
    keep[col:col + Ch] = False
    assert bool((buf[..., keep.cuda()] == 7.0).all())
    # again, without the state's gradient: the same bits
    less = ssd.ssd_conv1d_bwd(xv, d["w"], d["dx"], d["dB"], d["dC"], bias=d["bias"], state_in=d["state_in"],
                              dstate_out=d["dstate_out"], act=act, want_dstate_in=False)
    assert less["dstate_in"] is None
    for k in ("dw", "dbias"):
        assert torch.equal(less[k], got[k])
    assert torch.equal(less["dxbc"], got["dxbc"])


def test_conv_bwd_segments_chain():
    """A sequence cut in two, the second segment's dstate_in handed to the
    first as dstate_out, has the gradient of the whole one (float32: bars of
    two roundings' difference)."""
    torch.manual_seed(1)
    HP, GN, T, cut = 64, 16, 77, 40
    Ch = HP + 2 * GN
    x, w, b = torch.randn(2, T, Ch, device="cuda"), torch.randn(Ch, 4, device="cuda") * 0.5, torch.randn(Ch, device="cuda")
    gx, gB, gC = (torch.randn(2, T, n, device="cuda") for n in (HP, GN, GN))
    whole = ssd.ssd_conv1d_bwd(x, w, gx, gB, gC, bias=b)
    sl = lambda t, s: t[:, s].contiguous()  # noqa: E731
    first, second = slice(0, cut), slice(cut, T)
    st = sl(x, first)[:, -3:].contiguous()
    g2 = ssd.ssd_conv1d_bwd(sl(x, second), w, sl(gx, second), sl(gB, second), sl(gC, second), bias=b, state_in=st)
    g1 = ssd.ssd_conv1d_bwd(sl(x, first), w, sl(gx, first), sl(gB, first), sl(gC, first), bias=b,
                            dstate_out=g2["dstate_in"])
    d = torch.cat([g1["dxbc"], g2["dxbc"]], 1)
    assert float((d - whole["dxbc"]).abs().max()) <= 16 * 2.0 ** -24 * float(whole["dxbc"].abs().max())
    for k in ("dw", "dbias"):
        s = (g1[k] + g2[k])
        assert float((s - whole[k]).abs().max()) <= 2 * T * 2.0 ** -24 * float(whole[k].abs().max())


def test_conv_bwd_stream_graph_and_workspace():
    torch.manual_seed(2)
    HP, GN = 128, 32
    x, w, b = torch.randn(2, 100, HP + 2 * GN, device="cuda"), torch.randn(HP + 2 * GN, 4, device="cuda"), torch.randn(HP + 2 * GN, device="cuda")
    gx, gB, gC = (torch.randn(2, 100, n, device="cuda") for n in (HP, GN, GN))
    step = lambda **k: list(ssd.ssd_conv1d_bwd(x, w, gx, gB, gC, bias=b, **k).values())  # noqa: E731
    ref = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws = torch.full((ssd.ssd_conv1d_bwd_workspace_size(2, 100, HP, GN),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = step(stream=side, workspace=ws)  # a workspace full of NaN patterns
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(3):
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, step())), k


LONG = [
    # Bsz, T, HP, GN, ld, col, type, state; run lengths as the plan has them at this writing
    (9, 301, 2048, 64, 2184, 8, "f32", True),      # runs of 12, the last of one token
    (7, 301, 4096, 128, 4352, 0, "bf16", False),   # 16
    (4, 1203, 2048, 64, 2176, 0, "f32", True),     # 20, the last of three
    (5, 1203, 2048, 64, 2184, 8, "bf16", True),    # 24, the last of three
    (2, 2048, 4096, 128, 8512, 4096, "bf16", True),  # 28: the bf16 layer, in in_proj rows
    (4, 2049, 2048, 64, 2176, 0, "bf16", True),    # 32, the last of one token
    # more (sequence, run) units than a wave of the grid has one each
    (8, 4096, 64, 8, 80, 0, "bf16", True),
    (1, 20000, 32, 8, 56, 8, "f32", True),
]


@pytest.mark.parametrize("Bsz,T,HP,GN,ld,col,t,state", LONG)
def test_conv_bwd_long_runs(Bsz, T, HP, GN, ld, col, t, state):
    test_conv_bwd(Bsz, T, HP, GN, ld, col, t, 1, state, True)


@pytest.mark.parametrize("T,t", [(5, "bf16"), (11, "f32")])
def test_conv_bwd_more_units_than_waves(T, t):
    """Sequences enough that every wave walks several: twice the largest
    partial-sum table's rows times four waves, and some more."""
    HP, GN = 64, 8
    parts = ssd.ssd_conv1d_bwd_workspace_size(65535, T, HP, GN) // (20 * (HP + 2 * GN))
    test_conv_bwd(4 * parts * 2 + 77, T, HP, GN, 80, 0, t, 1, True, True)


def test_conv_bwd_past_32_bit_offsets():
    """One sequence of 2^31 + elements with gradients at its two ends: rows,
    sums and the carried state's gradient against the oracle on the ends, and
    no gradient between them."""
    HP, GN, T, E, Z = 2032, 8, (1 << 20) + 40, 48, 8  # ends of 48 tokens, the inner 8 without gradient
    Ch = HP + 2 * GN
    rng = np.random.default_rng(10)
    w, bias, st, dso = normal(rng, (Ch, 4), mul=0.5), normal(rng, Ch, mul=0.5), normal(rng, (1, 3, Ch)), normal(rng, (1, 3, Ch))
    ends = [dict(x=normal(rng, (1, E, Ch), "bf16"), dx=normal(rng, (1, E, HP), "bf16"), dB=normal(rng, (1, E, GN)),
                 dC=normal(rng, (1, E, GN))) for _ in range(2)]
    for e, quiet in zip(ends, (slice(E - Z, E), slice(0, Z))):
        for k in ("dx", "dB", "dC"):
            e[k][:, quiet] = 0
    make = lambda n, t, fill: torch.full((1, T, n), fill, dtype=t, device="cuda")  # noqa: E731
    d = dict(x=make(Ch, torch.bfloat16, 1.0), dx=make(HP, torch.bfloat16, 0.0), dB=make(GN, torch.float32, 0.0),
             dC=make(GN, torch.float32, 0.0))
    for k, v in d.items():
        v[:, :E], v[:, -E:] = _gpu.to_dev(ends[0][k]), _gpu.to_dev(ends[1][k])
    up = _gpu.to_dev
    got = ssd.ssd_conv1d_bwd(d["x"], up(w), d["dx"], d["dB"], d["dC"], bias=up(bias), state_in=up(st), dstate_out=up(dso))
    ones = np.ones((1, 3, Ch), np.float32)  # the inputs before the last tokens
    sums = {}
    for e, s, o, rows in ((ends[0], st, None, slice(0, E)), (ends[1], ones, dso, slice(T - E, T))):
        dout = np.concatenate([wide(e["dx"]), e["dB"], e["dC"]], 2).astype(np.float64)
        ref = layer.conv1d_bwd(e["x"], w, dout, bias, s, o, 1)
        seq = np.concatenate([np.abs(wide(s)), np.abs(wide(e["x"]))], 1)
        v = 1.0 + np.abs(wide(bias)) + sum(np.abs(wide(w))[:, j] * seq[:, j:j + E] for j in range(4))
        mag = layer.conv1d_bwd(seq[:, 3:], np.abs(w), np.abs(dout) * v, None, seq[:, :3], None if o is None else np.abs(o), 0)
        within(got["dxbc"][:, rows], ref["dxbc"], "bf16", C, mag["dxbc"], "dxbc")
        if o is None:
            within(got["dstate_in"], ref["dstate_in"], "f32", C, mag["dstate_in"], "dstate_in")
        for k in ("dw", "dbias"):
            a, b = sums.get(k, (0.0, 0.0))
            sums[k] = a + ref[k], b + mag[k]
    assert float(got["dxbc"][:, E:T - E].abs().max()) == 0.0
    for k, (ref, mag) in sums.items():  # the terms between the ends are zeros, which add no rounding
        within(got[k], ref, "f32", C + 2 * E / 8 + 80, mag, k)
