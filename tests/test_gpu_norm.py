"""GPU parity of the residual norm and the gated norm, forward and backward,
against the float64 oracle.

Roundings on the longest path (c of the bars, in units of 2^-24): a sum of
squares adds at most 32 terms in a lane, 10 steps over lanes and waves, all of
one sign, so its relative error is below 46; half of that reaches 1/sqrt, plus
2 for the hardware reciprocal root: 25.  Products and the r = residual + scale x
before it add less than 15: C_FWD = 40.  The gate adds 1.5 |z| + 6 below |z| =
12 (the exponent's argument is rounded): 24 more.  A gradient holds a second
such sum, of terms of both signs, so its bar's magnitude takes their absolute
values: C_BWD = 2 * 40 + 24.  A sum over M rows adds at most M / 16 + 80 terms
in sequence (rows of a team, teams, parts)."""
import numpy as np
import pytest
import torch

import selective_state_space_09_amd as ssd
from oracle import layer
from _layer import TYPES, normal, rows_in, wide, within
import _gpu

pytestmark = pytest.mark.gpu

C_FWD, C_GATE, C_BWD = 40, 64, 104
EPS = 1e-5


def rows_c(M):
    return M / 16 + 80 + C_BWD


ADD = [
    # M, D, x, residual's, out's type, residual?, scale?
    (1, 2048, "bf16", "f32", "bf16", True, True),
    (5, 1, "f32", "f32", "f32", True, True),            # one channel: out is +-w
    (3, 7, "bf16", "bf16", "bf16", True, False),        # shorter than a vector
    (9, 128, "f32", "bf16", "f32", True, True),         # a full 16-lane team
    (7, 129, "bf16", "f32", "f32", False, True),        # one channel past it
    (33, 512, "f32", "f32", "bf16", True, False),
    (6, 1001, "bf16", "bf16", "f32", True, True),       # odd rows: 2-byte aligned vectors
    (130, 1027, "f32", "f32", "f32", True, True),
    (17, 2049, "bf16", "f32", "bf16", True, True),      # a workgroup per row
    (4, 4096, "f32", "f32", "bf16", False, False),
    (3, 8191, "bf16", "f32", "bf16", True, True),
    (2, 16384, "bf16", "bf16", "bf16", True, True),     # the longest row
    (2, 16383, "f32", "f32", "f32", True, True),
    (5000, 64, "bf16", "f32", "bf16", True, True),      # many short rows, one to a team: partial sums over 157 parts
]


def add_case(M, D, x, res, out, with_res, with_scale, seed=0):
    rng = np.random.default_rng(1000 * M + D + seed)
    return dict(x=normal(rng, (M, D), x), w=normal(rng, D, mul=0.2, add=1.0),
                residual=normal(rng, (M, D), res, mul=2.0) if with_res else None,
                scale=normal(rng, D, mul=0.5) if with_scale else None)


@pytest.mark.parametrize("M,D,x,res,out,with_res,with_scale", ADD)
def test_add_norm_fwd(M, D, x, res, out, with_res, with_scale):
    print(f"add_norm_fwd M={M} D={D} {x} {res} {out} {with_res} {with_scale}", flush=True)
    a = add_case(M, D, x, res, out, with_res, with_scale)
    ref, r = layer.add_norm(eps=EPS, **a)
    d = {k: _gpu.to_dev(v) for k, v in a.items()}
    got, gr = ssd.ssd_add_norm_fwd(d["x"], d["w"], residual=d["residual"], scale=d["scale"], eps=EPS,
                                   out_dtype=TYPES[out], res_dtype=TYPES[res])
    mag = np.abs(wide(a["x"]) * (1.0 if a["scale"] is None else wide(a["scale"])))
    mag = mag + (0.0 if a["residual"] is None else np.abs(wide(a["residual"])))
    rstd = 1 / np.sqrt((r * r).mean(-1, keepdims=True) + EPS)
    within(gr, r, res, 2, mag, "r")
    # r's own rounding errors reach out through r and, at worst times mean(mag |r|) rstd^2, through rstd
    amp = mag * rstd + np.abs(r) * rstd ** 3 * (mag * np.abs(r)).mean(-1, keepdims=True)
    within(got, ref, out, C_FWD, np.abs(wide(a["w"])) * amp, "out")


@pytest.mark.parametrize("M,D,x,res,out,with_res,with_scale", ADD)
def test_add_norm_bwd(M, D, x, res, out, with_res, with_scale):
    print(f"add_norm_bwd M={M} D={D} {x} {res} {out} {with_res} {with_scale}", flush=True)
    a = add_case(M, D, x, res, out, with_res, with_scale)
    rng = np.random.default_rng(D + 7)
    r = normal(rng, (M, D), res, mul=2.0)
    dout = normal(rng, (M, D), out)
    dres = normal(rng, (M, D), res) if with_res else None
    ref = layer.add_norm_bwd(dout, r, a["w"], dres=dres, scale=a["scale"], x=a["x"], eps=EPS)
    d = {k: _gpu.to_dev(v) for k, v in a.items()}
    got = ssd.ssd_add_norm_bwd(_gpu.to_dev(dout), _gpu.to_dev(r), d["w"], dres=_gpu.to_dev(dres), scale=d["scale"],
                               x=d["x"], eps=EPS)
    R, rstd = wide(r), None
    rstd = 1 / np.sqrt((R * R).mean(-1, keepdims=True) + EPS)
    n, dn = np.abs(R * rstd), np.abs(wide(dout) * wide(a["w"]))
    mag = rstd * (dn + n * (dn * n).mean(-1, keepdims=True)) + (0.0 if dres is None else np.abs(wide(dres)))
    scale = 1.0 if a["scale"] is None else np.abs(wide(a["scale"]))
    within(got["dresidual"], ref["dresidual"], res, C_BWD, mag, "dresidual")
    within(got["dx"], ref["dx"], x, C_BWD, mag * scale, "dx")
    within(got["dw"], ref["dw"], "f32", rows_c(M), (np.abs(wide(dout)) * n).sum(0), "dw")
    within(got["dscale"], ref["dscale"], "f32", rows_c(M), (mag * np.abs(wide(a["x"]))).sum(0), "dscale")
    # without x there is no dscale, and the rest is the same, bit for bit
    less = ssd.ssd_add_norm_bwd(_gpu.to_dev(dout), _gpu.to_dev(r), d["w"], dres=_gpu.to_dev(dres), scale=d["scale"],
                                x_dtype=TYPES[x], eps=EPS)
    assert less["dscale"] is None
    for k in ("dresidual", "dx", "dw"):
        assert torch.equal(less[k], got[k]), k


GATED = [
    # M, D, groups, ld, col, y, z, out, before
    (1, 4096, 1, 8512, 0, "f32", "bf16", "bf16", False),
    (37, 4096, 8, 8512, 0, "bf16", "bf16", "bf16", False),
    (5, 24, 3, 24, 0, "f32", "f32", "f32", True),
    (5, 1, 1, 3, 1, "f32", "f32", "f32", False),         # one channel
    (9, 1001, 1, 2003, 5, "bf16", "bf16", "f32", False),  # odd rows, odd stride, odd offset
    (12, 1027, 1, 1040, 3, "f32", "f32", "f32", True),
    (6, 6000, 2, 6001, 1, "bf16", "f32", "bf16", True),   # two norms of 3000
    (3, 16384, 1, 16384, 0, "bf16", "bf16", "bf16", False),
    (700, 520, 65, 600, 40, "f32", "bf16", "f32", False),  # 65 groups of 8
    (5000, 128, 2, 128, 0, "bf16", "bf16", "bf16", False),
]


def gated_case(M, D, groups, ld, col, y, z, out):
    rng = np.random.default_rng(M + 31 * D + groups)
    return (normal(rng, (M, D), y), normal(rng, (M, D), z, mul=2.0), normal(rng, D, mul=0.2, add=1.0),
            normal(rng, (M, D), out))


def grp(a, groups):
    return a.reshape(a.shape[0], groups, -1)


@pytest.mark.parametrize("M,D,groups,ld,col,y,z,out,before", GATED)
def test_gated_norm_fwd(M, D, groups, ld, col, y, z, out, before):
    print(f"gated_norm_fwd M={M} D={D} groups={groups} ld={ld} {y} {z} {out} {before}", flush=True)
    ya, za, w, _ = gated_case(M, D, groups, ld, col, y, z, out)
    ref = layer.gated_norm(ya, za, w, groups, EPS, before)
    zv, _ = rows_in(za, ld, col, fill=float("nan"))  # the other columns are never read
    got = ssd.ssd_gated_norm_fwd(_gpu.to_dev(ya), zv, _gpu.to_dev(w), groups=groups, eps=EPS,
                                 norm_before_gate=before, out_dtype=TYPES[out])
    within(got, ref, out, C_GATE, np.abs(ref), "out")  # no sums but of squares: relative


@pytest.mark.parametrize("M,D,groups,ld,col,y,z,out,before", GATED)
def test_gated_norm_bwd(M, D, groups, ld, col, y, z, out, before):
    print(f"gated_norm_bwd M={M} D={D} groups={groups} ld={ld} {y} {z} {out} {before}", flush=True)
    ya, za, w, dout = gated_case(M, D, groups, ld, col, y, z, out)
    ref = layer.gated_norm_bwd(dout, ya, za, w, groups, EPS, before)
    zv, _ = rows_in(za, ld, col, fill=float("nan"))
    dzv, buf = rows_in(np.zeros_like(za), ld, col, fill=7.0)
    got = ssd.ssd_gated_norm_bwd(_gpu.to_dev(dout), _gpu.to_dev(ya), zv, _gpu.to_dev(w), groups=groups, eps=EPS,
                                 norm_before_gate=before, dz=dzv)
    Y, Z, W, DO = (np.abs(wide(v)) for v in (ya, za, w, dout))
    zs = wide(za)
    sig = layer.sigmoid(zs)
    gate, dgate = Z * sig, sig * (1 + Z * (1 - sig))
    u = Y if before else Y * gate
    dn = DO * W * (gate if before else 1.0)
    rstd = 1 / np.sqrt((grp(u, groups) ** 2).mean(-1, keepdims=True) + EPS)
    n = grp(u, groups) * rstd
    du = (rstd * (grp(dn, groups) + n * (grp(dn, groups) * n).mean(-1, keepdims=True))).reshape(M, D)
    n = n.reshape(M, D)
    within(got["dy"], ref["dy"], y, C_BWD, du if before else du * gate, "dy")
    within(got["dz"], ref["dz"], z, C_BWD, (DO * W * n if before else du * Y) * dgate, "dz")
    within(got["dw"], ref["dw"], "f32", rows_c(M), (DO * n * (gate if before else 1.0)).sum(0), "dw")
    keep = torch.ones(ld, dtype=torch.bool)
    keep[col:col + D] = False
    assert bool((buf[:, keep.cuda()] == 7.0).all())  # columns beside dz stay


def test_norms_of_zero_rows_and_large_values():
    """A row of zeros gives zeros (eps keeps it finite); values of 1e17 keep
    their squares inside float32; an infinity or NaN stays in its own row."""
    D = 300
    x = torch.zeros(5, D, device="cuda")
    x[1] = 1e17
    x[2, 7] = float("inf")
    x[3, 9] = float("nan")
    x[4] = torch.arange(D, device="cuda")
    w = torch.ones(D, device="cuda")
    out, r = ssd.ssd_add_norm_fwd(x, w)
    assert torch.equal(r[4], x[4]) and float(out[0].abs().max()) == 0.0
    np.testing.assert_allclose(out[1].cpu().numpy(), 1.0, rtol=40 * 2.0 ** -24)
    alone, _ = ssd.ssd_add_norm_fwd(x[4:], w)
    assert torch.equal(out[4], alone[0])
    assert bool(out[3].isnan().all())
    g = ssd.ssd_add_norm_bwd(torch.ones_like(x), x, w)
    assert bool(g["dresidual"][[0, 1, 4]].isfinite().all())
    # a closed gate (z very negative) and a far open one, both signs of y
    y = torch.tensor([[1.0, -2.0, 3.0, -4.0]], device="cuda")
    z = torch.tensor([[-300.0, 300.0, -90.0, 90.0]], device="cuda")
    w4 = torch.ones(4, device="cuda")
    ref = layer.gated_norm(y.cpu().numpy(), z.cpu().numpy(), w4.cpu().numpy())
    np.testing.assert_allclose(ssd.ssd_gated_norm_fwd(y, z, w4).cpu().numpy(), ref, rtol=1e-5, atol=1e-30)
    gz = ssd.ssd_gated_norm_bwd(torch.ones_like(y), y, z, w4)
    assert bool(gz["dz"].isfinite().all() and gz["dy"].isfinite().all())


def test_norm_shapes_strides_and_empty_batches():
    dev = "cuda"
    proj = torch.randn(3, 4, 40, device=dev)
    y, w = torch.randn(3, 4, 16, device=dev), torch.randn(16, device=dev)
    z = proj[:, :, 8:24]
    whole = ssd.ssd_gated_norm_fwd(y, z, w)
    assert whole.shape == y.shape
    assert torch.equal(whole, ssd.ssd_gated_norm_fwd(y, z.contiguous(), w))
    # the last token of each sequence: rows T*ld apart
    last = ssd.ssd_gated_norm_fwd(y[:, -1].contiguous(), proj[:, -1, 8:24], w)
    assert torch.equal(last, whole[:, -1])
    last3 = ssd.ssd_gated_norm_fwd(y[:, -1:].contiguous(), proj[:, -1:, 8:24], w)
    assert torch.equal(last3[:, 0], whole[:, -1])
    one = ssd.ssd_gated_norm_fwd(y[:1, 0].contiguous(), z[:1, 0].expand(1, 16), w)
    assert torch.equal(one[0], whole[0, 0])
    with pytest.raises(ValueError, match="evenly spaced|overlap"):
        ssd.ssd_gated_norm_fwd(y, z[:, :1].expand(3, 4, 16), w)
    with pytest.raises(ValueError, match="contiguous last dim"):
        ssd.ssd_gated_norm_fwd(y, torch.randn(3, 16, 4, device=dev).transpose(1, 2), w)
    with pytest.raises(ValueError, match="contiguous"):
        ssd.ssd_gated_norm_fwd(torch.randn(3, 16, 4, device=dev).transpose(1, 2), z, w)
    e = torch.empty(0, 16, device=dev)
    out, r = ssd.ssd_add_norm_fwd(e, w)
    assert out.shape == r.shape == (0, 16)
    assert ssd.ssd_gated_norm_fwd(e, e, w).shape == (0, 16)
    g = ssd.ssd_add_norm_bwd(e, e, w, x=e)
    assert float(g["dw"].abs().max()) == 0.0 and float(g["dscale"].abs().max()) == 0.0
    assert float(ssd.ssd_gated_norm_bwd(e, e, e, w, groups=2)["dw"].abs().max()) == 0.0


def test_residual_in_place_and_refused_overlap():
    x, res, w = (torch.randn(*s, device="cuda") for s in ((6, 50), (6, 50), (50,)))
    out, r = ssd.ssd_add_norm_fwd(x, w, residual=res)
    out2, r2 = ssd.ssd_add_norm_fwd(x, w, residual=res, residual_out=res)
    assert r2 is res and torch.equal(r2, r) and torch.equal(out2, out)
    with pytest.raises(ssd.SSDError, match="overlap"):
        ssd.ssd_add_norm_fwd(x, w, out=x)
    with pytest.raises(ssd.SSDError, match="overlap"):
        ssd.ssd_gated_norm_bwd(out, x, res, w, dz=res)


def test_rows_past_32_bit_offsets():
    """2^31 + elements: the last rows equal a call on them alone."""
    D, M = 2048, (1 << 20) + 8
    x = torch.empty(M, D, dtype=torch.bfloat16, device="cuda")
    x[:8].normal_()
    x[-8:].normal_()
    x[8:-8] = 1.0
    w = torch.randn(D, device="cuda")
    out, r = ssd.ssd_add_norm_fwd(x, w, res_dtype=torch.bfloat16)
    tail, tr = ssd.ssd_add_norm_fwd(x[-8:], w, res_dtype=torch.bfloat16)
    assert torch.equal(out[-8:], tail) and torch.equal(r[-8:], tr)
    del out, r
    z = x.view(-1)[: M * D].view(M, D)
    o = ssd.ssd_gated_norm_fwd(x, z, w)
    assert torch.equal(o[-8:], ssd.ssd_gated_norm_fwd(x[-8:].clone(), z[-8:], w))


def test_norms_on_another_stream_and_in_a_graph():
    """The same bits on a side stream given explicitly, and from a captured
    forward and backward replayed with eager work between the replays."""
    torch.manual_seed(0)
    x, res, y = (torch.randn(300, 1024, device="cuda") for _ in range(3))
    z = torch.randn(300, 1500, device="cuda")
    w, sc = torch.randn(1024, device="cuda"), torch.randn(1024, device="cuda")

    def step(stream=None):
        out, r = ssd.ssd_add_norm_fwd(x, w, residual=res, scale=sc, stream=stream)
        g = ssd.ssd_add_norm_bwd(out, r, w, dres=res, scale=sc, x=x, stream=stream)
        o = ssd.ssd_gated_norm_fwd(y, z[:, :1024], w, groups=4, stream=stream)
        h = ssd.ssd_gated_norm_bwd(o, y, z[:, :1024], w, groups=4, stream=stream)
        return [out, r, g["dresidual"], g["dx"], g["dw"], g["dscale"], o, h["dy"], h["dz"], h["dw"]]

    ref = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(3):
        x.normal_()
        z.normal_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b), k


def walked(parts, rows):
    """A number of rows at which every team of a backward pass walks `rows`
    rows and some one more.  parts(M): the rows of its partial-sum table, one
    per workgroup."""
    most = parts(1 << 20)
    teams = next(m for m in range(1, 1 << 10) if parts(m + 1) == 2)  # one row a team fills the first workgroup
    return most * teams * rows + most * teams // 3 + 1


WALKED_ADD = [
    # D, x, residual's, out's type, residual?, scale?
    (64, "bf16", "f32", "bf16", True, True),      # 16-lane teams
    (512, "f32", "f32", "bf16", True, True),      # a wave
    (1000, "bf16", "bf16", "f32", False, True),   # a wave, two vectors a lane
    (1027, "f32", "f32", "f32", True, True),      # from here on a workgroup per row: a barrier in the walk
    (2048, "bf16", "f32", "bf16", True, True),
    (2049, "bf16", "f32", "f32", True, False),
    (4100, "f32", "bf16", "bf16", True, True),
    (8200, "f32", "f32", "f32", True, True),      # the widest, two vectors a lane
    (16383, "bf16", "f32", "bf16", True, True),
]


@pytest.mark.parametrize("D,x,res,out,with_res,with_scale", WALKED_ADD)
def test_add_norm_bwd_walks_rows(D, x, res, out, with_res, with_scale):
    M = walked(lambda m: ssd.ssd_add_norm_bwd_workspace_size(m, D) // (8 * D), 3)
    test_add_norm_bwd(M, D, x, res, out, with_res, with_scale)


WALKED_GATED = [
    # D, groups, ld, col, y, z, out, before
    (128, 1, 136, 4, "bf16", "f32", "bf16", False),
    (500, 1, 1003, 3, "bf16", "bf16", "f32", True),
    (1024, 1, 1024, 0, "f32", "bf16", "bf16", False),
    (2048, 1, 2056, 8, "bf16", "bf16", "bf16", False),
    (2048, 1, 2048, 0, "f32", "f32", "f32", True),
    (4096, 1, 4100, 1, "f32", "bf16", "f32", False),
    (4096, 8, 8512, 0, "bf16", "bf16", "bf16", False),
    (6000, 2, 6001, 1, "bf16", "f32", "bf16", True),
    (8192, 1, 8200, 0, "f32", "bf16", "f32", False),
    (16384, 1, 16384, 0, "f32", "f32", "bf16", False),
]


@pytest.mark.parametrize("D,groups,ld,col,y,z,out,before", WALKED_GATED)
def test_gated_norm_bwd_walks_rows(D, groups, ld, col, y, z, out, before):
    M = walked(lambda m: ssd.ssd_gated_norm_bwd_workspace_size(m, D, groups) // (4 * D), 3)
    test_gated_norm_bwd(M, D, groups, ld, col, y, z, out, before)


@pytest.mark.parametrize("M,D", [(40000, 300), (4096 * 3 + 5, 1027), (4096 * 3 + 5, 2100)])
def test_norms_forward_walk_rows(M, D):
    """More rows than the forward has teams for (4096 workgroups)."""
    test_add_norm_fwd(M, D, "bf16", "f32", "bf16", True, True)
    test_gated_norm_fwd(M, D, 1, D + 3, 1, "bf16", "bf16", "bf16", False)


@pytest.mark.parametrize("D", [1, 7, 300, 1027, 2048, 8200, 16384])
@pytest.mark.parametrize("size,eps", [(1e18, 1e-5), (1e-18, 0.0)])
def test_norms_over_the_range_of_values(D, size, eps):
    """Rows of values up to 1e18, whose squares alone add up past float32, and
    down to 1e-18 with eps 0: within the bars of ordinary rows."""
    print(f"norms over the range D={D} size={size} eps={eps}", flush=True)
    rng = np.random.default_rng(D)
    M = 5
    r = (rng.uniform(0.5, 1.0, (M, D)) * rng.choice([-1.0, 1.0], (M, D)) * size).astype(np.float32)
    w, dout = normal(rng, D, mul=0.2, add=1.0), normal(rng, (M, D))
    up = _gpu.to_dev
    out, kept = ssd.ssd_add_norm_fwd(up(r), up(w), eps=eps)
    ref, _ = layer.add_norm(r, w, eps=eps)
    assert torch.equal(kept, up(r))
    within(out, ref, "f32", C_FWD, 2 * np.abs(ref), "out")
    g = ssd.ssd_add_norm_bwd(up(dout), up(r), up(w), eps=eps)
    gref = layer.add_norm_bwd(dout, r, w, eps=eps)
    rstd = 1 / np.sqrt((wide(r) ** 2).mean(-1, keepdims=True) + eps)
    n, dn = np.abs(wide(r) * rstd), np.abs(wide(dout) * wide(w))
    within(g["dx"], gref["dx"], "f32", C_BWD, rstd * (dn + n * (dn * n).mean(-1, keepdims=True)), "dx")
    within(g["dw"], gref["dw"], "f32", rows_c(M), (np.abs(wide(dout)) * n).sum(0), "dw")
    # the gated norm's u = y silu(z): 1e9 each way, or a small y
    big = size > 1
    y = (r / np.float32(1e9) if big else r).astype(np.float32)
    z = (rng.uniform(1.0, 4.0, (M, D)) * (2.5e8 if big else 1.0)).astype(np.float32)
    ref = layer.gated_norm(y, z, w, 1, eps)
    within(ssd.ssd_gated_norm_fwd(up(y), up(z), up(w), eps=eps), ref, "f32", C_GATE, np.abs(ref), "gated")
    h = ssd.ssd_gated_norm_bwd(up(dout), up(y), up(z), up(w), eps=eps)
    href = layer.gated_norm_bwd(dout, y, z, w, 1, eps)
    Y, Z = np.abs(wide(y)), np.abs(wide(z))
    sig = layer.sigmoid(Z)
    u = Y * Z * sig
    rstd = 1 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    n = u * rstd
    du = rstd * (dn + n * (dn * n).mean(-1, keepdims=True))
    within(h["dy"], href["dy"], "f32", C_BWD, du * Z * sig, "dy")
    within(h["dz"], href["dz"], "f32", C_BWD, du * Y * sig * (1 + Z * (1 - sig)), "dz")
    within(h["dw"], href["dw"], "f32", rows_c(M), (np.abs(wide(dout)) * n).sum(0), "gated dw")


def test_gradients_past_32_bit_offsets():
    """Backward passes over 2^31 + elements: the last rows equal a call on them
    alone, the rows between have no gradient, and the sums over rows are those
    of the first and last rows."""
    D, M, E = 2048, (1 << 20) + 8, 8
    rng = np.random.default_rng(9)
    ends = normal(rng, (2 * E, D), "bf16")
    dends, w = normal(rng, (2 * E, D), "bf16"), normal(rng, D, mul=0.2, add=1.0)
    r = torch.ones(M, D, dtype=torch.bfloat16, device="cuda")
    dout = torch.zeros(M, D, dtype=torch.bfloat16, device="cuda")
    for t, v in ((r, _gpu.to_dev(ends)), (dout, _gpu.to_dev(dends))):
        t[:E], t[-E:] = v[:E], v[E:]
    wd = _gpu.to_dev(w)
    rstd = 1 / np.sqrt((wide(ends) ** 2).mean(-1, keepdims=True) + EPS)
    n, dn = np.abs(wide(ends)) * rstd, np.abs(wide(dends) * wide(w))
    mag = (np.abs(wide(dends)) * n).sum(0)
    g = ssd.ssd_add_norm_bwd(dout, r, wd, x=r)
    tail = ssd.ssd_add_norm_bwd(dout[-E:], r[-E:], wd, x=r[-E:])
    for k in ("dresidual", "dx"):
        assert torch.equal(g[k][-E:], tail[k])
        assert float(g[k][E:-E].abs().max()) == 0.0
    ref = layer.add_norm_bwd(dends, ends, w, x=ends, eps=EPS)
    within(g["dw"], ref["dw"], "f32", rows_c(2 * E), mag, "dw")
    rmag = rstd * (dn + n * (dn * n).mean(-1, keepdims=True))
    within(g["dscale"], ref["dscale"], "f32", rows_c(2 * E), (rmag * np.abs(wide(ends))).sum(0), "dscale")
    del g
    h = ssd.ssd_gated_norm_bwd(dout, r, r, wd)
    tail = ssd.ssd_gated_norm_bwd(dout[-E:], r[-E:], r[-E:], wd)
    for k in ("dy", "dz"):
        assert torch.equal(h[k][-E:], tail[k])
        assert float(h[k][E:-E].abs().max()) == 0.0
    ref = layer.gated_norm_bwd(dends, ends, ends, w, 1, EPS)
    u = np.abs(wide(ends) * layer.silu(wide(ends)))
    n = u / np.sqrt((u * u).mean(-1, keepdims=True) + EPS)
    within(h["dw"], ref["dw"], "f32", rows_c(2 * E), (np.abs(wide(dends)) * n).sum(0), "gated dw")
