"""GPU parity of the fused single-token step against the float64 oracle and
against the separate convolution and decode steps.

Roundings (c, in units of 2^-24): v is 5 products and sums, SiLU at |v| < 12
adds 24; the decay's exponent is A delta with |A delta| <= 1.6 here (A in
[-16, -1], delta <= 0.1), so exp and delta's own error (softplus: 8 units of
delta) reach the state by 1.6 * (8 + 2) + 3 < 20 units; the update adds 3:
C_H = 60.  y sums N terms (8 in sequence, 6 over lanes) on top: C_Y = 90."""
import numpy as np
import pytest
import torch

import selective_state_space_09_amd as ssd
from oracle import layer
from _layer import TYPES, normal, rows_in, wide, within
import _gpu

pytestmark = pytest.mark.gpu
C_H, C_Y = 60, 90
LO, HI = 1e-3, 1e-1

CASES = [
    # Bsz, nslots, H, P, G, N, rows' type, y's, slots, act, optional inputs
    (1, 1, 64, 64, 1, 128, "bf16", "f32", None, 1, True),
    (3, 5, 4, 16, 2, 16, "f32", "f32", None, 0, False),
    (6, 9, 8, 33, 8, 32, "f32", "bf16", "map", 1, True),      # H == G, odd P
    (5, 4, 6, 1, 3, 64, "bf16", "f32", "map", 1, True),       # P = 1, more rows than slots
    (37, 64, 24, 48, 8, 64, "f32", "f32", "map", 1, True),
    (4, 6, 3, 130, 1, 256, "bf16", "bf16", "map", 1, True),   # several passes over the rows
    (2, 3, 2, 1024, 1, 16, "f32", "f32", "map", 1, True),     # the largest P
    (300, 310, 4, 8, 2, 32, "bf16", "f32", "map", 1, True),
]


def case(Bsz, nslots, H, P, G, N, t, slots, opt, seed=0):
    rng = np.random.default_rng(Bsz + H * P + N + seed)
    Ch = H * P + 2 * G * N
    a = dict(conv_state=normal(rng, (nslots, 3, Ch)), h=normal(rng, (nslots, H, P, N)), xbc=normal(rng, (Bsz, Ch), t),
             dt=normal(rng, (Bsz, H), t), w=normal(rng, (Ch, 4), mul=0.4),
             A=-np.exp(rng.uniform(0, np.log(16.0), H)).astype(np.float32))
    a.update(bias=normal(rng, Ch, mul=0.4) if opt else None, D=normal(rng, H) if opt else None,
             dt_bias=normal(rng, H, mul=2.0, add=-3.0) if opt else None)
    if slots:
        m = rng.permutation(nslots + Bsz)[:Bsz]
        m = np.where(m < nslots, m, -1 - (m % 3)).astype(np.int32)  # some rows are padding
        if Bsz > 3:
            m[Bsz - 1] = m[0]      # a slot named twice
            m[1] = nslots + 5      # past the pool
            m[2] = -2 ** 31
        a["slots"] = m
    else:
        a["slots"] = None
    return a


def run(a, d, G, **k):
    arrivals = torch.zeros(a["h"].shape[0], G, dtype=torch.int32, device="cuda")
    y = ssd.ssd_mixer_step(d["conv_state"], d["h"], arrivals, d["xbc"], d["dt"], d["w"], d["A"], bias=d["bias"], D=d["D"],
                           dt_bias=d["dt_bias"], dt_min=LO, dt_max=HI, slots=d["slots"], **k)
    torch.cuda.synchronize()
    assert int(arrivals.abs().max()) == 0  # left as they were found
    return y


@pytest.mark.parametrize("Bsz,nslots,H,P,G,N,t,yt,slots,act,opt", CASES)
def test_mixer_step(Bsz, nslots, H, P, G, N, t, yt, slots, act, opt):
    print(f"mixer_step Bsz={Bsz} nslots={nslots} H={H} P={P} G={G} N={N} {t} {yt} {slots} act={act}", flush=True)
    a = case(Bsz, nslots, H, P, G, N, t, slots, opt)
    keys = ("conv_state", "h", "xbc", "dt", "w", "A")
    ref = layer.mixer_step(*[a[k] for k in keys], G, a["bias"], a["D"], a["dt_bias"], LO, HI, a["slots"], act)
    Ch = H * P + 2 * G * N
    d = {k: _gpu.to_dev(v) for k, v in a.items()}
    # xbc and dt in place in rows of odd length, at odd columns
    d["xbc"], _ = rows_in(a["xbc"], Ch + 7, 3, fill=float("nan"))
    d["dt"], _ = rows_in(a["dt"], H + 5, 1, fill=float("nan"))
    y = run(a, d, G, act=act, y_dtype=TYPES[yt])
    np.testing.assert_array_equal(_gpu.to_host64(d["conv_state"]), ref[1])  # raw inputs: bit for bit
    # magnitudes from the same step on absolute values, decay 1, no clamp on the small side
    ab = {k: None if a[k] is None else np.abs(wide(a[k])) for k in keys + ("bias", "D")}
    win = lambda b, s: np.concatenate([ab["conv_state"][s], ab["xbc"][b][None]])  # noqa: E731
    seen = set()
    mag_h, mag_y = ab["h"].copy(), np.zeros((Bsz, H, P))
    for b in range(Bsz):
        s = b if a["slots"] is None else int(a["slots"][b])
        if not 0 <= s < nslots or s in seen:
            continue
        seen.add(s)
        v = 1.0 + (win(b, s) * ab["w"].T).sum(0) + (0.0 if not opt else ab["bias"])
        x, Bm, Cm = v[:H * P].reshape(H, P), v[H * P:H * P + G * N].reshape(G, N), v[H * P + G * N:].reshape(G, N)
        Bh, Chh = np.repeat(Bm, H // G, 0), np.repeat(Cm, H // G, 0)
        mag_h[s] += HI * x[:, :, None] * Bh[:, None, :]
        mag_y[b] = (mag_h[s] * Chh[:, None, :]).sum(-1) + (0.0 if not opt else ab["D"][:, None] * x)
    within(d["h"], ref[2], "f32", C_H, mag_h, "h")
    within(y, ref[0], yt, C_Y, mag_y, "y")
    untouched = [s for s in range(nslots) if s not in seen]
    np.testing.assert_array_equal(_gpu.to_host64(d["h"])[untouched], a["h"].astype(np.float64)[untouched])


def test_many_steps_equal_the_separate_kernels():
    """40 steps of a batch on its own slots against ssd_conv1d_step and
    ssd_step_decode: conv rows bit for bit, states and outputs within 40 steps'
    roundings; both chains see the same rows."""
    torch.manual_seed(3)
    B, H, P, G, N = 5, 8, 16, 2, 32
    HP, GN = H * P, G * N
    Ch = HP + 2 * GN
    conv, h = torch.randn(B, 3, Ch, device="cuda"), torch.randn(B, H, P, N, device="cuda")
    conv2, h2 = conv.clone(), h.clone()
    arr = torch.zeros(B, G, dtype=torch.int32, device="cuda")
    w, bias = torch.randn(Ch, 4, device="cuda") * 0.4, torch.randn(Ch, device="cuda") * 0.4
    A, D = -torch.rand(H, device="cuda") * 4 - 1, torch.randn(H, device="cuda")
    for k in range(40):
        row = torch.randn(B, Ch + H, device="cuda")
        y = ssd.ssd_mixer_step(conv, h, arr, row[:, :Ch], row[:, Ch:], w, A, bias=bias, D=D, dt_max=0.1)
        x, Bm, Cm = ssd.ssd_conv1d_step(conv2, row[:, :Ch].contiguous(), w, HP, GN, bias=bias)
        y2 = ssd.ssd_step_decode(h2, x.view(B, H, P), row[:, Ch:].contiguous(), A, Bm.view(B, G, N), Cm.view(B, G, N),
                                 D=D, dt_max=0.1)
        assert torch.equal(conv, conv2), k
        top = float(y2.abs().max()) + float(h2.abs().max())
        assert float((y - y2).abs().max()) <= 1e-5 * top and float((h - h2).abs().max()) <= 1e-5 * top, k


def test_slots_past_32_bit_offsets():
    """A pool of 8.6 GB: the slot at its end gives what the same states give in
    a pool of one."""
    H, P, G, N, nslots = 64, 64, 1, 128, 4104
    Ch = H * P + 2 * G * N
    pool = torch.empty(nslots, H, P, N, device="cuda")
    conv = torch.empty(nslots, 3, Ch, device="cuda")
    arr = torch.zeros(nslots, G, dtype=torch.int32, device="cuda")
    pool[-1].normal_()
    conv[-1].normal_()
    pool[0].fill_(3.0)
    h1, c1 = pool[-1:].clone(), conv[-1:].clone()
    row = torch.randn(1, Ch + H, device="cuda")
    w, A = torch.randn(Ch, 4, device="cuda"), -torch.rand(H, device="cuda")
    slots = torch.tensor([nslots - 1], dtype=torch.int32, device="cuda")
    y = ssd.ssd_mixer_step(conv, pool, arr, row[:, :Ch], row[:, Ch:], w, A, slots=slots)
    y1 = ssd.ssd_mixer_step(c1, h1, arr[:1], row[:, :Ch], row[:, Ch:], w, A)
    assert torch.equal(y, y1) and torch.equal(pool[-1:], h1) and torch.equal(conv[-1:], c1)
    assert bool((pool[0] == 3.0).all())


def test_two_graphs_and_two_streams_on_one_pool():
    """Captured steps of two disjoint batches of one pool, replayed on two
    streams at once, against the same steps run eagerly one after the other."""
    torch.manual_seed(4)
    H, P, G, N, nslots = 16, 32, 1, 64, 12
    Ch = H * P + 2 * G * N
    pool, conv = torch.randn(nslots, H, P, N, device="cuda"), torch.randn(nslots, 3, Ch, device="cuda")
    arr = torch.zeros(nslots, G, dtype=torch.int32, device="cuda")
    w, A = torch.randn(Ch, 4, device="cuda") * 0.4, -torch.rand(H, device="cuda") - 0.5
    slots = [torch.tensor(s, dtype=torch.int32, device="cuda") for s in ([1, 3, 5, -1], [0, 2, 11, 7])]
    rows = [torch.randn(4, Ch + H, device="cuda") for _ in range(2)]
    start = pool.clone(), conv.clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, ys = [], []
    step = lambda k, p, c, ar: ssd.ssd_mixer_step(c, p, ar, rows[k][:, :Ch], rows[k][:, Ch:], w, A, slots=slots[k], dt_max=0.1)  # noqa: E731
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ys.append(step(k, pool, conv, arr))
        graphs.append(g)
    pool.copy_(start[0])
    conv.copy_(start[1])
    p2, c2, a2 = start[0].clone(), start[1].clone(), torch.zeros_like(arr)
    torch.cuda.synchronize()
    for it in range(4):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(step(k, p2, c2, a2), ys[k]), (it, k)
        assert torch.equal(pool, p2) and torch.equal(conv, c2)
        for r in rows:
            r.normal_()
        torch.cuda.synchronize()
    assert int(arr.abs().max()) == 0


def test_empty_batch_and_all_padding():
    H, P, G, N = 2, 4, 1, 16
    Ch = H * P + 2 * G * N
    h, conv = torch.randn(2, H, P, N, device="cuda"), torch.randn(2, 3, Ch, device="cuda")
    h0, c0 = h.clone(), conv.clone()
    arr = torch.zeros(2, G, dtype=torch.int32, device="cuda")
    w, A = torch.randn(Ch, 4, device="cuda"), -torch.ones(H, device="cuda")
    y = ssd.ssd_mixer_step(conv, h, arr, torch.empty(0, Ch, device="cuda"), torch.empty(0, H, device="cuda"), w, A)
    assert y.shape == (0, H, P)
    y = ssd.ssd_mixer_step(conv, h, arr, torch.randn(3, Ch, device="cuda"), torch.randn(3, H, device="cuda"), w, A,
                           slots=torch.full((3,), -1, dtype=torch.int32, device="cuda"))
    assert float(y.abs().max()) == 0.0
    assert torch.equal(h, h0) and torch.equal(conv, c0)


@pytest.mark.parametrize("B", [257, 258, 260, 511, 2304, 2305, 5003])
def test_repeated_slots_of_long_batches(B):
    """A row whose slot an earlier row has is padding wherever the two stand:
    the same bits as with the later rows' slots set outside the pool."""
    print(f"mixer_step repeated slots B={B}", flush=True)
    H, P, G, N, ns = 2, 4, 1, 16, B
    Ch = H * P + 2 * G * N
    rng = np.random.default_rng(B)
    m = rng.permutation(B)
    for i, j in ((0, B - 1), (3, 256), (255, B - 2), (252, B - 3), (B - 5, B - 4), (7, 128)):  # pairs at the edges
        m[j] = m[i]
    some = rng.random(B) < 0.1
    some[[0, 3, 7, 252, 255, B - 5]] = False
    m = np.where(some, rng.integers(-2, ns + 2, B), m)  # others anywhere, and outside
    once = m.copy()
    seen = set()
    for b, s in enumerate(m):
        if s in seen:
            once[b] = -1
        seen.add(s)
    assert (once != m).sum() >= 4 and (once >= 0).sum() > B // 2
    torch.manual_seed(B)
    dev = dict(device="cuda")
    conv, h = torch.randn(ns, 3, Ch, **dev), torch.randn(ns, H, P, N, **dev)
    row, w, A = torch.randn(B, Ch + H, **dev), torch.randn(Ch, 4, **dev) * 0.4, -torch.rand(H, **dev) - 1
    got = []
    for s in (m, once):
        c, hh, arr = conv.clone(), h.clone(), torch.zeros(ns, G, dtype=torch.int32, **dev)
        y = ssd.ssd_mixer_step(c, hh, arr, row[:, :Ch], row[:, Ch:], w, A, dt_max=0.1,
                               slots=torch.from_numpy(s.astype(np.int32)).cuda())
        assert int(arr.abs().max()) == 0
        got.append((y, c, hh))
    for x, x2 in zip(*got):
        assert torch.equal(x, x2)
    off = torch.from_numpy((once < 0) | (once >= ns)).cuda()
    assert float(got[0][0][off].abs().max()) == 0.0 and float(got[0][0][~off].abs().min(-1)[0].max()) > 0.0
