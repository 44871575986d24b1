"""rotary_table_fwd, rotary_fwd and qk_norm_rotary_fwd against the plain 64-bit form, and their refusals."""
import math

import numpy as np
import pytest

import attention_ref as ref
import stencil_conv2d_fwd_gb300 as scl

BF16, F32 = scl.SC_BF16, scl.SC_F32
HALF, INTER = scl.SC_ROT_HALF, scl.SC_ROT_INTERLEAVED


def make(torch, dtype, *shape, seed=0, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(*shape, generator=g) * gain
    return (t.bfloat16() if dtype == BF16 else t).cuda()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def table_for(torch, sc, positions, pairs, **kw):
    t = torch.empty(positions, pairs, 2, device="cuda")
    sc.check(sc.rotary_table_fwd(t, positions, pairs, **kw), "rotary_table_fwd")
    return t


def bound(mag, y, D, bf16, norm):
    """The table's rounding, two products and a sum: 4 u of |a| + |b|; the norm's sum of D squares, root and
    products: 6 sqrt(D) + 8 u (rsqrt: 2 ulp); one rounding to bf16."""
    b = ref.U * (4 + (6 * math.sqrt(D) + 8 if norm else 0)) * mag + 1e-30
    return b + ref.UB * np.abs(y) if bf16 else b


def positions_for(torch, axes, tokens, positions, seed):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, positions, (axes, tokens), generator=g, dtype=torch.int32)
    p[:, 0] = positions - 1
    p[:, -1] = 0
    return p.cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("rule,factor,original", [(0, 1.0, 0.0), (1, 4.0, 0.0), (2, 8.0, 0.0), (3, 8.0, 4096.0)])
@pytest.mark.parametrize("pairs,base", [(4, 10000.0), (64, 500000.0), (20, 100.0)])
def test_table(sc, rule, factor, original, pairs, base):
    import torch
    positions = 70001
    t = f64(table_for(torch, sc, positions, pairs, base=base, rule=rule, factor=factor, original=original))
    f, m = ref.frequencies(pairs, base, rule, factor, original)
    angle = np.arange(positions)[:, None] * f[None, :]
    # one rounding to fp32 of values up to m, and the angle's own 64-bit rounding (70001 * 2^-51)
    tol = 2.0 ** -24 * max(1.0, m) * 2 + 70001 * 2.0 ** -49
    assert np.abs(t[..., 0] - m * np.cos(angle)).max() <= tol
    assert np.abs(t[..., 1] - m * np.sin(angle)).max() <= tol


CASES = [  # tokens, heads, D, rot, axes
    (1, 1, 8, 8, 1), (5, 3, 64, 64, 1), (77, 12, 80, 32, 1), (77, 5, 80, 80, 2), (33, 4, 128, 128, 1), (9, 7, 24, 16, 1),
    (130, 1, 32, 32, 2), (17, 9, 96, 24, 1), (40, 2, 256, 256, 1), (40, 6, 256, 48, 2), (1000, 8, 64, 56, 1),
    (3, 33, 40, 40, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mode", [HALF, INTER])
@pytest.mark.parametrize("case", CASES)
def test_rotary(sc, case, mode, dtype):
    import torch
    tokens, heads, D, rot, axes = case
    positions = 300
    x = make(torch, dtype, tokens, heads, D, seed=1, gain=1.5)
    pos = positions_for(torch, axes, tokens, positions, 2)
    t = table_for(torch, sc, positions, rot // (2 * axes))
    y = torch.full_like(x, float("nan"))
    sc.check(sc.rotary_fwd(x, y, t, pos, tokens, heads, D, rot, positions, mode, axes, dtype=dtype))
    f, m = ref.frequencies(rot // (2 * axes))
    want, mag = ref.rotate(f64(x), pos.cpu().numpy(), rot, mode, axes, f)
    err = np.abs(f64(y) - want)
    assert (err <= bound(mag, want, D, dtype == BF16, False)).all()
    assert torch.equal(y[..., rot:], x[..., rot:])
    # in place, and back
    z = x.clone()
    sc.check(sc.rotary_fwd(z, z, t, pos, tokens, heads, D, rot, positions, mode, axes, dtype=dtype))
    assert torch.equal(z, y)
    sc.check(sc.rotary_fwd(z, z, t, pos, tokens, heads, D, rot, positions, mode, axes, inverse=True, dtype=dtype))
    back, mag = ref.rotate(f64(y), pos.cpu().numpy(), rot, mode, axes, f, inverse=True)
    assert (np.abs(f64(z) - back) <= bound(mag, back, D, dtype == BF16, False)).all()
    sc.check(sc.sc_last_device_status())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mode", [HALF, INTER])
@pytest.mark.parametrize("case", CASES + [(20, 4, 64, 0, 1), (6, 2, 120, 0, 2)])
def test_norm_rotary(sc, case, mode, dtype):
    """Queries and keys of different counts; weights or none; a row of zeros."""
    import torch
    tokens, heads, D, rot, axes = case
    positions, eps = 300, 1e-5
    q, k = make(torch, dtype, tokens, heads, D, seed=3, gain=3.0), make(torch, dtype, 2 * tokens + 1, 2, D, seed=4)
    k[0] = 0
    wq = 1 + 0.3 * torch.randn(D, generator=torch.Generator().manual_seed(5)).cuda()
    pq, pk = (positions_for(torch, axes, x.shape[0], positions, 6) for x in (q, k))
    t = table_for(torch, sc, positions, rot // (2 * axes)) if rot else None
    yq, yk = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    sc.check(sc.qk_norm_rotary_fwd((q, yq, wq, pq, tokens, heads), (k, yk, None, pk, 2 * tokens + 1, 2), t, D, rot,
                                   positions, eps, mode, axes, dtype=dtype))
    f, m = ref.frequencies(rot // (2 * axes)) if rot else (np.zeros(0), 1.0)
    eps32 = float(np.float32(eps))
    for x, y, w, p in ((q, yq, f64(wq), pq), (k, yk, None, pk)):
        want, mag = ref.rotate(ref.rms_norm(f64(x), w, eps32), p.cpu().numpy(), rot, mode, axes, f)
        assert (np.abs(f64(y) - want) <= bound(mag, want, D, dtype == BF16, True)).all()
    # either alone, and in place: the same bits
    z = q.clone()
    sc.check(sc.qk_norm_rotary_fwd((z, z, wq, pq, tokens, heads), None, t, D, rot, positions, eps, mode, axes,
                                   dtype=dtype))
    assert torch.equal(z, yq)
    z = k.clone()
    sc.check(sc.qk_norm_rotary_fwd(None, (z, z, None, pk, 2 * tokens + 1, 2), t, D, rot, positions, eps, mode, axes,
                                   dtype=dtype))
    assert torch.equal(z, yk)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_fused_projection_in_place(sc, dtype):
    """Queries, keys and values in one row: the first two changed in place, the values left alone; and heads before tokens."""
    import torch
    tokens, Hq, Hkv, D, positions = 50, 6, 2, 64, 64
    row = make(torch, dtype, tokens, (Hq + 2 * Hkv) * D, seed=7)
    before = row.clone()
    pos = positions_for(torch, 1, tokens, positions, 8)
    t = table_for(torch, sc, positions, D // 2)
    q, k = row[:, :Hq * D], row[:, Hq * D:(Hq + Hkv) * D]
    st = (row.stride(0), D, row.stride(0), D)
    sc.check(sc.qk_norm_rotary_fwd((q, q, None, pos, tokens, Hq, *st), (k, k, None, pos, tokens, Hkv, *st), t, D, D,
                                   positions, 1e-6, dtype=dtype))
    f, m = ref.frequencies(D // 2)
    n = Hq + Hkv
    want, mag = ref.rotate(ref.rms_norm(f64(before)[:, :n * D].reshape(tokens, n, D), None, 1e-6), pos.cpu().numpy(), D,
                           HALF, 1, f)
    err = np.abs(f64(row)[:, :n * D].reshape(tokens, n, D) - want)
    assert (err <= bound(mag, want, D, dtype == BF16, True)).all()
    assert torch.equal(row[:, n * D:], before[:, n * D:])
    x = make(torch, dtype, Hq, tokens, D, seed=9)   # heads before tokens
    y = torch.empty_like(x)
    sc.check(sc.rotary_fwd(x, y, t, pos, tokens, Hq, D, D, positions, dtype=dtype, x_strides=(D, tokens * D),
                           y_strides=(D, tokens * D)))
    want, mag = ref.rotate(f64(x).transpose(1, 0, 2), pos.cpu().numpy(), D, HALF, 1, f)
    assert (np.abs(f64(y).transpose(1, 0, 2) - want) <= bound(mag, want, D, dtype == BF16, False)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,heads,shared", [(40, 6, "both"), (1, 5, "both"), (7, 1, "both"), (1, 1, "both"),
                                                 (40, 6, "tokens"), (40, 6, "heads")])
def test_rows_shared_by_stride_zero(sc, tokens, heads, shared, dtype):
    """One row for all tokens and heads (both strides 0), one for all tokens, one for all heads of a token; memory
    right behind the shared rows is someone else's."""
    import torch
    D, positions = 64, 50
    rows = {"both": (1, 1), "tokens": (1, heads), "heads": (tokens, 1)}[shared]
    store = torch.full((rows[0] * rows[1] + tokens * heads, D), float("nan"),
                       dtype=torch.bfloat16 if dtype == BF16 else torch.float32, device="cuda")
    base = store[:rows[0] * rows[1]].view(*rows, D)
    base.copy_(make(torch, dtype, *rows, D, seed=17))
    x = base.expand(tokens, heads, D)
    xs = (0 if rows[0] == 1 else heads * D if shared == "tokens" else D, D if shared == "tokens" else 0)
    pos = positions_for(torch, 1, tokens, positions, 18)
    t = table_for(torch, sc, positions, D // 2)
    y = store[rows[0] * rows[1]:].view(tokens, heads, D)     # next to x: overlaps the one only if the other is packed
    sc.check(sc.rotary_fwd(base, y, t, pos, tokens, heads, D, D, positions, dtype=dtype, x_strides=xs))
    f, m = ref.frequencies(D // 2)
    want, mag = ref.rotate(f64(x), pos.cpu().numpy(), D, HALF, 1, f)
    assert (np.abs(f64(y) - want) <= bound(mag, want, D, dtype == BF16, False)).all()


@pytest.mark.gpu
def test_long_context_positions(sc):
    """The last positions of a long scaled context: the angle is not lost to 32 bits."""
    import torch
    positions, D, heads = 1 << 20, 64, 2
    t = table_for(torch, sc, positions, D // 2, base=500000.0, rule=scl.SC_ROT_SCALE_BANDS, factor=16.0, original=65536.0)
    pos = torch.arange(positions - 40, positions, dtype=torch.int32).cuda()
    x = make(torch, F32, 40, heads, D, seed=10)
    y = torch.empty_like(x)
    sc.check(sc.rotary_fwd(x, y, t, pos, 40, heads, D, D, positions))
    f, m = ref.frequencies(D // 2, 500000.0, 3, 16.0, 65536.0)
    want, mag = ref.rotate(f64(x), pos.cpu().numpy()[None].astype(np.float64), D, HALF, 1, f, m)
    assert (np.abs(f64(y) - want) <= bound(mag, want, D, False, False)).all()


@pytest.mark.gpu
def test_adjoint_of_the_rotation(sc):
    """<R x, g> = <x, R' g>: inverse is the gradient's map; and R's differences along a direction are R of it."""
    import torch
    tokens, heads, D, positions = 30, 3, 48, 50
    t = table_for(torch, sc, positions, D // 2)
    pos = positions_for(torch, 1, tokens, positions, 11)
    x, g = make(torch, F32, tokens, heads, D, seed=12), make(torch, F32, tokens, heads, D, seed=13)
    rx, rg, rxg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    sc.check(sc.rotary_fwd(x, rx, t, pos, tokens, heads, D, D, positions))
    sc.check(sc.rotary_fwd(g, rg, t, pos, tokens, heads, D, D, positions, inverse=True))
    sc.check(sc.rotary_fwd(x + g, rxg, t, pos, tokens, heads, D, D, positions))
    lhs, rhs = (f64(rx) * f64(g)).sum(), (f64(x) * f64(rg)).sum()
    size = (np.abs(f64(rx) * f64(g))).sum()
    assert abs(lhs - rhs) <= 16 * ref.U * size
    rd = torch.empty_like(x)
    sc.check(sc.rotary_fwd(g, rd, t, pos, tokens, heads, D, D, positions))
    assert np.abs(f64(rxg) - f64(rx) - f64(rd)).max() <= 16 * ref.U * (f64(x.abs().max()) + f64(g.abs().max())) * 2


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [-1, 50, 2 ** 31 - 1, -2 ** 31])
def test_position_outside_the_table(sc, bad):
    """Nothing is read for it: its elements are NaN, the device status says so, the other tokens are right."""
    import torch
    tokens, heads, D, rot, positions = 6, 2, 64, 32, 50
    t = table_for(torch, sc, positions, rot // 2)
    pos = torch.tensor([0, 1, bad, 3, 49, 5], dtype=torch.int32).cuda()
    x = make(torch, F32, tokens, heads, D, seed=14)
    y = torch.zeros_like(x)
    sc.check(sc.sc_last_device_status())
    sc.check(sc.rotary_fwd(x, y, t, pos, tokens, heads, D, rot, positions))
    assert sc.sc_last_device_status() == scl.SC_ERR_RANGE
    assert sc.sc_last_device_status() == scl.SC_OK
    assert torch.isnan(y[2, :, :rot]).all() and torch.equal(y[2, :, rot:], x[2, :, rot:])
    keep = [0, 1, 3, 4, 5]
    f, m = ref.frequencies(rot // 2)
    want, mag = ref.rotate(f64(x)[keep], pos.cpu().numpy()[None, keep], rot, HALF, 1, f)
    assert (np.abs(f64(y)[keep] - want) <= bound(mag, want, D, False, False)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mode", [HALF, INTER])
@pytest.mark.parametrize("bad_axes", [(0,), (1,), (0, 1)])
@pytest.mark.parametrize("norm", [False, True])
def test_position_outside_the_table_on_one_axis(sc, norm, bad_axes, mode, dtype):
    """Two axes: NaN where the bad position turns, the other axis's pairs and the rest of the head are right."""
    import torch
    tokens, heads, D, rot, positions = 9, 5, 80, 64, 40
    t = table_for(torch, sc, positions, rot // 4)
    pos = positions_for(torch, 2, tokens, positions, 19)
    for a in bad_axes:
        pos[a, 4] = positions
    x = make(torch, dtype, tokens, heads, D, seed=20)
    y = torch.zeros_like(x)
    sc.check(sc.sc_last_device_status())
    if norm:
        sc.check(sc.qk_norm_rotary_fwd((x, y, None, pos, tokens, heads), None, t, D, rot, positions, 1e-6, mode, 2, dtype))
    else:
        sc.check(sc.rotary_fwd(x, y, t, pos, tokens, heads, D, rot, positions, mode, 2, dtype=dtype))
    assert sc.sc_last_device_status() == scl.SC_ERR_RANGE
    pair = np.arange(rot // 2)
    a, b = (pair, pair + rot // 2) if mode == HALF else (2 * pair, 2 * pair + 1)
    bad = np.zeros((tokens, heads, D), bool)
    for axis in bad_axes:
        mine = pair // (rot // 4) == axis
        bad[4][:, np.concatenate([a[mine], b[mine]])] = True
    got = f64(y)
    assert np.isnan(got[bad]).all()
    f, m = ref.frequencies(rot // 4)
    src = ref.rms_norm(f64(x), None, 1e-6) if norm else f64(x)
    want, mag = ref.rotate(src, pos.cpu().numpy() % positions, rot, mode, 2, f)
    ok = np.abs(got - want) <= bound(mag, want, D, dtype == BF16, norm)
    assert (ok | bad).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_offsets_beyond_32_bits(sc, dtype):
    import torch
    tokens, heads, D, positions = (1 << 31) // (16 * 128) + 77, 16, 128, 64
    x = torch.zeros(tokens, heads, D, dtype=torch.bfloat16 if dtype == BF16 else torch.float32, device="cuda")
    x[-5:] = make(torch, dtype, 5, heads, D, seed=15)
    last = x[-5:].clone()
    pos = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    pos[-5:] = torch.tensor([63, 1, 2, 3, 40], dtype=torch.int32).cuda()
    t = table_for(torch, sc, positions, D // 2)
    sc.check(sc.rotary_fwd(x, x, t, pos, tokens, heads, D, D, positions, dtype=dtype))
    f, m = ref.frequencies(D // 2)
    want, mag = ref.rotate(f64(last), pos[-5:].cpu().numpy()[None], D, HALF, 1, f)
    assert (np.abs(f64(x[-5:]) - want) <= bound(mag, want, D, dtype == BF16, False)).all()


A, B, T, P, W = 1 << 30, 1 << 32, 1 << 34, 1 << 36, 1 << 38   # fake, aligned, far apart: never dereferenced


@pytest.mark.parametrize("change,expect", [
    (dict(x=None), scl.SC_ERR_NULL),
    (dict(y=None), scl.SC_ERR_NULL),
    (dict(table=None), scl.SC_ERR_NULL),
    (dict(pos=None), scl.SC_ERR_NULL),
    (dict(tokens=0), scl.SC_ERR_SHAPE),
    (dict(heads=-1), scl.SC_ERR_SHAPE),
    (dict(positions=0), scl.SC_ERR_SHAPE),
    (dict(rot=-8), scl.SC_ERR_SHAPE),
    (dict(D=0), scl.SC_ERR_SHAPE),
    (dict(D=20), scl.SC_ERR_UNSUPPORTED),
    (dict(D=264), scl.SC_ERR_UNSUPPORTED),
    (dict(rot=72), scl.SC_ERR_UNSUPPORTED),
    (dict(rot=12), scl.SC_ERR_UNSUPPORTED),
    (dict(rot=24, axes=2), scl.SC_ERR_UNSUPPORTED),
    (dict(axes=3), scl.SC_ERR_UNSUPPORTED),
    (dict(mode=2), scl.SC_ERR_UNSUPPORTED),
    (dict(dtype=2), scl.SC_ERR_UNSUPPORTED),
    (dict(x=A + 4), scl.SC_ERR_ALIGN),
    (dict(table=T + 8), scl.SC_ERR_ALIGN),
    (dict(pos=P + 2), scl.SC_ERR_ALIGN),
    (dict(xs=(258, 64)), scl.SC_ERR_ALIGN),
    (dict(ys=(256, -64)), scl.SC_ERR_SHAPE),
    (dict(ys=(256, 32)), scl.SC_ERR_ALIAS),
    (dict(ys=(0, 0)), scl.SC_ERR_ALIAS),
    (dict(ys=(256, 0)), scl.SC_ERR_ALIAS),
    (dict(ys=(0, 64)), scl.SC_ERR_ALIAS),
    (dict(y=A, xs=(0, 0), ys=(0, 0)), scl.SC_ERR_ALIAS),
    (dict(y=A, xs=(0, 0)), scl.SC_ERR_ALIAS),
    (dict(y=A + 64), scl.SC_ERR_ALIAS),
    (dict(y=A, ys=(512, 64)), scl.SC_ERR_ALIAS),
    (dict(table=B + 64), scl.SC_ERR_ALIAS),
    (dict(pos=B + 64), scl.SC_ERR_ALIAS),
])
def test_rotary_refusals(change, expect):
    a = dict(x=A, y=B, table=T, pos=P, tokens=10, heads=4, D=64, rot=32, positions=16, mode=HALF, axes=1, dtype=F32,
             xs=None, ys=None)
    a.update(change)
    rc = scl.rotary_fwd(a["x"], a["y"], a["table"], a["pos"], a["tokens"], a["heads"], a["D"], a["rot"], a["positions"],
                        a["mode"], a["axes"], dtype=a["dtype"], x_strides=a["xs"], y_strides=a["ys"], stream=0)
    assert rc == expect, scl.sc_status_string(rc)


@pytest.mark.parametrize("change,expect", [
    (dict(q=None, k=None), scl.SC_ERR_NULL),
    (dict(eps=-1.0), scl.SC_ERR_UNSUPPORTED),
    (dict(eps=math.nan), scl.SC_ERR_UNSUPPORTED),
    (dict(q=(A, B, W + 4, P, 4, 4)), scl.SC_ERR_ALIGN),
    (dict(q=(A, B, B, P, 4, 4)), scl.SC_ERR_ALIAS),
    (dict(k=(A + (1 << 20), B, None, P, 4, 4)), scl.SC_ERR_ALIAS),          # both write the same rows
    (dict(k=(B, B, None, P, 4, 4)), scl.SC_ERR_ALIAS),
    (dict(k=(A + (1 << 20), A, None, P, 4, 4)), scl.SC_ERR_ALIAS),          # k's output over q's input
    (dict(k=(A + (1 << 20), B + (1 << 20), None, None, 4, 4)), scl.SC_ERR_NULL),
    (dict(k=(A + (1 << 20), B + (1 << 20), B, P, 4, 4)), scl.SC_ERR_ALIAS),  # k's weight inside q's output
])
def test_norm_rotary_refusals(change, expect):
    a = dict(q=(A, B, None, P, 4, 4), k=None, eps=1e-6)
    a.update(change)
    rc = scl.qk_norm_rotary_fwd(a["q"], a["k"], T, 64, 32, 16, a["eps"], dtype=F32, stream=0)
    assert rc == expect, scl.sc_status_string(rc)


@pytest.mark.parametrize("change,expect", [
    (dict(table=None), scl.SC_ERR_NULL),
    (dict(table=T + 4), scl.SC_ERR_ALIGN),
    (dict(positions=0), scl.SC_ERR_SHAPE),
    (dict(pairs=0), scl.SC_ERR_SHAPE),
    (dict(base=1.0), scl.SC_ERR_UNSUPPORTED),
    (dict(base=math.inf), scl.SC_ERR_UNSUPPORTED),
    (dict(rule=4), scl.SC_ERR_UNSUPPORTED),
    (dict(rule=1, factor=0.5), scl.SC_ERR_UNSUPPORTED),
    (dict(rule=2, factor=math.nan), scl.SC_ERR_UNSUPPORTED),
    (dict(rule=2, factor=2.0, pairs=1), scl.SC_ERR_UNSUPPORTED),
    (dict(rule=3, factor=2.0, original=0.0), scl.SC_ERR_UNSUPPORTED),
])
def test_table_refusals(change, expect):
    a = dict(table=T, positions=16, pairs=8, base=10000.0, rule=0, factor=1.0, original=0.0)
    a.update(change)
    rc = scl.rotary_table_fwd(a["table"], a["positions"], a["pairs"], a["base"], a["rule"], a["factor"], a["original"],
                              stream=0)
    assert rc == expect, scl.sc_status_string(rc)
