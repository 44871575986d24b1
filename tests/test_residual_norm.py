"""residual_norm_fwd against the plain 64-bit form, and its refusals (bounds: layer_ref.py)."""
import math

import pytest

import layer_ref as ref
import stencil_conv2d_fwd_gb300 as scl

BF16, F32 = scl.SC_BF16, scl.SC_F32
NONE, RMS, LAYER = scl.SC_NORM_NONE, scl.SC_NORM_RMS, scl.SC_NORM_LAYER
EPS = 1e-6


def tensors(torch, dtype, rows, C, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = torch.bfloat16 if dtype == BF16 else torch.float32
    x, r = (torch.randn(rows, C, generator=g) * k + o for k, o in ((1.0, 0.5), (2.0, -0.3)))
    w = [1 + 0.3 * torch.randn(C, generator=g) for _ in range(2)] + [0.2 * torch.randn(C, generator=g) for _ in range(2)]
    return x.to(t).cuda(), r.to(t).cuda(), [v.cuda() for v in w]


def reference(x, r, post, pre, gate_of_row, scale, C, bf16):
    """sum and y, and their bounds: norms of C elements, each norm passing its input's error on by no
    more than the norm of the error's own size (the mean's and the variance's change with it: three times)."""
    fp = ref.U * (6 * math.sqrt(C) + 24)
    t, mag = ref.normed(x.double(), *post)
    err = fp * mag
    if gate_of_row is not None:
        t, mag, err = t * gate_of_row.double(), mag * gate_of_row.double().abs(), err * gate_of_row.double().abs()
    s, smag = t, mag
    if r is not None:
        s, smag = t + scale * r.double(), mag + abs(scale) * r.double().abs()
    serr = err + fp * smag
    y, ymag = ref.normed(s, *pre)
    if pre[0] == NONE:
        yerr = serr
    else:
        v = s - s.mean(dim=-1, keepdim=True) if pre[0] == LAYER else s
        rr = 1 / (v.pow(2).mean(dim=-1, keepdim=True) + pre[3]).sqrt()
        g = 1.0 if pre[1] is None else pre[1].double().abs()
        rms = serr.pow(2).mean(dim=-1, keepdim=True).sqrt()
        unit = (v * rr).abs() * g
        yerr = (serr + 2 * rms) * rr * g + unit * rms * rr + fp * ymag
    half = ref.UB if bf16 else ref.U
    return (s, serr + half * s.abs() + 1e-37), (y, yerr + half * y.abs() + 1e-37)


def check(torch, got, want, what):
    w, bound = want
    err = (got.double() - w).abs()
    assert torch.isfinite(got.float()).all(), what
    worst = (err / bound).max().item()
    assert worst <= 1, f"{what}: {worst:.2f} of its bound"


# C: one chunk to the widest, odd numbers of chunks, around a warp's and a thread's share
WIDTHS = [8, 16, 72, 256, 264, 504, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 5000, 8192, 8200, 16376, 16384]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [1, 7, 700])
@pytest.mark.parametrize("C", WIDTHS)
def test_widths(sc, C, rows, dtype):
    import torch
    x, r, (w0, w1, b0, b1) = tensors(torch, dtype, rows, C)
    post, pre = (RMS, w0, None, EPS), (LAYER, w1, b1, EPS)
    s, y = torch.full_like(x, math.nan), torch.full_like(x, math.nan)
    sc.check(sc.residual_norm_fwd(x, r, s, y, rows, C, post, pre, scale=0.5, dtype=dtype), "residual_norm_fwd")
    want = reference(x, r, post, pre, None, 0.5, C, dtype == BF16)
    check(torch, s, want[0], "sum")
    check(torch, y, want[1], "y")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("post", [None, NONE, RMS, LAYER])
@pytest.mark.parametrize("pre", [None, RMS, LAYER])
@pytest.mark.parametrize("have", ["all", "no residual", "no sum", "no y", "no vectors"])
@pytest.mark.parametrize("gate_rows", [0, 1, 3, 50])
def test_forms(sc, post, pre, have, gate_rows, dtype):
    """Every kind of norm, what may be left out, gates by row, by groups that do not divide the rows, and one for all."""
    import torch
    rows, C = 50, 328
    x, r, (w0, w1, b0, b1) = tensors(torch, dtype, rows, C, seed=1)
    gate = None
    if gate_rows:
        n = -(-rows // gate_rows)
        gate = torch.randn(n, C, generator=torch.Generator().manual_seed(2)).cuda()
    if have == "no vectors":
        w0 = w1 = b0 = b1 = None
    p0 = None if post is None else (post, w0, b0, EPS)
    p1 = None if pre is None else (pre, w1, b1, EPS)
    rr = None if have == "no residual" else r
    s = None if have == "no sum" else torch.full_like(x, math.nan)
    y = None if have == "no y" else torch.full_like(x, math.nan)
    sc.check(sc.residual_norm_fwd(x, rr, s, y, rows, C, p0, p1, gate=gate, gate_rows=max(1, gate_rows), scale=-1.5,
                                  dtype=dtype), "residual_norm_fwd")
    of_row = None if gate is None else gate.repeat_interleave(gate_rows, dim=0)[:rows]
    none = (NONE, None, None, EPS)
    want = reference(x, rr, p0 or none, p1 or none, of_row, -1.5, C, dtype == BF16)
    if s is not None:
        check(torch, s, want[0], "sum")
    if y is not None:
        check(torch, y, want[1], "y")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,C", [(5, 1024), (700, 1000), (900, 4096)])
def test_in_place_and_strides(sc, rows, C, dtype):
    import torch
    x, r, (w0, w1, b0, b1) = tensors(torch, dtype, rows, C, seed=3)
    post, pre = (LAYER, w0, b0, EPS), (RMS, w1, None, EPS)
    want = reference(x, r, post, pre, None, 1.0, C, dtype == BF16)
    s, y = r.clone(), x.clone()
    sc.check(sc.residual_norm_fwd(y, s, s, y, rows, C, post, pre, dtype=dtype), "residual_norm_fwd")
    check(torch, s, want[0], "sum in the residual's place")
    check(torch, y, want[1], "y in x's place")
    # rows inside wider ones, guard elements between them; a residual row that all share
    pitch = C + 24
    buf = torch.full((3, rows, pitch), 7.0, dtype=x.dtype, device="cuda")
    buf[0, :, 8:8 + C] = x
    sc.check(sc.residual_norm_fwd(buf[0, 0, 8:], r, buf[1, 0, 16:], buf[2], rows, C, post, pre, dtype=dtype,
                                  strides=(pitch, 0, pitch, pitch)), "residual_norm_fwd")
    want = reference(x, r[:1].expand(rows, C), post, pre, None, 1.0, C, dtype == BF16)
    check(torch, buf[1, :, 16:16 + C], want[0], "strided sum")
    check(torch, buf[2, :, :C], want[1], "strided y")
    buf[0, :, 8:8 + C] = buf[1, :, 16:16 + C] = buf[2, :, :C] = 7.0
    assert (buf == 7.0).all(), "something between the rows was written"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_hard_rows(sc, dtype):
    """A row of zeros, one far from its mean's size, constant rows, large and tiny values; a NaN stays in its row."""
    import torch
    rows, C = 8, 512
    x, r, (w0, w1, b0, b1) = tensors(torch, dtype, rows, C, seed=4)
    x[0] = 0
    x[1] = 1000.0 + x[1]
    x[2] = 3.0
    x[3] *= 2.0 ** 50
    x[4] *= 2.0 ** -60
    post, pre = (LAYER, w0, b0, 1e-5), (RMS, w1, None, 1e-5)
    s, y = torch.empty_like(x), torch.empty_like(x)
    sc.check(sc.residual_norm_fwd(x, None, s, y, rows, C, post, pre, dtype=dtype), "residual_norm_fwd")
    want = reference(x, None, post, pre, None, 1.0, C, dtype == BF16)
    check(torch, s, want[0], "sum")
    check(torch, y, want[1], "y")
    x[5, 77] = math.nan
    t = torch.empty_like(x)
    sc.check(sc.residual_norm_fwd(x, None, s, t, rows, C, post, pre, dtype=dtype), "residual_norm_fwd")
    assert t[5].isnan().all()
    keep = torch.arange(rows, device="cuda") != 5
    assert torch.equal(t[keep], y[keep])


@pytest.mark.gpu
def test_offsets_beyond_32_bits_and_graph(sc):
    import torch
    rows, C, pitch = 3, 64, 1 << 30
    x, r, (w0, w1, b0, b1) = tensors(torch, BF16, rows, C, seed=5)
    buf = torch.empty(2 * pitch + 128, dtype=torch.bfloat16, device="cuda")
    for i in range(rows):
        buf[i * pitch:i * pitch + C] = x[i]
    pre = (RMS, w1, None, EPS)
    s = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sc.check(sc.residual_norm_fwd(buf, r, s, buf[64:], rows, C, None, pre, dtype=BF16,
                                      strides=(pitch, C, C, pitch)), "residual_norm_fwd")
    graph.replay()
    torch.cuda.synchronize()
    want = reference(x, r, (NONE, None, None, EPS), pre, None, 1.0, C, True)
    check(torch, s, want[0], "sum")
    check(torch, torch.stack([buf[i * pitch + 64:i * pitch + 64 + C] for i in range(rows)]), want[1], "y")


A, B, C_, D_, E, G = (1 << k for k in (20, 24, 28, 32, 34, 36))


@pytest.mark.parametrize("change,expect", [
    (dict(x=None), scl.SC_ERR_NULL), (dict(sum=None, y=None), scl.SC_ERR_NULL),
    (dict(rows=0), scl.SC_ERR_SHAPE), (dict(C=0), scl.SC_ERR_SHAPE), (dict(rows=(1 << 30) + 1), scl.SC_ERR_SHAPE),
    (dict(gate=E, gate_rows=0), scl.SC_ERR_SHAPE), (dict(dtype=5), scl.SC_ERR_UNSUPPORTED),
    (dict(C=60), scl.SC_ERR_UNSUPPORTED), (dict(C=16392), scl.SC_ERR_UNSUPPORTED), (dict(scale=math.inf), scl.SC_ERR_UNSUPPORTED),
    (dict(scale=math.nan), scl.SC_ERR_UNSUPPORTED),
    (dict(pre=(3, None, None, EPS)), scl.SC_ERR_UNSUPPORTED), (dict(post=(-1, None, None, EPS)), scl.SC_ERR_UNSUPPORTED),
    (dict(pre=(1, None, None, -1.0)), scl.SC_ERR_UNSUPPORTED), (dict(post=(1, None, None, math.nan)), scl.SC_ERR_UNSUPPORTED),
    (dict(pre=(1, G + 4, None, EPS)), scl.SC_ERR_ALIGN), (dict(post=(2, None, G + 8, EPS)), scl.SC_ERR_ALIGN),
    (dict(x=A + 4), scl.SC_ERR_ALIGN), (dict(residual=B + 8), scl.SC_ERR_ALIGN), (dict(sum=C_ + 4), scl.SC_ERR_ALIGN),
    (dict(y=D_ + 8), scl.SC_ERR_ALIGN), (dict(gate=E + 4), scl.SC_ERR_ALIGN),
    (dict(strides=(66, 64, 64, 64)), scl.SC_ERR_ALIGN), (dict(strides=(64, 64, 64, 65)), scl.SC_ERR_ALIGN),
    (dict(strides=(-64, 64, 64, 64)), scl.SC_ERR_SHAPE), (dict(strides=(64, 1 << 60, 64, 64)), scl.SC_ERR_SHAPE),
    (dict(strides=(64, 64, 0, 64)), scl.SC_ERR_ALIAS), (dict(strides=(64, 64, 64, 32)), scl.SC_ERR_ALIAS),
    (dict(sum=A + 64), scl.SC_ERR_ALIAS), (dict(y=B + 16), scl.SC_ERR_ALIAS), (dict(y=C_), scl.SC_ERR_ALIAS),
    (dict(sum=B, strides=(64, 72, 64, 64)), scl.SC_ERR_ALIAS), (dict(y=E, gate=E), scl.SC_ERR_ALIAS),
    (dict(y=G, pre=(1, G + 16, None, EPS)), scl.SC_ERR_ALIAS), (dict(sum=G, post=(2, None, G, EPS)), scl.SC_ERR_ALIAS),
])
def test_refusals(change, expect):
    a = dict(x=A, residual=B, sum=C_, y=D_, rows=5, C=64, post=None, pre=None, gate=None, gate_rows=1, scale=1.0, dtype=F32,
             strides=None)
    a.update(change)
    rc = scl.residual_norm_fwd(a["x"], a["residual"], a["sum"], a["y"], a["rows"], a["C"], a["post"], a["pre"], a["gate"],
                               a["gate_rows"], a["scale"], a["dtype"], a["strides"], stream=0)
    assert rc == expect, scl.sc_status_string(rc)
