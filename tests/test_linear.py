"""linear_fwd against the plain 64-bit form, and its refusals (bounds: layer_ref.py)."""
import pytest

import layer_ref as ref
import stencil_conv2d_fwd_gb300 as scl

BF16, F32 = scl.SC_BF16, scl.SC_F32


def tensors(torch, dtype, rows, Cin, Cout, seed=0, bias=True, residual=True):
    g = torch.Generator().manual_seed(seed)
    t = torch.bfloat16 if dtype == BF16 else torch.float32
    x = torch.randn(rows, Cin, generator=g).to(t).cuda()
    w = (torch.randn(Cout, Cin, generator=g) * Cin ** -0.5).to(t).cuda()
    b = torch.randn(Cout, generator=g).cuda() if bias else None
    r = torch.randn(rows, Cout, generator=g).to(t).cuda() if residual else None
    return x, w, b, r


def check(torch, y, x, w, b, r, act, dtype):
    want, mag, a = ref.linear(x, w, b, r, act)
    bound = ref.linear_bound(want, mag, a, x.shape[1], dtype == BF16)
    err = (y.double() - want).abs()
    assert torch.isfinite(y.float()).all()
    worst = (err / bound).max().item()
    assert worst <= 1, f"{worst:.2f} of its bound at {(err / bound).argmax().item()} of {tuple(y.shape)}"


def run(torch, sc, x, w, b, r, act, dtype, stream=None):
    (rows, Cin), Cout = x.shape, w.shape[0]
    y = torch.full((rows, Cout), float("nan"), dtype=x.dtype, device="cuda")
    sc.check(sc.linear_fwd(x, w, b, y, rows, Cin, Cout, act, dtype, residual=r, stream=stream), "linear_fwd")
    sc.check(sc.sc_last_device_status(stream), "device status")
    return y


# (rows, Cin, Cout): one row to many, around tiles, odd rows and outputs, narrow and long sums
SHAPES = [
    (1, 8, 1), (1, 64, 7), (1, 1024, 1024), (1, 4096, 257), (2, 520, 1000), (3, 512, 4001), (4, 1024, 1024), (5, 72, 33),
    (8, 2048, 515), (9, 136, 129), (15, 1000, 64), (16, 512, 2048), (17, 512, 2048), (17, 8, 1), (31, 264, 77), (33, 64, 128),
    (64, 1024, 63), (77, 512, 512), (100, 2000, 1001), (127, 1024, 127), (128, 64, 256), (129, 128, 257), (255, 640, 513),
    (300, 320, 129), (513, 72, 640), (1001, 512, 300), (4000, 256, 130), (2, 32, 20001), (700, 2048, 2051), (130, 4104, 70),
    (20000, 64, 24),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(sc, shape, dtype):
    import torch
    x, w, b, r = tensors(torch, dtype, *shape)
    check(torch, run(torch, sc, x, w, b, r, sc.SC_ACT_NONE, dtype), x, w, b, r, sc.SC_ACT_NONE, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", [ref.ACT_NONE, ref.ACT_RELU, ref.ACT_GELU, ref.ACT_SILU])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("shape", [(3, 256, 130), (140, 256, 200), (700, 128, 515), (1100, 264, 132), (1030, 256, 515)])
def test_epilogues(sc, shape, bias, residual, act, dtype):
    import torch
    x, w, b, r = tensors(torch, dtype, *shape, seed=1, bias=bias, residual=residual)
    if b is not None:
        b *= 3   # arguments of the activations from -10 to 10
    check(torch, run(torch, sc, x, w, b, r, act, dtype), x, w, b, r, act, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 12, 300, 1100])
def test_fp32_gelu_keeps_its_digits_on_the_negative_side(sc, rows):
    """Products that are one element exactly, from -12.5 to 12.5, against v erfc(-v / sqrt 2) / 2.  The exponent v^2 / 2 log2 e
    has three roundings (v^2, the constant, the product), each U of it, so exp(-v^2 / 2) is off by 1.5 v^2 U, and by 4 U of
    the exponential's own 2 ulp; the reciprocal has 2 U; 1 + 0.28 v, nine fused steps of a polynomial without cancellation (the
    last two count, the earlier ones less and less), the fit's 5.8e-8 and four products are 1 U each: 2 v^2 + 16 in all."""
    import torch
    Cin, Cout = 8, 40
    x, w = torch.zeros(rows, Cin, device="cuda"), torch.zeros(Cout, Cin, device="cuda")
    w[:, 0] = torch.linspace(-12.5, 12.5, Cout, device="cuda")
    x[:, 0] = 1.0
    y = run(torch, sc, x, w, None, None, sc.SC_ACT_GELU, F32)
    v = w[:, 0].double()
    want = 0.5 * v * torch.erfc(-v / 2.0 ** 0.5)   # (ndtr is 1 + erf, which cancels in 64 bits too)
    err = (y.double() - want).abs()
    assert (err <= ref.U * (2 * v * v + 16) * want.abs()).all(), (err / want.abs()).amax(dim=0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(3, 128, 50), (16, 256, 100), (200, 128, 131), (513, 512, 264), (1100, 256, 264)])
@pytest.mark.parametrize("pad", [8, 40])
def test_strides(sc, shape, pad, dtype):
    """Rows inside wider ones (a fused projection), y at an odd address and pitch, guard bytes around y."""
    import torch
    rows, Cin, Cout = shape
    x, w, b, r = tensors(torch, dtype, *shape, seed=2)
    xw, ww = torch.full((rows, Cin + pad), float("nan"), dtype=x.dtype, device="cuda"), \
        torch.full((Cout, Cin + pad), float("nan"), dtype=x.dtype, device="cuda")
    xw[:, 8:8 + Cin], ww[:, :Cin] = x, w
    for off, pitch in ((0, Cout + 8), (1, Cout + 3)):
        buf = torch.full((rows * pitch + 16,), 7.0, dtype=x.dtype, device="cuda")
        rbuf = torch.full((rows * pitch + 16,), 7.0, dtype=x.dtype, device="cuda")
        view = buf[off:off + rows * pitch].view(rows, pitch)
        rbuf[off:off + rows * pitch].view(rows, pitch)[:, :Cout] = r
        sc.check(sc.linear_fwd(xw[0, 8:], ww, b, view, rows, Cin, Cout, 0, dtype,
                               residual=rbuf[off:], strides=(Cin + pad, Cin + pad, pitch, pitch)), "linear_fwd")
        sc.check(sc.sc_last_device_status())
        check(torch, view[:, :Cout], x, w, b, r, 0, dtype)
        view[:, :Cout] = 7.0
        assert (buf == 7.0).all(), "something outside y was written"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rows", [(F32, 3), (F32, 12), (F32, 1100), (BF16, 12), (BF16, 40), (BF16, 300)])
@pytest.mark.parametrize("Cout", [1, 2, 3, 5, 6, 7, 9, 31, 33, 34, 63, 65, 127, 129, 130, 423, 1377])
@pytest.mark.parametrize("residual", [False, True])
def test_nothing_beside_y_is_written(sc, dtype, rows, Cout, residual):
    """Any number of outputs in rows of whole 16-byte units, y and the residual a slice of something wider: the columns
    behind y's last one stay as they are."""
    import torch
    Cin = 64
    x, w, b, r = tensors(torch, dtype, rows, Cin, Cout, seed=12, residual=True)
    pitch = (Cout + 16) // 8 * 8
    wide, rwide = (torch.full((rows, pitch), 7.0, dtype=x.dtype, device="cuda") for _ in range(2))
    rwide[:, :Cout] = r
    sc.check(sc.linear_fwd(x, w, b, wide, rows, Cin, Cout, 0, dtype, residual=rwide if residual else None,
                           strides=(Cin, Cin, pitch, pitch)), "linear_fwd")
    sc.check(sc.sc_last_device_status())
    check(torch, wide[:, :Cout], x, w, b, r if residual else None, 0, dtype)
    assert (wide[:, Cout:] == 7.0).all(), f"columns {sorted(set((wide[:, Cout:] != 7.0).nonzero()[:, 1].tolist()))} behind y"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(4, 256, 512), (300, 256, 515), (1100, 256, 512), (2000, 1024, 2048)])
def test_residual_in_place_and_shared(sc, shape, dtype):
    import torch
    rows, Cin, Cout = shape
    x, w, b, r = tensors(torch, dtype, *shape, seed=3)
    y = r.clone()
    sc.check(sc.linear_fwd(x, w, b, y, rows, Cin, Cout, 0, dtype, residual=y), "linear_fwd")
    check(torch, y, x, w, b, r, 0, dtype)
    y = torch.empty_like(r)
    sc.check(sc.linear_fwd(x, w, b, y, rows, Cin, Cout, sc.SC_ACT_SILU, dtype, residual=r,
                           strides=(Cin, Cin, Cout, 0)), "linear_fwd")
    check(torch, y, x, w, b, r[:1].expand(rows, -1), sc.SC_ACT_SILU, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [2, 40, 1500])
def test_not_finite(sc, rows, dtype):
    """An infinity or NaN reaches the outputs of its row (x) or column (w), and no others."""
    import torch
    x, w, b, r = tensors(torch, dtype, rows, 256, 140, seed=4)
    clean = run(torch, sc, x, w, b, r, sc.SC_ACT_RELU, dtype)
    x[1, 100] = float("nan")
    w[9, 30] = float("inf")
    y = run(torch, sc, x, w, b, r, sc.SC_ACT_NONE, dtype)
    assert y[1].isnan().all()
    col = y[:, 9]
    want = torch.where(x[:, 30] > 0, float("inf"), float("-inf")).to(col.dtype)
    assert (col[0] == want[0]) and (col[2:] == want[2:]).all() and col[1].isnan()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[1], keep[:, 9] = False, False
    again = run(torch, sc, x, w, b, r, sc.SC_ACT_RELU, dtype)
    assert torch.equal(again[keep], clean[keep])
    assert again[1].isnan().all()   # a NaN passes the activation


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 12, 100, 1500])
@pytest.mark.parametrize("big", [3e38, 1e-30])
def test_ends_of_fp32(sc, rows, big):
    """Values above bf16's largest, and products near fp32's smallest."""
    import torch
    x, w, b, r = tensors(torch, F32, rows, 64, 40, seed=5, bias=False, residual=False)
    if big > 1:
        x = torch.where(torch.arange(64, device="cuda") == 5, big * torch.sign(x), 0 * x)
        x[:, 5] *= 1.13   # 3.39e38: between bf16's largest and fp32's
        w = w.clamp(-1, 1)
    else:
        x, w = x * 1e-20, w * 1e-8
    y = run(torch, sc, x, w, None, None, 0, F32)
    want, mag, a = ref.linear(x, w, None, None, 0)
    assert ((y.double() - want).abs() <= ref.linear_bound(want, mag, a, 64, False)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(4, 512, 700), (200, 1024, 300), (1500, 512, 1100)])
def test_streams_graph_and_same_bits(sc, shape, dtype):
    """Two streams at once, a captured call replayed on other inputs, and the same bits every time."""
    import torch
    x, w, b, r = tensors(torch, dtype, *shape, seed=6)
    first = run(torch, sc, x, w, b, r, sc.SC_ACT_GELU, dtype)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(first) for _ in range(12)]
    torch.cuda.synchronize()
    for i, y in enumerate(outs):
        sc.check(sc.linear_fwd(x, w, b, y, *x.shape, w.shape[0], sc.SC_ACT_GELU, dtype, residual=r,
                               stream=streams[i % 3]), "linear_fwd")
    torch.cuda.synchronize()
    assert all(torch.equal(y, first) for y in outs)
    y, z, xin = torch.empty_like(first), torch.empty_like(first), torch.zeros_like(x)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, out in zip(graphs, (y, z)):   # two graphs, each with its own temporary buffers
        with torch.cuda.graph(graph):
            sc.check(sc.linear_fwd(xin, w, b, out, *x.shape, w.shape[0], sc.SC_ACT_GELU, dtype, residual=r), "linear_fwd")
    xin.copy_(x)
    torch.cuda.synchronize()
    for graph, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first) and torch.equal(z, first)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rows", [(F32, 2), (BF16, 2), (BF16, 40)])
def test_offsets_beyond_32_bits(sc, dtype, rows):
    """The last row of x, w and y lies more than 2^31 elements behind the first."""
    import torch
    Cin, Cout = 64, 24
    x, w, b, r = tensors(torch, dtype, rows, Cin, Cout, seed=7)
    big = ((1 << 31) // (rows - 1) + 8192) // 64 * 64
    buf = torch.empty(big * (rows - 1) + 128, dtype=x.dtype, device="cuda")
    for i in range(rows):
        buf[i * big:i * big + Cin] = x[i]
        buf[i * big + Cin:i * big + Cin + Cout] = 7.0
    y = buf[Cin:]
    sc.check(sc.linear_fwd(buf, w, b, y, rows, Cin, Cout, 0, dtype, residual=r, strides=(big, Cin, big, Cout)), "linear_fwd")
    sc.check(sc.sc_last_device_status())
    got = torch.stack([y[i * big:i * big + Cout] for i in range(rows)])
    check(torch, got, x, w, b, r, 0, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rows", [(F32, 2), (F32, 8), (F32, 40), (F32, 1100), (BF16, 2), (BF16, 12), (BF16, 40), (BF16, 300)])
@pytest.mark.parametrize("odd", [False, True])
def test_every_operand_beyond_32_bits(sc, dtype, rows, odd):
    """The last row of each of x, w, y and the residual lies more than 2^31 elements behind its first, y's and the
    residual's pitches whole 16-byte units (TMA takes them to and from the tensor cores' epilogue) or odd, in every kernel:
    FMA, MMAs of few rows, three planes, tensor cores."""
    import torch
    Cin, Cout = 64, 24

    def far(t, unit):
        n, cols = t.shape
        pitch = (((1 << 31) + 4096) // (n - 1) // unit + 1) * unit | (unit == 1)
        v = torch.empty(pitch * (n - 1) + cols + 16, dtype=t.dtype, device="cuda").as_strided((n, cols), (pitch, 1))
        v.copy_(t)
        return v, pitch

    x, w, b, r = tensors(torch, dtype, rows, Cin, Cout, seed=11)
    unit = 1 if odd else 16
    (xf, xs), (wf, ws), (rf, rs) = far(x, 16), far(w, 16), far(r, unit)
    yf, ys = far(torch.full_like(r, float("nan")), unit)
    assert min(xs * (rows - 1), ws * (Cout - 1), rs * (rows - 1), ys * (rows - 1)) > 1 << 31
    sc.check(sc.linear_fwd(xf, wf, b, yf, rows, Cin, Cout, 0, dtype, residual=rf, strides=(xs, ws, ys, rs)), "linear_fwd")
    sc.check(sc.sc_last_device_status())
    check(torch, yf.contiguous(), x, w, b, r, 0, dtype)


A, B, C, D_ = 1 << 20, 1 << 24, 1 << 28, 1 << 32   # addresses, 16-byte aligned, never dereferenced


@pytest.mark.parametrize("change,expect", [
    (dict(x=None), scl.SC_ERR_NULL), (dict(w=None), scl.SC_ERR_NULL), (dict(y=None), scl.SC_ERR_NULL),
    (dict(rows=0), scl.SC_ERR_SHAPE), (dict(Cin=-8), scl.SC_ERR_SHAPE), (dict(Cout=0), scl.SC_ERR_SHAPE),
    (dict(rows=(1 << 30) + 1), scl.SC_ERR_SHAPE), (dict(rows=1 << 30, Cin=1 << 30), scl.SC_ERR_SHAPE),
    (dict(Cin=12), scl.SC_ERR_UNSUPPORTED), (dict(act=4), scl.SC_ERR_UNSUPPORTED), (dict(act=-1), scl.SC_ERR_UNSUPPORTED),
    (dict(dtype=2), scl.SC_ERR_UNSUPPORTED), (dict(x=A + 8), scl.SC_ERR_ALIGN), (dict(w=B + 4), scl.SC_ERR_ALIGN),
    (dict(y=C + 2), scl.SC_ERR_ALIGN), (dict(b=D_ + 2), scl.SC_ERR_ALIGN), (dict(residual=D_ + 2), scl.SC_ERR_ALIGN),
    (dict(strides=(66, 64, 32, 32)), scl.SC_ERR_ALIGN), (dict(strides=(64, 70, 32, 32)), scl.SC_ERR_ALIGN),
    (dict(strides=(0, 64, 32, 32)), scl.SC_ERR_UNSUPPORTED), (dict(strides=(64, 56, 32, 32)), scl.SC_ERR_UNSUPPORTED),
    (dict(strides=(-64, 64, 32, 32)), scl.SC_ERR_SHAPE), (dict(strides=(64, 64, 32, -1), residual=D_), scl.SC_ERR_SHAPE),
    (dict(strides=(1 << 60, 64, 32, 32)), scl.SC_ERR_SHAPE), (dict(strides=(1 << 38, 64, 32, 32)), scl.SC_ERR_UNSUPPORTED),
    (dict(strides=(64, 64, 31, 32)), scl.SC_ERR_ALIAS), (dict(strides=(64, 64, 0, 32)), scl.SC_ERR_ALIAS),
    (dict(y=A + 64), scl.SC_ERR_ALIAS), (dict(y=B), scl.SC_ERR_ALIAS), (dict(y=C, b=C + 16), scl.SC_ERR_ALIAS),
    (dict(residual=C + 4), scl.SC_ERR_ALIAS), (dict(residual=C, strides=(64, 64, 32, 40)), scl.SC_ERR_ALIAS),
    (dict(residual=C, strides=(64, 64, 32, 0)), scl.SC_ERR_ALIAS),
])
def test_refusals(change, expect):
    a = dict(x=A, w=B, b=None, y=C, rows=5, Cin=64, Cout=32, act=0, dtype=F32, residual=None, strides=None)
    a.update(change)
    rc = scl.linear_fwd(a["x"], a["w"], a["b"], a["y"], a["rows"], a["Cin"], a["Cout"], a["act"], a["dtype"],
                        residual=a["residual"], strides=a["strides"], stream=0)
    assert rc == expect, scl.sc_status_string(rc)


@pytest.mark.parametrize("act", [scl.SC_ACT_GELU, scl.SC_ACT_SILU])
def test_convolutions_take_no_other_activation(act):
    assert scl.conv2d_fwd(A, B, None, C, 1, 8, 8, 8, 8, 1, 1, scl.SC_NHWC, act, stream=0) == scl.SC_ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,drop_copy", [((40, 256, 300), 0), ((300, 1024, 700), 3), ((5000, 512, 2100), 17)])
def test_expired_wait_is_reported(sc, shape, drop_copy, dtype):
    """Stages whose copies are never issued: the waits run out, the status says so, and the next call is right."""
    import torch
    x, w, _, _ = tensors(torch, dtype, *shape, seed=8, bias=False, residual=False)
    y = torch.empty(shape[0], shape[2], dtype=x.dtype, device="cuda")
    sc.check(sc.sc_test_linear_wait_expiry(x, w, y, *shape, dtype, drop_copy, 2000), "sc_test_linear_wait_expiry")
    assert sc.sc_last_device_status() == sc.SC_ERR_DEVICE_TIMEOUT
    assert sc.sc_last_device_status() == sc.SC_OK
    check(torch, run(torch, sc, x, w, None, None, 0, dtype), x, w, None, None, 0, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(40, 256, 300), (1030, 1024, 700), (5000, 1024, 2100)])
def test_waits_that_expire_anywhere(sc, shape, dtype):
    """No copy is left out, but the waits' limit is as short as the waits themselves, so that they run out in one warp or
    another, in one CTA of a pair or in both, at the start or in the middle: each call ends, says so or not, and the next
    ordinary one is right.  Then a stage left out early in a long product, where the pair's second CTA is left waiting."""
    import torch
    x, w, _, _ = tensors(torch, dtype, *shape, seed=9, bias=False, residual=False)
    y = torch.empty(shape[0], shape[2], dtype=x.dtype, device="cuda")
    seen = set()
    for drop_copy, limit in [(1 << 30, t) for t in (1, 2, 3, 5, 8, 13, 20, 30) for _ in range(8)] + [(1, 100), (9, 100)]:
        sc.check(sc.sc_test_linear_wait_expiry(x, w, y, *shape, dtype, drop_copy, limit), "sc_test_linear_wait_expiry")
        torch.cuda.synchronize()
        seen.add(sc.sc_last_device_status())
    assert seen <= {sc.SC_OK, sc.SC_ERR_DEVICE_TIMEOUT} and sc.SC_ERR_DEVICE_TIMEOUT in seen
    check(torch, run(torch, sc, x, w, None, None, 0, dtype), x, w, None, None, 0, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(40, 256, 320), (1030, 512, 704), (5000, 512, 2112)])
def test_waits_that_expire_beside_copies_of_the_residual(sc, shape, dtype):
    """Waits that run out while parts of the residual are on their way to the epilogue's staging: every call ends, the
    residual stays as it is, and the next ordinary call is right."""
    import torch
    x, w, _, r = tensors(torch, dtype, *shape, seed=10, bias=False)
    keep, y, seen = r.clone(), torch.empty_like(r), set()
    for drop_copy, limit in [(1 << 30, t) for t in (1, 2, 3, 5, 8, 13, 20, 30) for _ in range(8)] + [(2, 100)]:
        sc.check(sc.sc_test_linear_wait_expiry(x, w, y, *shape, dtype, drop_copy, limit, residual=r), "sc_test_linear_wait_expiry")
        torch.cuda.synchronize()
        seen.add(sc.sc_last_device_status())
    assert seen <= {sc.SC_OK, sc.SC_ERR_DEVICE_TIMEOUT} and sc.SC_ERR_DEVICE_TIMEOUT in seen
    assert torch.equal(r, keep)
    check(torch, run(torch, sc, x, w, None, r, 0, dtype), x, w, None, r, 0, dtype)


def test_wait_expiry_hook_refusals():
    assert scl.sc_test_linear_wait_expiry(None, B, C, 5, 64, 32, BF16, 0, 10, stream=0) == scl.SC_ERR_NULL
    assert scl.sc_test_linear_wait_expiry(A, B, C, 5, 64, 32, BF16, -1, 10, stream=0) == scl.SC_ERR_SHAPE
    assert scl.sc_test_linear_wait_expiry(A, B, C, 5, 64, 32, BF16, 0, 0, stream=0) == scl.SC_ERR_SHAPE
    assert scl.sc_test_linear_wait_expiry(A, B, C, 5, 60, 32, BF16, 0, 10, stream=0) == scl.SC_ERR_UNSUPPORTED
