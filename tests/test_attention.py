"""cross_attention_fwd against the plain 64-bit form, and its refusals.

The bounds are those of attention_ref.py: fp32 scores and sums, one rounding
of the weights and of the output to bf16 for bf16 tensors."""
import math

import numpy as np
import pytest

import attention_ref as ref
import stencil_conv2d_fwd_gb300 as scl

BF16, F32 = scl.SC_BF16, scl.SC_F32


def make(torch, dtype, *shape, seed=0, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(*shape, generator=g) * gain
    return (t.bfloat16() if dtype == BF16 else t).cuda()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def valid_of(N, Tk, k_len=None, key_mask=None):
    valid = np.ones((N, Tk), bool)
    if k_len is not None:
        valid &= np.arange(Tk)[None, :] < np.asarray(k_len)[:, None]
    if key_mask is not None:
        valid &= np.asarray(key_mask) != 0
    return valid


def run_and_check(torch, sc, q, k, v, dtype, k_len=None, key_mask=None, scale=None, strides=None, out=None, stream=None,
                  ref_kv=None):
    N, Tq, Hq, D = q.shape
    Tk, Hkv = k.shape[1], k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    if out is None:
        out = torch.full((N, Tq, Hq, D), float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full((N, Hq, Tq), float("nan"), device="cuda")
    kl = None if k_len is None else torch.tensor(k_len, dtype=torch.int32, device="cuda")
    km = None if key_mask is None else torch.as_tensor(np.asarray(key_mask, np.uint8)).cuda()
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    sc.check(sc.cross_attention_fwd(q, k, v, out, N, Tq, Tk, Hq, Hkv, D, scale, dtype, k_len=kl, key_mask=km, lse=lse,
                                    strides=strides, stream=stream), "cross_attention_fwd")
    sc.check(sc.sc_last_device_status(stream), "device status")
    kk, vv = ref_kv if ref_kv is not None else (k, v)
    valid = None if k_len is None and key_mask is None else valid_of(N, Tk, k_len, key_mask)
    o, z, wabs, mag = ref.attention(f64(q), f64(kk), f64(vv), scale, valid)
    got, gz = f64(out), f64(lse)
    err = np.abs(got - o)
    bound = ref.out_bound(o, wabs, mag, D, Tk, dtype == BF16)
    assert np.isfinite(got).all()
    assert (err <= bound).all(), f"out: worst {np.max(err / bound):.2f} of its bound at {np.unravel_index(np.argmax(err / bound), err.shape)}"
    assert np.array_equal(np.isneginf(gz), np.isneginf(z))
    ok = np.isfinite(z)
    zerr = np.abs(np.where(ok, gz, 0) - np.where(ok, z, 0))
    assert (zerr <= ref.lse_bound(z, mag, D, Tk)).all(), f"lse: worst {np.max(zerr / ref.lse_bound(z, mag, D, Tk)):.2f}"
    return out, lse


# (N, Tq, Tk, Hq, Hkv, D): one token to many; lengths around tiles; odd widths; shared heads
SHAPES = [
    (1, 1, 1, 1, 1, 8),
    (1, 1, 960, 4, 4, 64),
    (2, 1, 257, 4, 2, 24),
    (3, 1, 1000, 5, 1, 64),
    (1, 1, 20000, 4, 1, 64),
    (2, 1, 333, 16, 2, 96),
    (2, 2, 129, 3, 3, 40),
    (2, 3, 700, 4, 4, 32),
    (1, 5, 128, 6, 2, 128),
    (1, 9, 130, 2, 1, 80),
    (2, 16, 640, 8, 2, 64),
    (1, 16, 9000, 2, 1, 128),
    (3, 77, 391, 4, 4, 64),
    (1, 100, 1, 2, 2, 48),
    (1, 127, 127, 3, 1, 128),
    (1, 128, 128, 1, 1, 64),
    (1, 129, 129, 2, 2, 16),
    (2, 255, 513, 2, 1, 72),
    (1, 257, 385, 5, 1, 104),
    (1, 300, 1300, 4, 4, 128),
    (1, 1000, 300, 2, 2, 56),
    (1, 500, 900, 3, 3, 64),
    (2, 260, 4100, 4, 1, 24),
    (1, 40, 20000, 2, 2, 72),
    (1, 1, 300, 150, 1, 32),
    (2, 3, 500, 200, 1, 64),
    (1, 10, 2000, 150, 1, 64),
    (1, 5, 1500, 260, 2, 128),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(sc, shape, dtype):
    import torch
    N, Tq, Tk, Hq, Hkv, D = shape
    q = make(torch, dtype, N, Tq, Hq, D, seed=1, gain=2.0)
    k, v = make(torch, dtype, N, Tk, Hkv, D, seed=2), make(torch, dtype, N, Tk, Hkv, D, seed=3)
    run_and_check(torch, sc, q, k, v, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Tq,G", [(1, 1), (1, 4), (3, 1), (77, 1), (70, 4), (300, 2)])
@pytest.mark.parametrize("Tk", [100, 128, 700, 4500])
def test_lengths(sc, dtype, Tq, G, Tk):
    """Lengths of zero, one, around a tile's end, all of Tk, above it and below zero; garbage beyond them."""
    import torch
    lens = [0, 1, 63, 64, min(Tk, 127), Tk - 1, Tk, Tk + 9, -3]
    N, Hkv, D = len(lens), 2, 64
    q = make(torch, dtype, N, Tq, Hkv * G, D, seed=4, gain=2.0)
    k, v = make(torch, dtype, N, Tk, Hkv, D, seed=5), make(torch, dtype, N, Tk, Hkv, D, seed=6)
    for n, L in enumerate(lens):
        k[n, max(0, L):] = float("nan")
        v[n, max(0, L):] = float("inf")
    out, lse = run_and_check(torch, sc, q, k, v, dtype, k_len=lens)
    assert (out[0] == 0).all() and (out[-1] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Tq,G,D", [(1, 1, 64), (1, 4, 128), (2, 2, 32), (77, 1, 64), (40, 3, 128), (290, 1, 80)])
def test_masks(sc, dtype, Tq, G, D):
    """Masks that leave nothing, one state, every other one, a padded map, and whole tiles empty;
    NaN and infinities in the masked places; a length on top."""
    import torch
    h, w = 25, 31
    Tk, N, Hkv = h * w, 6, 2
    rng = np.random.default_rng(7)
    mask = np.zeros((N, Tk), np.uint8)
    mask[1, 700] = 1
    mask[2, ::2] = 255
    m = np.zeros((h, w), np.uint8)
    m[:19, :17] = 1
    mask[3] = m.reshape(-1)
    mask[4] = rng.random(Tk) < 0.5
    mask[5, 300:520] = 2
    lens = [Tk, Tk, Tk, Tk, 333, 400]
    q = make(torch, dtype, N, Tq, Hkv * G, D, seed=8, gain=2.0)
    k, v = make(torch, dtype, N, Tk, Hkv, D, seed=9), make(torch, dtype, N, Tk, Hkv, D, seed=10)
    bad = torch.as_tensor(~valid_of(N, Tk, lens, mask)).cuda()
    k[bad] = float("nan")
    v[bad] = float("-inf")
    v[bad & (torch.arange(Tk, device="cuda") % 2 == 0)] = float("nan")
    out, lse = run_and_check(torch, sc, q, k, v, dtype, k_len=lens, key_mask=mask)
    assert (out[0] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("G,D", [(1, 64), (3, 40), (1, 128)])
@pytest.mark.parametrize("kind", ["all", "lengths", "mask"])
def test_more_row_tiles_than_sms(sc, dtype, G, D, kind):
    """Three row tiles of each of 66 (sequence, key head) pairs, the last of them partly full: tiles in pairs."""
    import torch
    N, Tk, Hkv = 11, 700, 6
    Tq = 300 // G
    lens = mask = None
    rng = np.random.default_rng(35)
    if kind == "lengths":
        lens = [0, 1, 127, 128, 129, 300, 384, 511, 640, 699, 700]
    elif kind == "mask":
        mask = (rng.random((N, Tk)) < 0.5).astype(np.uint8)
        mask[0] = 0
        mask[1, :400] = 0
        mask[2, 128:640] = 0
        mask[3] = 0
        mask[3, 699] = 1
    q = make(torch, dtype, N, Tq, Hkv * G, D, seed=36, gain=2.0)
    k, v = make(torch, dtype, N, Tk, Hkv, D, seed=37), make(torch, dtype, N, Tk, Hkv, D, seed=38)
    if kind != "all":
        bad = torch.as_tensor(~valid_of(N, Tk, lens, mask)).cuda()
        k[bad] = float("nan")
        v[bad] = float("inf")
    run_and_check(torch, sc, q, k, v, dtype, k_len=lens, key_mask=mask)


@pytest.mark.gpu
@pytest.mark.parametrize("Tq", [20, 300])
def test_long_masked_share(sc, Tq):
    """A mask over more states than a CTA looks through beforehand (no tile is skipped)."""
    import torch
    N, Tk, H, D = 20, 70001, 8, 64
    g = torch.Generator(device="cuda").manual_seed(39)
    q = torch.randn(N, Tq, H, D, device="cuda", generator=g).bfloat16()
    k, v = (torch.randn(N, Tk, H, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    mask = (torch.rand(N, Tk, device="cuda", generator=g) < 0.5).to(torch.uint8)
    mask[-1, :-3000] = 0
    bad = mask == 0
    k[bad] = float("nan")
    v[bad] = float("nan")
    out = torch.empty_like(q)
    sc.check(sc.cross_attention_fwd(q, k, v, out, N, Tq, Tk, H, H, D, 0.125, BF16, key_mask=mask))
    sc.check(sc.sc_last_device_status())
    for n, h in ((0, 0), (N - 1, H - 1)):
        keep = mask[n].bool()
        o, z, wabs, mag = ref.attention(f64(q[n:n + 1, :, h:h + 1]), f64(k[n:n + 1, keep, h:h + 1]),
                                        f64(v[n:n + 1, keep, h:h + 1]), 0.125)
        assert (np.abs(f64(out[n:n + 1, :, h:h + 1]) - o) <= ref.out_bound(o, wabs, mag, D, Tk, True)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Tq", [1, 2, 40, 140])
@pytest.mark.parametrize("order", ["rising", "falling", "one"])
def test_running_maximum(sc, dtype, Tq, order):
    """Scores that rise over the keys by far more than a rounding's range, that fall, and one key that outweighs all."""
    import torch
    N, Tk, H, D = 1, 1500, 2, 64
    q = make(torch, dtype, N, Tq, H, D, seed=11)
    k, v = make(torch, dtype, N, Tk, H, D, seed=12), make(torch, dtype, N, Tk, H, D, seed=13)
    q[..., 0] = 8.0
    if order == "one":
        k[:, 777, :, 0] = 60.0
    else:
        ramp = torch.linspace(-100, 100, Tk, device="cuda").view(1, Tk, 1)
        k[..., 0] = (ramp if order == "rising" else -ramp).to(k.dtype)
    run_and_check(torch, sc, q, k, v, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Tq", [1, 50, 200])
def test_strides(sc, dtype, Tq):
    """Keys and values of one fused projection, heads before tokens, a batch that shares its keys, and an
    output inside a wider row."""
    import torch
    N, Tk, Hq, Hkv, D = 2, 300, 6, 2, 40
    wide = make(torch, dtype, N, Tk, 2 * Hkv, D, seed=14)
    k, v = wide[:, :, :Hkv], wide[:, :, Hkv:]
    qh = make(torch, dtype, N, Hq, Tq, D, seed=15)
    q = qh.permute(0, 2, 1, 3)
    row = torch.zeros(N, Tq, Hq * D + 64, dtype=q.dtype, device="cuda")
    out = row[:, :, 32:32 + Hq * D].unflatten(2, (Hq, D))
    st = [t.stride()[:3] for t in (q, k, v, out)]
    run_and_check(torch, sc, q, k, v, dtype, strides=st, out=out)
    assert (row[:, :, :32] == 0).all() and (row[:, :, 32 + Hq * D:] == 0).all()
    one = k[:1].expand(N, -1, -1, -1)
    out2 = torch.empty(N, Tq, Hq, D, dtype=q.dtype, device="cuda")
    st = [q.stride()[:3], one.stride()[:3], v.stride()[:3], out2.stride()[:3]]
    assert st[1][0] == 0
    run_and_check(torch, sc, q, one, v, dtype, strides=st, out=out2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(2, 2, 300, 6, 2, 64), (3, 50, 700, 4, 2, 72), (2, 200, 700, 4, 2, 64), (2, 160, 900, 4, 4, 128)])
@pytest.mark.parametrize("which,axes", [("q", (0,)), ("q", (1,)), ("q", (2,)), ("q", (0, 1, 2)), ("k", (0,)), ("k", (2,)),
                                        ("v", (0,)), ("v", (2,)), ("kv", (0, 2)), ("k", (1,)), ("v", (1,)), ("qkv", (0,))])
@pytest.mark.parametrize("kind", ["all", "lengths", "mask"])
def test_shared_axes(sc, shape, dtype, which, axes, kind):
    """Strides of 0: queries, keys or values that the batch (0), the tokens or states (1) or the heads (2) share."""
    import torch
    N, Tq, Tk, Hq, Hkv, D = shape
    lens = [Tk, 130, 1][:N] if kind == "lengths" else None
    mask = None
    if kind == "mask":
        mask = (np.random.default_rng(111).random((N, Tk)) < 0.4).astype(np.uint8)
        mask[0, 128:300] = 0
    x, strides = {}, []
    for i, (name, T, H) in enumerate((("q", Tq, Hq), ("k", Tk, Hkv), ("v", Tk, Hkv))):
        size = [N, T, H]
        for a in axes if name in which else ():
            size[a] = 1
        x[name] = make(torch, dtype, *size, D, seed=112 + i, gain=2.0 if name == "q" else 1.0)
        if name != "q" and kind != "all" and size[:2] == [N, T]:     # states of its own: what is left out holds anything
            x[name][torch.as_tensor(~valid_of(N, Tk, lens, mask)).cuda()] = math.nan if name == "k" else math.inf
        x[name] = x[name].expand(N, T, H, D)
        strides.append([0 if size[j] == 1 else x[name].stride(j) for j in range(3)])
    out = torch.full((N, Tq, Hq, D), math.nan, dtype=x["q"].dtype, device="cuda")
    run_and_check(torch, sc, x["q"], x["k"], x["v"], dtype, k_len=lens, key_mask=mask, strides=strides + [out.stride()[:3]],
                  out=out)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["all", "mask"])
@pytest.mark.parametrize("axis", [0, 1, 2])
def test_shared_queries_in_paired_tiles(sc, axis, kind):
    """Queries that the batch, the tokens or the heads share, more row tiles than SMs."""
    import torch
    N, Tq, Tk, H, D = 11, 300, 700, 6, 64
    size = [N, Tq, H]
    size[axis] = 1
    q = make(torch, BF16, *size, D, seed=115, gain=2.0).expand(N, Tq, H, D)
    k, v = make(torch, BF16, N, Tk, H, D, seed=116), make(torch, BF16, N, Tk, H, D, seed=117)
    mask = (np.random.default_rng(118).random((N, Tk)) < 0.4).astype(np.uint8) if kind == "mask" else None
    out = torch.full((N, Tq, H, D), math.nan, dtype=q.dtype, device="cuda")
    run_and_check(torch, sc, q, k, v, BF16, key_mask=mask, strides=[t.stride()[:3] for t in (q, k, v, out)], out=out)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Tq,Hq,Hkv", [(1, 4, 1), (33, 3, 3)])
def test_offsets_beyond_32_bits(sc, dtype, Tq, Hq, Hkv):
    """Keys and values of more than 2^31 elements; the valid states are the last ones."""
    import torch
    D = 128
    Tk = (2 ** 31) // (Hkv * D) + 4099
    k = torch.empty(1, Tk, Hkv, D, dtype=torch.bfloat16 if dtype == BF16 else torch.float32, device="cuda")
    v = torch.empty_like(k)
    q = make(torch, dtype, 1, Tq, Hq, D, seed=16)
    tail = 4000
    k[:, -tail:] = make(torch, dtype, 1, tail, Hkv, D, seed=17)
    v[:, -tail:] = make(torch, dtype, 1, tail, Hkv, D, seed=18)
    mask = torch.zeros(1, Tk, dtype=torch.uint8, device="cuda")
    mask[:, -tail:] = 1
    out = torch.empty_like(q)
    sc.check(sc.cross_attention_fwd(q, k, v, out, 1, Tq, Tk, Hq, Hkv, D, D ** -0.5, dtype, key_mask=mask))
    sc.check(sc.sc_last_device_status())
    o, z, wabs, mag = ref.attention(f64(q), f64(k[:, -tail:]), f64(v[:, -tail:]), D ** -0.5)
    assert (np.abs(f64(out) - o) <= ref.out_bound(o, wabs, mag, D, Tk, dtype == BF16)).all()
    del k, v


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Tq", [1, 16, 150])
def test_other_stream_and_repeatable(sc, dtype, Tq):
    """A stream of the caller's; the same bits each time, on any stream and from a CUDA graph."""
    import torch
    N, Tk, Hq, Hkv, D = 1, 30000, 4, 2, 64
    q = make(torch, dtype, N, Tq, Hq, D, seed=19, gain=2.0)
    k, v = make(torch, dtype, N, Tk, Hkv, D, seed=20), make(torch, dtype, N, Tk, Hkv, D, seed=21)
    s = torch.cuda.Stream()
    first, lse1 = run_and_check(torch, sc, q, k, v, dtype, stream=s)
    second, lse2 = run_and_check(torch, sc, q, k, v, dtype)
    assert torch.equal(first, second) and torch.equal(lse1, lse2)
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sc.check(sc.cross_attention_fwd(q, k, v, out, N, Tq, Tk, Hq, Hkv, D, D ** -0.5, dtype))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    q.copy_(q * 0.5)
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out, first)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(9, 1, 700, 2, 2, 64), (2, 3, 3000, 8, 2, 128), (1, 16, 5000, 2, 2, 64), (4, 50, 900, 4, 2, 64),
                                   (2, 300, 700, 2, 2, 128)])
def test_same_bits_every_time(sc, shape, dtype):
    """Many calls one after the other, lengths and masks among them: no CTA, warp or copy may be late or early."""
    import torch
    N, Tq, Tk, Hq, Hkv, D = shape
    q = make(torch, dtype, N, Tq, Hq, D, seed=30, gain=2.0)
    k, v = make(torch, dtype, N, Tk, Hkv, D, seed=31), make(torch, dtype, N, Tk, Hkv, D, seed=32)
    lens = torch.tensor([Tk - 37 * i for i in range(N)], dtype=torch.int32).cuda()
    mask = (torch.rand(N, Tk, generator=torch.Generator().manual_seed(33)) < 0.6).to(torch.uint8).cuda()
    for kw in (dict(), dict(k_len=lens), dict(key_mask=mask)):
        outs = [torch.full_like(q, float("nan")) for _ in range(60)]
        for o in outs:
            sc.check(sc.cross_attention_fwd(q, k, v, o, N, Tq, Tk, Hq, Hkv, D, D ** -0.5, dtype, **kw))
        sc.check(sc.sc_last_device_status())
        assert torch.isfinite(outs[0]).all()
        for i, o in enumerate(outs):
            assert torch.equal(o, outs[0]), f"call {i} differs"


@pytest.mark.gpu
def test_calls_on_several_streams_at_once(sc):
    """Every kernel on streams of its own, side by side: workspaces, tensor memory and launch caches are not shared."""
    import torch
    cases = []
    for i, (dtype, N, Tq, Tk, Hq, Hkv, D) in enumerate([
            (BF16, 2, 300, 5000, 8, 4, 64), (F32, 2, 200, 3000, 4, 2, 64), (BF16, 4, 1, 9000, 8, 2, 128), (F32, 3, 2, 8000, 2, 2, 64),
            (BF16, 1, 40, 40000, 2, 2, 64), (F32, 2, 9, 4000, 4, 4, 128), (BF16, 3, 200, 900, 8, 8, 128), (F32, 1, 150, 6000, 2, 2, 96)]):
        q = make(torch, dtype, N, Tq, Hq, D, seed=50 + i, gain=2.0)
        k, v = make(torch, dtype, N, Tk, Hkv, D, seed=60 + i), make(torch, dtype, N, Tk, Hkv, D, seed=70 + i)
        want = torch.empty_like(q)
        call = (N, Tq, Tk, Hq, Hkv, D, D ** -0.5, dtype)
        sc.check(sc.cross_attention_fwd(q, k, v, want, *call))
        cases.append((q, k, v, want, call, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(6):
        for q, k, v, want, call, s in cases:
            out = torch.empty_like(q)
            sc.check(sc.cross_attention_fwd(q, k, v, out, *call, stream=s))
            outs.append((out, want))
    torch.cuda.synchronize()
    sc.check(sc.sc_last_device_status())
    for out, want in outs:
        assert torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("Tq", [1, 140])
def test_nan_in_a_valid_state_is_not_hidden(sc, Tq):
    import torch
    q, k, v = (make(torch, BF16, 1, t, 1, 64, seed=22 + i) for i, t in enumerate((Tq, 500, 500)))
    k[0, 300] = float("nan")
    out = torch.zeros_like(q)
    sc.check(sc.cross_attention_fwd(q, k, v, out, 1, Tq, 500, 1, 1, 64, 0.125, BF16))
    assert torch.isnan(out).all()


# (N, Tq, Tk, Hq, Hkv, D): 1, 3, 8, 16, 40 rows a key head on the kernels for few rows, 40 and 120 on the tensor cores
ROWS = [(1, 1, 500, 4, 4, 64), (2, 3, 700, 2, 2, 64), (2, 2, 500, 8, 2, 64), (1, 16, 900, 2, 2, 128), (1, 40, 600, 4, 4, 64),
        (1, 40, 6000, 4, 4, 64), (2, 40, 3000, 6, 2, 128)]


def check_close(torch, got, lse, q, k, v, dtype, skip=None, valid=None):
    """Against the 64-bit form at its bounds, but for the elements where skip holds."""
    D, Tk = q.shape[3], k.shape[1]
    o, z, wabs, mag = ref.attention(f64(q), f64(k), f64(v), D ** -0.5, valid)
    ok = np.abs(f64(got) - o) <= ref.out_bound(o, wabs, mag, D, Tk, dtype == BF16)
    assert (ok if skip is None else ok | skip).all()
    zok = np.abs(f64(lse) - z) <= ref.lse_bound(z, mag, D, Tk)
    assert (zok if skip is None else zok | skip.any(axis=3).transpose(0, 2, 1)).all()


def call(torch, sc, q, k, v, dtype):
    N, Tq, Hq, D = q.shape
    out, lse = torch.zeros_like(q), torch.zeros(N, Hq, Tq, device="cuda")
    sc.check(sc.cross_attention_fwd(q, k, v, out, N, Tq, k.shape[1], Hq, k.shape[2], D, D ** -0.5, dtype, lse=lse))
    sc.check(sc.sc_last_device_status())
    return out, lse


@pytest.mark.gpu
@pytest.mark.parametrize("shape", ROWS)
def test_largest_fp32_values(sc, shape):
    """A value, and a key where its queries are 0, above bf16's largest: finite results, as accurate as any."""
    import torch
    N, Tq, Tk, Hq, Hkv, D = shape
    q = make(torch, F32, N, Tq, Hq, D, seed=90)
    k, v = make(torch, F32, N, Tk, Hkv, D, seed=91), make(torch, F32, N, Tk, Hkv, D, seed=92)
    q[..., 2] = 0
    k[:, 301, :, 2] = 3.4e38
    v[:, 77, 0, 7] = 3.4e38
    v[:, 78, -1, D - 1] = -3.402e38
    out, lse = call(torch, sc, q, k, v, F32)
    check_close(torch, out, lse, q, k, v, F32)


@pytest.mark.gpu
@pytest.mark.parametrize("exponent", [-100, -112, -126])
@pytest.mark.parametrize("shape", ROWS)
def test_smallest_fp32_values(sc, shape, exponent):
    """Values under 2^-110: their last bf16 planes are subnormal, an element keeps 2^-134 (half of the least of them);
    the weights add up to 1 and their fp32 sums round by 2^-150 a term."""
    import torch
    N, Tq, Tk, Hq, Hkv, D = shape
    q = make(torch, F32, N, Tq, Hq, D, seed=105)
    k, v = make(torch, F32, N, Tk, Hkv, D, seed=106), make(torch, F32, N, Tk, Hkv, D, seed=107, gain=2.0 ** exponent)
    out, lse = call(torch, sc, q, k, v, F32)
    o, z, wabs, mag = ref.attention(f64(q), f64(k), f64(v), D ** -0.5)
    bound = ref.out_bound(o, wabs, mag, D, Tk, False) - 1e-30 + 2.0 ** -134 + Tk * 2.0 ** -150
    assert (np.abs(f64(out) - o) <= bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", ROWS)
def test_infinite_values(sc, shape, dtype):
    """An infinity in a valid state's value: its column is that infinity, and no other is touched."""
    import torch
    N, Tq, Tk, Hq, Hkv, D = shape
    q = make(torch, dtype, N, Tq, Hq, D, seed=93)
    k, v = make(torch, dtype, N, Tk, Hkv, D, seed=94), make(torch, dtype, N, Tk, Hkv, D, seed=95)
    plain = v.clone()
    v[0, 77, 0, 5] = math.inf
    v[0, 411, -1, 9] = -math.inf
    out, lse = call(torch, sc, q, k, v, dtype)
    G = Hq // Hkv
    assert (out[0, :, :G, 5] == math.inf).all() and (out[0, :, -G:, 9] == -math.inf).all()
    skip = np.zeros(out.shape, bool)
    skip[0, :, :G, 5] = skip[0, :, -G:, 9] = True
    o, z, wabs, mag = ref.attention(f64(q), f64(k), f64(plain), D ** -0.5)
    assert (np.abs(np.where(skip, 0, f64(out)) - np.where(skip, 0, o)) <=
            ref.out_bound(o, wabs, mag, D, Tk, dtype == BF16)).all()
    assert (np.abs(f64(lse) - z) <= ref.lse_bound(z, mag, D, Tk)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", ROWS)
def test_infinite_key(sc, shape, dtype):
    """A valid state whose score is -infinity has weight 0: the results are those without it."""
    import torch
    N, Tq, Tk, Hq, Hkv, D = shape
    q = make(torch, dtype, N, Tq, Hq, D, seed=96)
    k, v = make(torch, dtype, N, Tk, Hkv, D, seed=97), make(torch, dtype, N, Tk, Hkv, D, seed=98)
    q[..., 3] = q[..., 3].abs() + 0.125
    k[:, 200, :, 3] = -math.inf
    out, lse = call(torch, sc, q, k, v, dtype)
    valid = np.ones((N, Tk), bool)
    valid[:, 200] = False
    check_close(torch, out, lse, q, torch.nan_to_num(k, neginf=0.0), v, dtype, valid=valid)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", ROWS)
def test_every_score_minus_infinity(sc, shape, dtype):
    """As without a valid state."""
    import torch
    N, Tq, Tk, Hq, Hkv, D = shape
    q = make(torch, dtype, N, Tq, Hq, D, seed=108)
    k, v = make(torch, dtype, N, Tk, Hkv, D, seed=109), make(torch, dtype, N, Tk, Hkv, D, seed=110)
    q[..., 3] = q[..., 3].abs() + 0.125
    k[..., 3] = -math.inf
    out, lse = call(torch, sc, q, k, v, dtype)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", ROWS)
def test_infinite_query(sc, shape, dtype):
    """An infinity in a query: scores of both infinities, NaN in that row and no other."""
    import torch
    N, Tq, Tk, Hq, Hkv, D = shape
    q = make(torch, dtype, N, Tq, Hq, D, seed=99)
    k, v = make(torch, dtype, N, Tk, Hkv, D, seed=100), make(torch, dtype, N, Tk, Hkv, D, seed=101)
    plain = q.clone()
    q[0, -1, 0, 4] = math.inf
    out, lse = call(torch, sc, q, k, v, dtype)
    assert torch.isnan(out[0, -1, 0]).all() and torch.isnan(lse[0, 0, -1])
    skip = np.zeros(out.shape, bool)
    skip[0, -1, 0] = True
    check_close(torch, out, lse, plain, k, v, dtype, skip=skip)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", ROWS)
def test_nan_in_a_valid_fp32_state_is_not_hidden(sc, shape):
    import torch
    N, Tq, Tk, Hq, Hkv, D = shape
    q = make(torch, F32, N, Tq, Hq, D, seed=102)
    k, v = make(torch, F32, N, Tk, Hkv, D, seed=103), make(torch, F32, N, Tk, Hkv, D, seed=104)
    k[:, 300, :, 1] = math.nan
    out, lse = call(torch, sc, q, k, v, F32)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    k[:, 300, :, 1] = 0
    v[:, 300, :, 1] = math.nan
    out, lse = call(torch, sc, q, k, v, F32)
    assert torch.isnan(out[..., 1]).all() and torch.isfinite(out[..., 2:]).all() and torch.isfinite(lse).all()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 140, 1000, 2, 2, 64), (11, 300, 700, 6, 6, 64), (1, 40, 20000, 2, 2, 128)])
@pytest.mark.parametrize("drop_copy", [0, 1, 3])
def test_expired_wait_is_reported(sc, shape, drop_copy):
    """A copy that never comes: its waits run out, the status says so, and the next call is right."""
    import torch
    N, Tq, Tk, Hq, Hkv, D = shape
    q = make(torch, BF16, N, Tq, Hq, D, seed=40)
    k, v = make(torch, BF16, N, Tk, Hkv, D, seed=41), make(torch, BF16, N, Tk, Hkv, D, seed=42)
    out = torch.empty_like(q)
    sc.check(sc.sc_last_device_status())
    sc.check(sc.sc_test_attn_wait_expiry(q, k, v, out, N, Tq, Tk, Hq, Hkv, D, drop_copy, 300))
    assert sc.sc_last_device_status() == scl.SC_ERR_DEVICE_TIMEOUT
    assert sc.sc_last_device_status() == scl.SC_OK
    run_and_check(torch, sc, q, k, v, BF16)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,shape", [
    (BF16, (2, 140, 2500, 2, 2, 128)), (BF16, (11, 300, 1300, 6, 6, 128)), (BF16, (2, 140, 3300, 2, 2, 64)),
    (BF16, (11, 300, 2100, 6, 6, 40)), (F32, (2, 140, 1300, 4, 2, 128)), (F32, (2, 140, 1300, 2, 2, 64)),
    (F32, (11, 300, 900, 6, 6, 64))])
@pytest.mark.parametrize("kind", ["lengths", "mask"])
def test_late_clearing_warps(sc, shape, dtype, kind):
    """The warps that clear value rows far behind the products: no slot of the ring is refilled before they have
    seen its copy, so the result is the same, and no wait runs out."""
    import torch
    N, Tq, Tk, Hq, Hkv, D = shape
    q = make(torch, dtype, N, Tq, Hq, D, seed=80, gain=0.3)
    k, v = make(torch, dtype, N, Tk, Hkv, D, seed=81), make(torch, dtype, N, Tk, Hkv, D, seed=82)
    lens = mask = None
    if kind == "lengths":
        lens = torch.tensor([Tk - 3 - 90 * (n % 3) for n in range(N)], dtype=torch.int32).cuda()
    else:
        mask = (torch.rand(N, Tk, generator=torch.Generator().manual_seed(83)) < 0.5).to(torch.uint8).cuda()
    valid = torch.as_tensor(valid_of(N, Tk, None if lens is None else lens.cpu().numpy(),
                                     None if mask is None else mask.cpu().numpy())).cuda()
    k[~valid] = float("nan")
    v[~valid] = float("inf")
    outs = []
    for delay in (0, 20):
        outs.append(torch.full_like(q, float("nan")))
        sc.check(sc.sc_test_attn_slow_clear(q, k, v, outs[-1], lens, mask, N, Tq, Tk, Hq, Hkv, D, dtype, delay))
        sc.check(sc.sc_last_device_status(), "device status")
    o, z, wabs, mag = ref.attention(f64(q), f64(k), f64(v), 1.0, valid.cpu().numpy())
    assert (np.abs(f64(outs[0]) - o) <= ref.out_bound(o, wabs, mag, D, Tk, dtype == BF16)).all()
    assert torch.equal(outs[0], outs[1])


A, B, C, O = 1 << 30, 1 << 32, 1 << 34, 1 << 36   # fake, aligned, far apart: never dereferenced


@pytest.mark.parametrize("change,expect", [
    (dict(q=None), scl.SC_ERR_NULL),
    (dict(k=None), scl.SC_ERR_NULL),
    (dict(v=None), scl.SC_ERR_NULL),
    (dict(out=None), scl.SC_ERR_NULL),
    (dict(N=0), scl.SC_ERR_SHAPE),
    (dict(Tq=0), scl.SC_ERR_SHAPE),
    (dict(Tk=-1), scl.SC_ERR_SHAPE),
    (dict(Hkv=0), scl.SC_ERR_SHAPE),
    (dict(D=0), scl.SC_ERR_SHAPE),
    (dict(N=1 << 30, Tq=1 << 30), scl.SC_ERR_SHAPE),
    (dict(Tk=(1 << 30) + 1), scl.SC_ERR_SHAPE),
    (dict(Hkv=3), scl.SC_ERR_UNSUPPORTED),
    (dict(D=12), scl.SC_ERR_UNSUPPORTED),
    (dict(D=136), scl.SC_ERR_UNSUPPORTED),
    (dict(dtype=2), scl.SC_ERR_UNSUPPORTED),
    (dict(scale=0.0), scl.SC_ERR_UNSUPPORTED),
    (dict(scale=-1.0), scl.SC_ERR_UNSUPPORTED),
    (dict(scale=math.inf), scl.SC_ERR_UNSUPPORTED),
    (dict(scale=math.nan), scl.SC_ERR_UNSUPPORTED),
    (dict(q=A + 8), scl.SC_ERR_ALIGN),
    (dict(out=O + 2), scl.SC_ERR_ALIGN),
    (dict(lse=(1 << 38) + 2), scl.SC_ERR_ALIGN),
    (dict(k_len=(1 << 38) + 2), scl.SC_ERR_ALIGN),
    (dict(strides=[(2048, 256, 64), (2560, 130, 64), (2560, 128, 64), (2048, 256, 64)]), scl.SC_ERR_ALIGN),
    (dict(strides=[(2048, 256, 64), (2560, 128, 64), (2560, 128, 64), (-2048, 256, 64)]), scl.SC_ERR_SHAPE),
    (dict(strides=[(1 << 60, 256, 64), (2560, 128, 64), (2560, 128, 64), (2048, 256, 64)]), scl.SC_ERR_SHAPE),
    (dict(strides=[(2048, 256, 64), (2560, 128, 64), (2560, 128, 64), (2048, 256, 32)]), scl.SC_ERR_ALIAS),
    (dict(strides=[(2048, 256, 64), (2560, 128, 64), (2560, 128, 64), (0, 256, 64)]), scl.SC_ERR_ALIAS),
    (dict(out=A), scl.SC_ERR_ALIAS),
    (dict(out=B + 64), scl.SC_ERR_ALIAS),
    (dict(out=C + 128), scl.SC_ERR_ALIAS),
    (dict(lse=O + 64), scl.SC_ERR_ALIAS),
    (dict(lse=A + 64), scl.SC_ERR_ALIAS),
    (dict(k_len=O + 64), scl.SC_ERR_ALIAS),
    (dict(key_mask=O + 64), scl.SC_ERR_ALIAS),
    (dict(lse=1 << 38, key_mask=(1 << 38) + 3), scl.SC_ERR_ALIAS),
])
def test_refusals(change, expect):
    a = dict(q=A, k=B, v=C, out=O, N=2, Tq=8, Tk=20, Hq=4, Hkv=2, D=64, scale=0.125, dtype=BF16, k_len=None,
             key_mask=None, lse=None, strides=None)
    a.update(change)
    rc = scl.cross_attention_fwd(a["q"], a["k"], a["v"], a["out"], a["N"], a["Tq"], a["Tk"], a["Hq"], a["Hkv"], a["D"],
                                 a["scale"], a["dtype"], k_len=a["k_len"], key_mask=a["key_mask"], lse=a["lse"],
                                 strides=a["strides"], stream=0)
    assert rc == expect, scl.sc_status_string(rc)


def test_wait_expiry_hook_refusals():
    assert scl.sc_test_attn_wait_expiry(None, B, C, O, 1, 8, 20, 4, 2, 64, 0, 10, stream=0) == scl.SC_ERR_NULL
    assert scl.sc_test_attn_wait_expiry(A, B, C, O, 1, 8, 20, 4, 2, 64, -1, 10, stream=0) == scl.SC_ERR_SHAPE
    assert scl.sc_test_attn_wait_expiry(A, B, C, O, 1, 8, 20, 4, 2, 64, 0, 0, stream=0) == scl.SC_ERR_SHAPE
    assert scl.sc_test_attn_wait_expiry(A, B, C, O, 1, 8, 20, 4, 3, 64, 0, 10, stream=0) == scl.SC_ERR_UNSUPPORTED


def test_slow_clear_hook_refusals():
    L = 1 << 38
    assert scl.sc_test_attn_slow_clear(None, B, C, O, L, None, 1, 8, 20, 4, 2, 64, BF16, 10, stream=0) == scl.SC_ERR_NULL
    assert scl.sc_test_attn_slow_clear(A, B, C, O, None, None, 1, 8, 20, 4, 2, 64, BF16, 10, stream=0) == scl.SC_ERR_NULL
    assert scl.sc_test_attn_slow_clear(A, B, C, O, L, None, 1, 8, 20, 4, 2, 64, BF16, -1, stream=0) == scl.SC_ERR_SHAPE
    assert scl.sc_test_attn_slow_clear(A, B, C, O, L, None, 1, 8, 20, 4, 2, 64, BF16, 1001, stream=0) == scl.SC_ERR_SHAPE
    assert scl.sc_test_attn_slow_clear(A, B, C, O, L, None, 1, 8, 20, 4, 3, 64, BF16, 10, stream=0) == scl.SC_ERR_UNSUPPORTED
