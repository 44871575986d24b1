"""cross_attention_q8_fwd against the plain 64-bit form, and its refusals.

The bound: codes are exact, so a score has the error of an fp32 dot product of D
terms (fp32 queries in two planes of fp16: 2^-22 of each product more), the
scales' and the exponential's; bf16 tensors round a weight (with more than 16 rows a
key head, a weight times its scale) to fp16 (2^-11), and the output once; fp32 weights
have two planes of fp16 (2^-22) or three of bf16 (2^-24).  A weight enters the MMAs as a
fp16 number in which the largest of its group of 16 or 32 states is 2^14; fp16's
spacing is never under 2^-24, so a weight that is small in its group is off by up to
2^-25 / 2^14 = 2^-39 of that largest, whatever its own size.  That is seen where
the group's larger weights meet codes of 0: the bound has 2^-39 of the row's largest
weight times sum_j |v_j|.  With more than 16 rows and bf16 tensors it is a weight times
its scale, of which the row's largest is 2^6 or more: the bound has 2^-25 / 2^6 = 2^-31 of
that largest times the sum of the codes' sizes."""
import math

import numpy as np
import pytest

import layer_ref as ref
import stencil_conv2d_fwd_gb300 as scl

BF16, F32, I8, E4M3 = scl.SC_BF16, scl.SC_F32, scl.SC_CODE_I8, scl.SC_CODE_E4M3


def make(torch, dtype, code, N, Tq, Tk, Hq, Hkv, D, block, seed=0):
    """Queries, and codes with scales that differ from block to block by up to 2^6."""
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(N, Tq, Hq, D, generator=g) * 2).to(torch.bfloat16 if dtype == BF16 else torch.float32).cuda()
    out = [q]
    top = 448.0 if code == E4M3 else 127.0
    for _ in range(2):
        y = (torch.randn(N, Tk, Hkv, D, generator=g) * top / 3.5).clamp(-top, top)
        c = y.to(torch.float8_e4m3fn).view(torch.uint8) if code == E4M3 else y.round().to(torch.int8).view(torch.uint8)
        s = 3.5 / top * 2.0 ** (torch.rand(N, Hkv, -(-Tk // block), generator=g) * 6 - 5)
        out += [c.cuda(), s.cuda()]
    return out


def values(torch, c, code):
    return c.view(torch.float8_e4m3fn if code == E4M3 else torch.int8).double()


def bounds(out, lse, wabs, mag, D, Tk, bf16, largest):
    """largest: what a spacing of fp16 leaves, relative to a row's largest weight, [N][Tq][Hq][D]."""
    ds = ref.U * (6 * math.sqrt(D) + 16) * mag + 2.0 ** -21 + (0.0 if bf16 else 2.0 ** -22 * mag)
    # |lse| log2 e and m are rounded where they are subtracted: part of the score's own size
    b = wabs * (2 * ds.transpose(1, 2)[..., None] + (6 * math.sqrt(Tk) + 16) * ref.U + (2.0 ** -11 if bf16 else 2.0 ** -22)) + 1e-30
    b = b + largest
    if bf16:
        b = b + ref.UB * out.abs()
    z = ds + (6 * math.sqrt(Tk) + 16) * ref.U + 4 * ref.U * lse.abs().nan_to_num(posinf=0.0)
    return b, z


def run_and_check(torch, sc, data, dtype, code, block, k_len=None, key_mask=None, strides=None, out=None, stream=None,
                  plain=None, scale=None):
    q, k, ks, v, vs = data
    pk, pv = plain if plain is not None else (k, v)
    N, Tq, Hq, D = q.shape
    Tk, Hkv = pk.shape[1:3]
    scale = D ** -0.5 if scale is None else scale
    if out is None:
        out = torch.full((N, Tq, Hq, D), math.nan, dtype=q.dtype, device="cuda")
    lse = torch.full((N, Hq, Tq), math.nan, device="cuda")
    kl = None if k_len is None else torch.tensor(k_len, dtype=torch.int32, device="cuda")
    km = None if key_mask is None else torch.as_tensor(np.asarray(key_mask, np.uint8)).cuda()
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    sc.check(sc.cross_attention_q8_fwd(q, k, ks, v, vs, out, N, Tq, Tk, Hq, Hkv, D, scale, block, code, dtype, k_len=kl,
                                       key_mask=km, lse=lse, strides=strides, stream=stream), "cross_attention_q8_fwd")
    sc.check(sc.sc_last_device_status(stream), "device status")
    valid = torch.ones(N, Tk, dtype=torch.bool, device="cuda")
    if kl is not None:
        valid &= torch.arange(Tk, device="cuda")[None] < kl[:, None]
    if km is not None:
        valid &= km != 0
    kk, vv = (ref.dequantize(values(torch, c, code), s, block) for c, s in ((pk, ks), (pv, vs)))
    o, z, wabs, mag = ref.attention(q.double(), kk, vv, scale, valid)
    G = Hq // Hkv
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    ok = valid[:, :, None, None]
    if dtype == BF16 and Tq * G > 16:
        s = scale * (q.double().transpose(1, 2) @ torch.where(ok, kk, zero).repeat_interleave(G, dim=2).permute(0, 2, 3, 1))
        p = torch.exp(s - torch.where(z.isinf(), zero, z)[..., None]) * valid[:, None, None, :]
        size = torch.where(ok[..., 0], vs.double().abs().transpose(1, 2).repeat_interleave(block, dim=1)[:, :Tk], zero)
        most = (p * size.repeat_interleave(G, dim=2).transpose(1, 2)[:, :, None, :]).amax(dim=-1)            # [N][Hq][Tq]
        codes = torch.where(ok, values(torch, pv, code).abs(), zero).sum(dim=1).repeat_interleave(G, dim=1)     # [N][Hq][D]
        small = 2.0 ** -31 * (most[..., None] * codes[:, :, None, :]).transpose(1, 2)
    else:   # the weights sum to 1: none is above it
        small = 2.0 ** -39 * torch.where(ok, vv.abs(), zero).sum(dim=1).repeat_interleave(G, dim=1)[:, None]
    b, zb = bounds(o, z, wabs, mag, D, Tk, dtype == BF16, small)
    assert torch.isfinite(out.float()).all()
    err = (out.double() - o).abs()
    assert (err <= b).all(), f"out: worst {(err / b).max().item():.2f} of its bound"
    assert torch.equal(lse.isneginf(), z.isneginf())
    zerr = (lse.double() - z).abs().nan_to_num()
    assert (zerr <= zb).all(), f"lse: worst {(zerr / zb).max().item():.2f} of its bound"
    return out, lse


# (N, Tq, Tk, Hq, Hkv, D, block): one token to many; lengths around tiles; odd widths; shared heads
SHAPES = [
    (1, 1, 1, 1, 1, 16, 16),
    (1, 1, 960, 4, 4, 64, 64),
    (2, 1, 257, 4, 2, 32, 16),
    (3, 1, 1000, 5, 1, 64, 128),
    (1, 1, 20000, 4, 1, 64, 32),
    (1, 1, 20000, 8, 1, 128, 64),
    (2, 1, 333, 16, 2, 96, 16),
    (2, 2, 129, 3, 3, 48, 32),
    (2, 3, 700, 4, 4, 32, 64),
    (1, 5, 128, 6, 2, 128, 128),
    (1, 9, 130, 2, 1, 80, 16),
    (2, 16, 640, 8, 2, 64, 32),
    (1, 16, 9000, 2, 1, 128, 16),
    (3, 77, 391, 4, 4, 64, 64),
    (1, 100, 1, 2, 2, 48, 16),
    (1, 127, 127, 3, 1, 128, 128),
    (1, 128, 128, 1, 1, 64, 16),
    (1, 129, 129, 2, 2, 16, 32),
    (2, 255, 513, 2, 1, 80, 64),
    (1, 257, 385, 5, 1, 112, 16),
    (1, 300, 1300, 4, 4, 128, 32),
    (1, 500, 900, 3, 3, 64, 128),
    (1, 40, 20000, 2, 2, 80, 64),
    (1, 1, 300, 150, 1, 32, 16),
    (1, 10, 2000, 150, 1, 64, 64),
    (3, 700, 500, 8, 2, 64, 32),
    (2, 1000, 260, 16, 16, 128, 128),
]


@pytest.mark.gpu
@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(sc, shape, dtype, code):
    import torch
    run_and_check(torch, sc, make(torch, dtype, code, *shape, seed=1), dtype, code, shape[-1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,code,block", [(F32, I8, 64), (BF16, I8, 16), (BF16, E4M3, 128), (F32, E4M3, 32)])
@pytest.mark.parametrize("Tq,G", [(1, 1), (1, 4), (3, 3), (77, 1), (70, 4), (300, 2)])
@pytest.mark.parametrize("Tk", [100, 128, 700, 4500])
def test_lengths(sc, dtype, code, block, Tq, G, Tk):
    """Lengths of zero, one, around a tile's end, all of Tk, above it and below zero; behind them NaN codes, and NaN
    scales of blocks that no valid state is in."""
    import torch
    lens = [0, 1, 63, 64, min(Tk, 127), Tk - 1, Tk, Tk + 9, -3]
    N, Hkv, D = len(lens), 2, 64
    q, k, ks, v, vs = make(torch, dtype, code, N, Tq, Tk, Hkv * G, Hkv, D, block, seed=2)
    for n, L in enumerate(lens):
        L = max(0, L)
        k[n, L:], v[n, L:] = (0x7f, 0xff) if code == E4M3 else (0x80, 0x80)
        ks[n, :, -(-L // block):], vs[n, :, -(-L // block):] = math.nan, math.inf
    out, lse = run_and_check(torch, sc, (q, k, ks, v, vs), dtype, code, block, k_len=lens, plain=(k.clone(), v.clone()))
    assert (out[0] == 0).all() and (out[-1] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,code,block", [(F32, I8, 32), (BF16, I8, 128), (BF16, E4M3, 16), (F32, E4M3, 64)])
@pytest.mark.parametrize("Tq,G,D", [(1, 1, 64), (1, 4, 128), (2, 6, 32), (77, 1, 64), (40, 3, 128), (290, 1, 80)])
def test_masks(sc, dtype, code, block, Tq, G, D):
    """Masks that leave nothing, one state, every other one, a padded map, whole tiles empty; NaN codes in the masked
    places, NaN scales where a whole block is masked; a length on top."""
    import torch
    h, w = 25, 31
    Tk, N, Hkv = h * w, 6, 2
    rng = np.random.default_rng(7)
    mask = np.zeros((N, Tk), np.uint8)
    mask[1, 700] = 1
    mask[2, ::2] = 255
    m = np.zeros((h, w), np.uint8)
    m[:17, :22] = 1
    mask[3] = m.reshape(-1)
    mask[4, 128:140], mask[4, 600:] = 1, 1
    mask[5] = rng.integers(0, 2, Tk)
    q, k, ks, v, vs = make(torch, dtype, code, N, Tq, Tk, Hkv * G, Hkv, D, block, seed=3)
    on = torch.as_tensor(mask).cuda() != 0
    if code == E4M3:
        k[~on], v[~on] = 0x7f, 0xff
    blocks = torch.zeros(N, -(-Tk // block) * block, dtype=torch.bool, device="cuda")
    blocks[:, :Tk] = on
    empty = ~blocks.view(N, -1, block).any(dim=2)
    ks.transpose(1, 2)[empty], vs.transpose(1, 2)[empty] = math.nan, math.nan
    data = (q, k, ks, v, vs)
    out, _ = run_and_check(torch, sc, data, dtype, code, block, key_mask=mask)
    assert (out[0] == 0).all()
    run_and_check(torch, sc, data, dtype, code, block, key_mask=mask, k_len=[Tk, 700, 333, 400, 130, 64])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,code", [(F32, I8), (BF16, E4M3)])
@pytest.mark.parametrize("Tq", [1, 5, 60, 400])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_running_maximum(sc, dtype, code, Tq, order):
    """Scores that rise or fall over the keys by more than fp32's exponent."""
    import torch
    N, Tk, H, D, block = 1, 2000, 2, 64, 32
    q, k, ks, v, vs = make(torch, dtype, code, N, Tq, Tk, H, H, D, block, seed=4)
    k[:] = 0
    k[..., 0] = 0x70 if code == E4M3 else 100   # 128 or 100
    q[..., 0] = 4.0
    ramp = torch.linspace(-30, 30, ks.shape[2], device="cuda") if order == "rising" else torch.linspace(30, -30, ks.shape[2], device="cuda")
    ks[:] = ramp.abs() / 100 + 1e-3
    k[..., 0] = torch.where(ramp.repeat_interleave(block)[:Tk].view(1, Tk, 1) < 0, (0xf0 if code == E4M3 else 0x9c), k[..., 0].int()).to(torch.uint8)
    run_and_check(torch, sc, (q, k, ks, v, vs), dtype, code, block, scale=1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Tq", [1, 4, 90])
def test_scales_and_queries_far_apart(sc, dtype, Tq):
    """Blocks whose scales differ by 2^40, a zero scale, rows of queries from 2^-60 to 2^20 and of zeros."""
    import torch
    N, Tk, H, D, block = 1, 640, 2, 64, 16
    q, k, ks, v, vs = make(torch, dtype, I8, N, Tq, Tk, H, H, D, block, seed=5)
    e = torch.arange(vs.shape[2], device="cuda") % 41
    vs *= 2.0 ** (e - 20.0)
    vs[..., 3], ks[..., 5] = 0.0, 0.0
    ks[..., 8::7] *= -1   # no call writes such scales, but they have a meaning
    for t in range(Tq):
        f = [1.0, 2.0 ** -60, 2.0 ** 20, 0.0][t % 4]
        q[:, t] *= f
    run_and_check(torch, sc, (q, k, ks, v, vs), dtype, I8, block, scale=2.0 ** -18 / 8 if Tq > 2 else 0.125)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,code", [(BF16, I8), (BF16, E4M3), (F32, I8)])
@pytest.mark.parametrize("shape", [(3, 2, 64, 1500), (90, 2, 64, 700), (90, 2, 64, 9000), (40, 2, 128, 2000), (300, 80, 64, 700),
                                   (300, 80, 128, 700)])
@pytest.mark.parametrize("low,high", [(0.0, 2.0 ** 50), (0.0, 2.0 ** 80), (2.0 ** -80, 2.0 ** 60), (2.0 ** -70, 2.0 ** 80)])
def test_value_scales_over_the_documented_range(sc, shape, low, high, dtype, code):
    """Equal scores, value scales from the least (or 0) to the largest: in the first states or the last, in every other
    tile of 128 and in every third (so that each stream of a CTA has both), on few rows, one and two row tiles and split
    keys.  Equal scores make every weight a power of two and their sum exact, so that what is left of lse's error is m ln 2's
    and the logarithm's, numbers below 64: at most 2 ulp, 2^-17, where the bound has (6 sqrt(700) + 16) 2^-24, 1.3 * 2^-17."""
    import torch
    Tq, H, D, Tk = shape
    N, block = 1, 128
    q, k, ks, v, vs = make(torch, dtype, code, N, Tq, Tk, H, H, D, block, seed=14)
    q.zero_()
    b = torch.arange(vs.shape[2], device="cuda")
    n = vs.shape[2]
    for first in (b < n // 2, b >= n // 2, b % 2 == 0, b % 2 == 1, b % 3 == 0, b == n - 1):
        vs[:] = torch.where(first, low, high)
        run_and_check(torch, sc, (q, k, ks, v, vs), dtype, code, block)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,H,Tq", [(BF16, 160, 20), (F32, 160, 20), (BF16, 80, 260)])
def test_long_masked_share(sc, dtype, H, Tq):
    """More key tiles in a CTA's share than it lists (512 of 128 keys), most of them empty; one and two row tiles."""
    import torch
    Tk, D, block = 70000, 16, 128
    data = make(torch, dtype, E4M3, 1, Tq, Tk, H, H, D, block, seed=12)
    mask = np.zeros((1, Tk), np.uint8)
    mask[0, 3:40], mask[0, 40000:40300:3], mask[0, 69990:] = 1, 1, 1
    on = torch.as_tensor(mask).cuda() != 0
    data[1][~on], data[3][~on] = 0x7f, 0xff   # NaN codes where the mask is 0
    run_and_check(torch, sc, data, dtype, E4M3, block, key_mask=mask)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Tq,H,D", [(3, 2, 64), (90, 2, 64), (300, 80, 64), (300, 80, 128)])
@pytest.mark.parametrize("masked", [False, True])
def test_negative_scales(sc, dtype, Tq, H, D, masked):
    """Every other block of keys turned by its scale, under a mask and a length; one and two row tiles a CTA."""
    import torch
    N, Tk, block = 1, 400, 16
    q, k, ks, v, vs = make(torch, dtype, E4M3, N, Tq, Tk, H, H, D, block, seed=11)
    ks[..., 1::2] *= -1
    vs[..., ::3] *= -1
    mask = (np.random.default_rng(1).random((N, Tk)) < 0.7).astype(np.uint8) if masked else None
    run_and_check(torch, sc, (q, k, ks, v, vs), dtype, E4M3, block, key_mask=mask, k_len=[390] if masked else None)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Tq", [1, 6, 150])
def test_strides(sc, dtype, Tq):
    """Codes with gaps, a cache [Tk][2][Hkv][D] of keys and values together, heads before tokens, and a batch that shares
    its states by a stride of 0."""
    import torch
    N, Tk, Hq, Hkv, D, block = 2, 333, 4, 2, 48, 32
    q, k, ks, v, vs = make(torch, dtype, I8, N, Tq, Tk, Hq, Hkv, D, block, seed=6)
    both = torch.full((N, Tk, 2, Hkv, 64), 0x55, dtype=torch.uint8, device="cuda")
    both[:, :, 0, :, :D], both[:, :, 1, :, :D] = k, v
    qt = q.transpose(1, 2).contiguous()
    ot = torch.full_like(qt, math.nan)
    kvs = (Tk * 2 * Hkv * 64, 2 * Hkv * 64, 64)
    qs = (Hq * Tq * D, D, Tq * D)
    out, _ = run_and_check(torch, sc, (q, k, ks, v, vs), dtype, I8, block)
    lse = torch.empty(N, Hq, Tq, device="cuda")
    sc.check(sc.cross_attention_q8_fwd(qt, both, ks, both[0, 0, 1], vs, ot, N, Tq, Tk, Hq, Hkv, D, D ** -0.5, block, I8, dtype,
                                       lse=lse, strides=(qs, kvs, kvs, qs)), "cross_attention_q8_fwd")
    assert torch.equal(ot.transpose(1, 2), out)
    # one sequence's states for all (the scales are of each sequence)
    k[1], v[1], ks[1], vs[1] = k[0], v[0], ks[0], vs[0]
    out, _ = run_and_check(torch, sc, (q, k, ks, v, vs), dtype, I8, block)
    shared = (0, Hkv * D, D)
    packed = (Tq * Hq * D, Hq * D, D)
    o2 = torch.empty_like(out)
    sc.check(sc.cross_attention_q8_fwd(q, k, ks, v, vs, o2, N, Tq, Tk, Hq, Hkv, D, D ** -0.5, block, I8, dtype, lse=lse,
                                       strides=(packed, shared, shared, packed)), "cross_attention_q8_fwd")
    assert torch.equal(o2, out)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Tq", [1, 12, 200])
def test_nan_in_a_valid_state_is_not_hidden(sc, dtype, Tq):
    import torch
    N, Tk, H, D, block = 1, 400, 2, 64, 16
    for what in ("k", "v", "ks", "vs", "q"):
        q, k, ks, v, vs = make(torch, dtype, E4M3, N, Tq, Tk, H, H, D, block, seed=8)
        if what == "q":
            q[0, 0, 1, 5] = math.inf
        elif what in ("ks", "vs"):
            (ks if what == "ks" else vs)[0, 1, 7] = math.nan
        else:
            (k if what == "k" else v)[0, 150, 1, 9] = 0x7f
        out = torch.zeros(N, Tq, H, D, dtype=q.dtype, device="cuda")
        sc.check(sc.cross_attention_q8_fwd(q, k, ks, v, vs, out, N, Tq, Tk, H, H, D, 0.125, block, E4M3, dtype))
        assert torch.isfinite(out[:, :, 0].float()).all()
        if what == "v":
            assert out[:, :, 1, 9].isnan().all() and torch.isfinite(out[:, :, 1, :9].float()).all()
        elif what == "q":
            assert out[:, 0, 1].isnan().all() and torch.isfinite(out[:, 1:].float()).all()
        else:
            assert out[:, :, 1].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(2, 1, 3000, 8, 2, 64, 64), (1, 1, 100000, 4, 1, 128, 32), (2, 300, 900, 4, 2, 64, 128),
                                   (1, 60, 9000, 2, 2, 128, 64)])
def test_streams_graph_and_same_bits(sc, shape, dtype):
    import torch
    N, Tq, Tk, Hq, Hkv, D, block = shape
    q, k, ks, v, vs = make(torch, dtype, I8, *shape, seed=9)
    args = (N, Tq, Tk, Hq, Hkv, D, D ** -0.5, block, I8, dtype)
    first = torch.empty_like(q)
    sc.check(sc.cross_attention_q8_fwd(q, k, ks, v, vs, first, *args))
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(q) for _ in range(9)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        sc.check(sc.cross_attention_q8_fwd(q, k, ks, v, vs, o, *args, stream=streams[i % 3]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    qin, a, b = torch.zeros_like(q), torch.empty_like(q), torch.empty_like(q)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, o in zip(graphs, (a, b)):
        with torch.cuda.graph(graph):
            sc.check(sc.cross_attention_q8_fwd(qin, k, ks, v, vs, o, *args))
    qin.copy_(q)
    torch.cuda.synchronize()
    for graph, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, first) and torch.equal(b, first)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,Tq", [(F32, 1), (BF16, 1), (BF16, 100), (F32, 100)])
def test_offsets_beyond_32_bits(sc, dtype, Tq):
    """States 2^25 bytes apart: the last ones of 200 lie beyond 2^32."""
    import torch
    N, Tk, H, D, block, pitch = 1, 200, 1, 64, 32, 1 << 25
    q, k, ks, v, vs = make(torch, dtype, I8, N, Tq, Tk, H, H, D, block, seed=10)
    buf = torch.empty(pitch * (Tk - 1) + 2 * D, dtype=torch.uint8, device="cuda")
    buf.as_strided((Tk, D), (pitch, 1)).copy_(k[0, :, 0])
    buf.as_strided((Tk, D), (pitch, 1), D).copy_(v[0, :, 0])
    st, packed = (0, pitch, D), (Tq * H * D, H * D, D)
    run_and_check(torch, sc, (q, buf, ks, buf[D:], vs), dtype, I8, block, strides=(packed, st, st, packed), plain=(k, v))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("shape", [(1, 140, 1000, 2, 2, 64, 32), (11, 300, 700, 6, 6, 64, 64), (1, 40, 20000, 2, 2, 128, 128)])
@pytest.mark.parametrize("drop_copy", [0, 1, 5])
def test_expired_wait_is_reported(sc, shape, drop_copy, code, dtype):
    """A copy that never comes: its waits run out, the status says so, and the next call is right."""
    import torch
    data = make(torch, dtype, code, *shape, seed=13)
    q, k, ks, v, vs = data
    sc.check(sc.sc_last_device_status())
    sc.check(sc.sc_test_attn_q8_wait_expiry(q, k, ks, v, vs, torch.empty_like(q), *shape, code, dtype, drop_copy, 300))
    assert sc.sc_last_device_status() == scl.SC_ERR_DEVICE_TIMEOUT
    assert sc.sc_last_device_status() == scl.SC_OK
    run_and_check(torch, sc, data, dtype, code, shape[-1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 140, 1000, 2, 2, 64, 32), (11, 300, 700, 6, 6, 64, 64), (1, 40, 20000, 2, 2, 128, 128)])
def test_waits_that_expire_anywhere(sc, shape, dtype):
    """No copy is left out, but the waits' limit is as short as the waits themselves: each call ends, says so or not, and
    the next ordinary one is right; then the first copy left out with so short a limit."""
    import torch
    data = make(torch, dtype, I8, *shape, seed=16)
    q, k, ks, v, vs = data
    out, seen = torch.empty_like(q), set()
    for drop_copy, limit in [(1 << 30, t) for t in (1, 2, 3, 5, 8, 13, 20, 30) for _ in range(4)] + [(0, 1)]:
        sc.check(sc.sc_test_attn_q8_wait_expiry(q, k, ks, v, vs, out, *shape, I8, dtype, drop_copy, limit))
        torch.cuda.synchronize()
        seen.add(sc.sc_last_device_status())
    assert seen <= {scl.SC_OK, scl.SC_ERR_DEVICE_TIMEOUT} and scl.SC_ERR_DEVICE_TIMEOUT in seen
    run_and_check(torch, sc, data, dtype, I8, shape[-1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("shape", [(1, 1, 40, 1, 1, 16, 16), (3, 1, 3000, 8, 2, 64, 32), (2, 3, 5000, 4, 1, 128, 64),
                                   (1, 1, 60000, 4, 1, 64, 128), (64, 2, 700, 16, 2, 64, 64)])
def test_expired_wait_of_few_rows_is_reported(sc, shape, code, dtype):
    """A step that never comes (the first, a later one), then waits as short as the copies, that run out where they happen
    to: every call ends, the status says so, and the next call is right.  The rings' memory is the sums' at the end, so no
    copy may be on its way there."""
    import torch
    data = make(torch, dtype, code, *shape, seed=15)
    q, k, ks, v, vs = data
    out, seen = torch.empty_like(q), set()
    sc.check(sc.sc_last_device_status())
    for drop_copy, limit in [(0, 300), (0, 1)] + [(1 << 30, t) for t in (1, 1, 2, 2, 4, 8) for _ in range(4)]:
        sc.check(sc.sc_test_attn_q8_rows_wait_expiry(q, k, ks, v, vs, out, *shape, code, dtype, drop_copy, limit))
        torch.cuda.synchronize()
        seen.add(sc.sc_last_device_status())
        assert drop_copy > 0 or sc.SC_OK not in seen
    assert seen <= {scl.SC_OK, scl.SC_ERR_DEVICE_TIMEOUT}
    if shape[2] >= 60000:   # warps with many steps
        sc.check(sc.sc_test_attn_q8_rows_wait_expiry(q, k, ks, v, vs, out, *shape, code, dtype, 1, 300))
        assert sc.sc_last_device_status() == scl.SC_ERR_DEVICE_TIMEOUT
    assert sc.sc_last_device_status() == scl.SC_OK
    run_and_check(torch, sc, data, dtype, code, shape[-1])


def test_rows_wait_expiry_hook_refusals():
    args = (A, B, C, D_, E, G, 2, 4, 40, 2, 2, 32)
    assert scl.sc_test_attn_q8_rows_wait_expiry(None, *args[1:], 16, I8, F32, 0, 10, stream=0) == scl.SC_ERR_NULL
    assert scl.sc_test_attn_q8_rows_wait_expiry(*args, 16, I8, F32, -1, 10, stream=0) == scl.SC_ERR_SHAPE
    assert scl.sc_test_attn_q8_rows_wait_expiry(*args, 16, I8, F32, 0, 0, stream=0) == scl.SC_ERR_SHAPE


def test_wait_expiry_hook_refusals():
    args = (A, B, C, D_, E, G, 2, 4, 40, 2, 2, 32)
    assert scl.sc_test_attn_q8_wait_expiry(None, *args[1:], 16, I8, F32, 0, 10, stream=0) == scl.SC_ERR_NULL
    assert scl.sc_test_attn_q8_wait_expiry(*args, 20, I8, F32, 0, 10, stream=0) == scl.SC_ERR_UNSUPPORTED
    assert scl.sc_test_attn_q8_wait_expiry(*args, 16, I8, F32, -1, 10, stream=0) == scl.SC_ERR_SHAPE
    assert scl.sc_test_attn_q8_wait_expiry(*args, 16, I8, F32, 0, 0, stream=0) == scl.SC_ERR_SHAPE


A, B, C, D_, E, G = (1 << k for k in (20, 24, 28, 32, 34, 36))


@pytest.mark.parametrize("change,expect", [
    (dict(q=None), scl.SC_ERR_NULL), (dict(k=None), scl.SC_ERR_NULL), (dict(v=None), scl.SC_ERR_NULL),
    (dict(ks=None), scl.SC_ERR_NULL), (dict(vs=None), scl.SC_ERR_NULL), (dict(out=None), scl.SC_ERR_NULL),
    (dict(N=0), scl.SC_ERR_SHAPE), (dict(Tk=0), scl.SC_ERR_SHAPE), (dict(Tq=-1), scl.SC_ERR_SHAPE),
    (dict(Tk=(1 << 30) + 1), scl.SC_ERR_SHAPE), (dict(Hq=3), scl.SC_ERR_UNSUPPORTED), (dict(D=24), scl.SC_ERR_UNSUPPORTED),
    (dict(D=144), scl.SC_ERR_UNSUPPORTED), (dict(block=8), scl.SC_ERR_UNSUPPORTED), (dict(block=100), scl.SC_ERR_UNSUPPORTED),
    (dict(code=7), scl.SC_ERR_UNSUPPORTED), (dict(dtype=2), scl.SC_ERR_UNSUPPORTED), (dict(scale=0.0), scl.SC_ERR_UNSUPPORTED),
    (dict(scale=math.inf), scl.SC_ERR_UNSUPPORTED), (dict(q=A + 8), scl.SC_ERR_ALIGN), (dict(k=B + 8), scl.SC_ERR_ALIGN),
    (dict(ks=C + 2), scl.SC_ERR_ALIGN), (dict(vs=C + 1), scl.SC_ERR_ALIGN), (dict(out=G + 8), scl.SC_ERR_ALIGN),
    (dict(strides=((256, 64, 32), (1280, 40, 16), (1280, 32, 16), (256, 64, 32))), scl.SC_ERR_ALIGN),
    (dict(strides=((256, 64, 32), (1280, -32, 16), (1280, 32, 16), (256, 64, 32))), scl.SC_ERR_SHAPE),
    (dict(strides=((256, 64, 32), (1280, 64, 32), (1280, 0, 32), (256, 64, 32))), scl.SC_ERR_UNSUPPORTED),
    (dict(strides=((256, 64, 32), (1 << 40, 64, 32), (1280, 64, 32), (256, 64, 32)), k=1 << 50), scl.SC_ERR_UNSUPPORTED),
    (dict(strides=((256, 64, 32), (1280, 32, 16), (1280, 32, 16), (256, 32, 32))), scl.SC_ERR_ALIAS),
    (dict(out=A), scl.SC_ERR_ALIAS), (dict(out=B + 16), scl.SC_ERR_ALIAS), (dict(out=C), scl.SC_ERR_ALIAS),
    (dict(out=G, lse=G + 4), scl.SC_ERR_ALIAS), (dict(lse=C + 4), scl.SC_ERR_ALIAS), (dict(lse=B), scl.SC_ERR_ALIAS),
])
def test_refusals(change, expect):
    a = dict(q=A, k=B, ks=C, v=D_, vs=E, out=G, lse=None, N=2, Tq=4, Tk=40, Hq=2, Hkv=2, D=32, block=16, code=I8, dtype=F32,
             scale=1.0, strides=None)
    a.update(change)
    rc = scl.cross_attention_q8_fwd(a["q"], a["k"], a["ks"], a["v"], a["vs"], a["out"], a["N"], a["Tq"], a["Tk"], a["Hq"],
                                    a["Hkv"], a["D"], a["scale"], a["block"], a["code"], a["dtype"], lse=a["lse"],
                                    strides=a["strides"], stream=0)
    assert rc == expect, scl.sc_status_string(rc)
