"""kv_quantize_fwd against the plain 64-bit form, code for code, and its refusals."""
import math

import numpy as np
import pytest

import layer_ref as ref
import stencil_conv2d_fwd_gb300 as scl

BF16, F32, I8, E4M3 = scl.SC_BF16, scl.SC_F32, scl.SC_CODE_I8, scl.SC_CODE_E4M3


def states(torch, dtype, *shape, seed=0, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * gain).to(torch.bfloat16 if dtype == BF16 else torch.float32).cuda()


def valid_of(torch, N, T, k_len=None, key_mask=None):
    valid = torch.ones(N, T, dtype=torch.bool, device="cuda")
    if k_len is not None:
        valid &= torch.arange(T, device="cuda")[None] < torch.tensor(k_len, device="cuda")[:, None]
    if key_mask is not None:
        valid &= torch.as_tensor(np.asarray(key_mask)).cuda() != 0
    return valid


def buffers(torch, x, block):
    N, T, H, D = x.shape
    codes = torch.full((N, T, H, D), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.full((N, H, -(-T // block)), -7.0, device="cuda")
    return codes, scale


def check(torch, x, codes, scale, valid, block, code):
    want, ws = ref.quantize(x, valid, block, code == E4M3)
    got = codes.view(torch.float8_e4m3fn if code == E4M3 else torch.int8).double()
    out = ~valid[:, :, None, None].expand_as(got)
    assert (codes[out] == 0x55).all(), "codes of states that are not valid were written"
    wrong = (got != want) & ~out
    assert not wrong.any(), f"{int(wrong.sum())} codes differ, first at {wrong.nonzero()[0].tolist()}"
    kept = ws.isinf()
    assert (scale[kept] == -7.0).all(), "scales of blocks without a valid state were written"
    s, ws = scale.double()[~kept], ws[~kept]
    assert ((s == ws) | (s.isnan() & ws.isnan())).all()


def run(torch, sc, x, block, code, dtype, k_len=None, key_mask=None, stream=None):
    """x as keys, and its negative, shifted by a state, as values."""
    N, T, H, D = x.shape
    y = -x.roll(1, dims=1)
    kl = None if k_len is None else torch.tensor(k_len, dtype=torch.int32, device="cuda")
    km = None if key_mask is None else torch.as_tensor(np.asarray(key_mask, np.uint8)).cuda()
    (kc, ks), (vc, vs) = buffers(torch, x, block), buffers(torch, x, block)
    sc.check(sc.kv_quantize_fwd((x, kc, ks), (y, vc, vs), N, T, H, D, block, code, dtype, k_len=kl, key_mask=km,
                                stream=stream), "kv_quantize_fwd")
    sc.check(sc.sc_last_device_status(stream))
    valid = valid_of(torch, N, T, k_len, key_mask)
    check(torch, x, kc, ks, valid, block, code)
    check(torch, y, vc, vs, valid, block, code)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 1, 1, 16), (1, 15, 1, 16), (2, 16, 3, 48), (1, 17, 2, 64), (3, 129, 1, 80),
                                   (2, 300, 4, 128), (1, 1000, 8, 64), (2, 127, 5, 112)])
def test_shapes(sc, shape, block, code, dtype):
    import torch
    run(torch, sc, states(torch, dtype, *shape), block, code, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("block", [16, 64, 128])
def test_lengths_and_masks(sc, block, code, dtype):
    """Lengths around a block's end, none, above T and below zero; masks that leave nothing, one state, padded maps;
    NaN in states that are not valid."""
    import torch
    T, H, D = 300, 2, 64
    lens = [0, 1, block - 1, block, block + 1, T, T + 5, -2]
    x = states(torch, dtype, len(lens), T, H, D, seed=1)
    for n, L in enumerate(lens):
        x[n, max(0, L) + 1:] = math.nan   # (the values are a state later)
    run(torch, sc, x, block, code, dtype, k_len=[min(T, L) if L > T else L for L in lens])
    mask = np.zeros((5, T), np.uint8)
    mask[1, 170] = 1
    mask[2, ::2] = 255
    mask[3, :20 * 10].reshape(20, 10)[:, :6] = 1
    mask[4] = 1
    x = states(torch, dtype, 5, T, H, D, seed=2)
    x[1, :160], x[3, 201:] = math.nan, math.inf
    run(torch, sc, x, block, code, dtype, key_mask=mask)
    run(torch, sc, states(torch, dtype, 5, T, H, D, seed=3), block, code, dtype, k_len=[10, 200, 99, 150, 0], key_mask=mask)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("code", [I8, E4M3])
def test_borders_and_ends(sc, code, dtype):
    """Values on and next to the borders between codes, tiny and huge blocks, zeros, an infinity, a NaN."""
    import torch
    T, H, D, block = 16 * 40, 1, 16, 16
    t = torch.bfloat16 if dtype == BF16 else torch.float32
    g = torch.Generator().manual_seed(4)
    top = 448.0 if code == E4M3 else 127.0
    x = torch.zeros(1, T, H, D, dtype=torch.float64)
    if code == E4M3:
        values = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    else:
        values = torch.arange(128).double()
    borders = (values[1:] + values[:-1]) / 2
    for b in range(40):
        a = 2.0 ** int(torch.randint(-120, 100, (), generator=g)) * (1 + int(torch.randint(0, 128, (), generator=g)) / 128)
        pick = borders[torch.randint(0, borders.numel(), (block * D,), generator=g)] * a / top
        nudge = 1 + torch.randint(-2, 3, (block * D,), generator=g) * 2.0 ** -23
        y = pick * nudge * (torch.randint(0, 2, (block * D,), generator=g) * 2 - 1)
        y[0] = a
        x[0, b * block:(b + 1) * block, 0] = y.view(block, D)
    x = x.float()
    x[0, :16] = 0
    x[0, 16:32] = 0
    x[0, 20, 0, 3] = -0.0
    x[0, 32:48] *= 0
    x[0, 40, 0, 5] = 2.0 ** -149 * 77        # a subnormal largest value
    x[0, 41, 0, 5] = -2.0 ** -149 * 31
    x[0, 48:64] = torch.randn(16, 1, 16, generator=g) * 2.0 ** 125
    x[0, 70, 0, 1] = math.inf
    x[0, 90, 0, 2] = math.nan
    x[0, 101, 0, 2], x[0, 102, 0, 2] = math.nan, -math.inf
    run(torch, sc, x.to(t).cuda(), block, code, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("code", [I8, E4M3])
def test_strides_streams_and_appending(sc, code, dtype):
    """States inside a fused projection, codes with a pitch; a cache that grows by whole blocks; a captured call."""
    import torch
    N, T, H, D, block = 2, 192, 3, 32, 32
    x = states(torch, dtype, N, T, H, D, seed=5)
    fused = states(torch, dtype, N, T, 3, H, D, seed=6)
    fused[:, :, 1] = x
    codes = torch.full((N, T + 64, H, 64), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.full((N, H, T // block), -7.0, device="cuda")
    t = (fused[0, 0, 1], codes, scale, (T * 3 * H * D, 3 * H * D, D), ((T + 64) * H * 64, H * 64, 64))
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        sc.check(sc.kv_quantize_fwd(None, t, N, T, H, D, block, code, dtype), "kv_quantize_fwd")
    torch.cuda.synchronize()
    assert (codes == 0x55).all()
    with torch.cuda.stream(stream):
        graph.replay()
    torch.cuda.synchronize()
    check(torch, x, codes[:, :T, :, :D], scale, valid_of(torch, N, T), block, code)
    assert (codes[:, T:] == 0x55).all() and (codes[..., D:] == 0x55).all()
    # one sequence's blocks appended in two calls
    kc, ks = buffers(torch, x[:1, :, :1], block)
    for b0, b1 in ((0, 2), (2, 6)):
        part = x[:1, b0 * block:b1 * block, :1].contiguous()
        sc.check(sc.kv_quantize_fwd((part, kc[:, b0 * block:], ks[:, :, b0:]), None, 1, (b1 - b0) * block, 1, D, block, code,
                                    dtype, stream=stream if b0 else None), "kv_quantize_fwd")
        torch.cuda.synchronize()
    check(torch, x[:1, :, :1], kc, ks, valid_of(torch, 1, T), block, code)


@pytest.mark.gpu
@pytest.mark.parametrize("code", [I8, E4M3])
def test_keys_and_values_in_one_cache(sc, code):
    """Codes of keys and values side by side in one [N][T][2][H][D] cache, which grows by whole blocks under masks."""
    import torch
    N, T, H, D, block = 3, 256, 2, 48, 64
    k, v = states(torch, BF16, N, T, H, D, seed=8), states(torch, BF16, N, T, H, D, seed=9)
    both = torch.full((N, T, 2, H, D), 0x55, dtype=torch.uint8, device="cuda")
    ks, vs = (torch.full((N, H, T // block), -7.0, device="cuda") for _ in range(2))
    cs = (T * 2 * H * D, 2 * H * D, D)
    for b0, b1 in ((0, 1), (1, 3), (3, 4)):
        mask = torch.zeros(N, T, dtype=torch.uint8, device="cuda")
        mask[:, b0 * block:b1 * block] = 1
        old = both.clone(), ks.clone(), vs.clone()
        sc.check(sc.kv_quantize_fwd((k, both, ks, None, cs), (v, both[0, 0, 1], vs, None, cs), N, T, H, D, block, code, BF16,
                                    key_mask=mask), "kv_quantize_fwd")
        sc.check(sc.sc_last_device_status())
        assert torch.equal(both[:, :b0 * block], old[0][:, :b0 * block]) and (both[:, b1 * block:] == 0x55).all()
        assert torch.equal(ks[..., :b0], old[1][..., :b0]) and (vs[..., b1:] == -7.0).all()
    for x, i, s in ((k, 0, ks), (v, 1, vs)):
        check(torch, x, both[:, :, i].contiguous(), s, valid_of(torch, N, T), block, code)


@pytest.mark.gpu
def test_offsets_beyond_32_bits(sc):
    import torch
    T, D, pitch = 48, 16, 1 << 26   # states 2^26 elements apart: the last at 47 * 2^26
    x = states(torch, BF16, 1, T, 1, D, seed=7)
    buf = torch.empty(pitch * (T - 1) + D, dtype=torch.bfloat16, device="cuda")
    cbuf = torch.empty(pitch * (T - 1) + D, dtype=torch.uint8, device="cuda")
    buf.as_strided((T, D), (pitch, 1)).copy_(x[0, :, 0])
    scale = torch.full((1, 1, 3), -7.0, device="cuda")
    sc.check(sc.kv_quantize_fwd((buf, cbuf, scale, (0, pitch, 0), (0, pitch, 0)), None, 1, T, 1, D, 16, I8, BF16))
    sc.check(sc.sc_last_device_status())
    codes = cbuf.as_strided((T, D), (pitch, 1)).clone().view(1, T, 1, D)
    check(torch, x, codes, scale, valid_of(torch, 1, T), 16, I8)


A, B, C, D_, E, G = (1 << k for k in (20, 24, 28, 32, 34, 36))


@pytest.mark.parametrize("change,expect", [
    (dict(k=None, v=None), scl.SC_ERR_NULL), (dict(k=(None, B, C)), scl.SC_ERR_NULL), (dict(k=(A, None, C)), scl.SC_ERR_NULL),
    (dict(v=(D_, E, None)), scl.SC_ERR_NULL), (dict(N=0), scl.SC_ERR_SHAPE), (dict(Tk=-1), scl.SC_ERR_SHAPE),
    (dict(Hkv=0), scl.SC_ERR_SHAPE), (dict(D=24), scl.SC_ERR_UNSUPPORTED), (dict(D=144), scl.SC_ERR_UNSUPPORTED),
    (dict(block=48), scl.SC_ERR_UNSUPPORTED), (dict(block=0), scl.SC_ERR_UNSUPPORTED), (dict(block=256), scl.SC_ERR_UNSUPPORTED),
    (dict(code=2), scl.SC_ERR_UNSUPPORTED), (dict(dtype=3), scl.SC_ERR_UNSUPPORTED),
    (dict(k=(A + 8, B, C)), scl.SC_ERR_ALIGN), (dict(k=(A, B + 8, C)), scl.SC_ERR_ALIGN), (dict(k=(A, B, C + 2)), scl.SC_ERR_ALIGN),
    (dict(k_len=G + 2), scl.SC_ERR_ALIGN), (dict(k=(A, B, C, (4096, 66, 32), None)), scl.SC_ERR_ALIGN),
    (dict(k=(A, B, C, None, (4096, 72, 32))), scl.SC_ERR_ALIGN), (dict(k=(A, B, C, (-64, 64, 32), None)), scl.SC_ERR_SHAPE),
    (dict(k=(A, B, C, None, (4096, 32, 32))), scl.SC_ERR_ALIAS), (dict(k=(A, B, C, None, (0, 64, 32))), scl.SC_ERR_ALIAS),
    (dict(k=(A, A, C)), scl.SC_ERR_ALIAS), (dict(k=(A, B, A + 64)), scl.SC_ERR_ALIAS), (dict(k=(A, B, B)), scl.SC_ERR_ALIAS),
    (dict(v=(D_, B + 16, G)), scl.SC_ERR_ALIAS), (dict(v=(D_, E, C)), scl.SC_ERR_ALIAS), (dict(v=(D_, A, G)), scl.SC_ERR_ALIAS),
    (dict(key_mask=B + 3), scl.SC_ERR_ALIAS), (dict(k_len=C), scl.SC_ERR_ALIAS),
])
def test_refusals(change, expect):
    a = dict(k=(A, B, C), v=(D_, E, G), N=2, Tk=40, Hkv=2, D=32, block=16, code=I8, dtype=F32, k_len=None, key_mask=None)
    a.update(change)
    rc = scl.kv_quantize_fwd(a["k"], a["v"], a["N"], a["Tk"], a["Hkv"], a["D"], a["block"], a["code"], a["dtype"],
                             k_len=a["k_len"], key_mask=a["key_mask"], stream=0)
    assert rc == expect, scl.sc_status_string(rc)
