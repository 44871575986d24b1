"""The decoder layer's operators one after the other, as a layer over a feature map uses them, against the plain
64-bit forms: each operator's result within its own bound for the inputs that it was given, and the layer's result
near the layer computed in 64 bits throughout; then the same layer captured into a graph, for one new token."""
import math
import os
import sys

import pytest

import layer_ref as ref
import stencil_conv2d_fwd_gb300 as scl

HEADS, KEY_HEADS, D, WIDTH, MLP, BLOCK = 8, 2, 64, 512, 1536, 32


def make_weights(torch, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = torch.bfloat16 if dtype == scl.SC_BF16 else torch.float32

    def matrix(cout, cin):
        return (torch.randn(cout, cin, generator=g) * cin ** -0.5).to(t).cuda()

    def vector(n, gain=0.2, one=1.0):
        return (one + gain * torch.randn(n, generator=g)).cuda()

    return {"q": matrix(HEADS * D, WIDTH), "out": matrix(WIDTH, HEADS * D), "up": matrix(MLP, WIDTH), "down": matrix(WIDTH, MLP),
            "up_b": vector(MLP, 0.1, 0.0), "down_b": vector(WIDTH, 0.1, 0.0), "norm_in": vector(WIDTH), "norm_post": vector(WIDTH),
            "norm_mlp": vector(WIDTH)}


class Layer:
    """Buffers of a layer for N x T tokens, run in place on the residual stream."""

    def __init__(self, torch, sc, w, N, T, dtype, code):
        t = torch.bfloat16 if dtype == scl.SC_BF16 else torch.float32
        self.sc, self.w, self.N, self.T, self.dtype, self.code = sc, w, N, T, dtype, code
        n = N * T
        self.h, self.q, self.a, self.o, self.s, self.m, self.u = (torch.empty(n, c, dtype=t, device="cuda") for c in
                                                                 (WIDTH, HEADS * D, HEADS * D, WIDTH, WIDTH, WIDTH, MLP))

    def run(self, x, cache, gate, k_len):
        sc, w, N, T, dt = self.sc, self.w, self.N, self.T, self.dtype
        n, Tk = N * T, cache["k"].shape[1]
        rms = lambda v: (sc.SC_NORM_RMS, v, None, 1e-6)  # noqa: E731
        sc.check(sc.residual_norm_fwd(x, None, None, self.h, n, WIDTH, pre=rms(w["norm_in"]), dtype=dt))
        sc.check(sc.linear_fwd(self.h, w["q"], None, self.q, n, WIDTH, HEADS * D, dtype=dt))
        sc.check(sc.cross_attention_q8_fwd(self.q, cache["k"], cache["ks"], cache["v"], cache["vs"], self.a, N, T, Tk, HEADS,
                                           KEY_HEADS, D, D ** -0.5, BLOCK, self.code, dt, k_len=k_len))
        sc.check(sc.linear_fwd(self.a, w["out"], None, self.o, n, HEADS * D, WIDTH, dtype=dt))
        sc.check(sc.residual_norm_fwd(self.o, x, self.s, self.m, n, WIDTH, post=rms(w["norm_post"]), pre=rms(w["norm_mlp"]),
                                      gate=gate, gate_rows=T, dtype=dt))
        sc.check(sc.linear_fwd(self.m, w["up"], w["up_b"], self.u, n, WIDTH, MLP, sc.SC_ACT_GELU, dt))
        sc.check(sc.linear_fwd(self.u, w["down"], w["down_b"], self.s, n, MLP, WIDTH, dtype=dt, residual=self.s))
        return self.s


def reference(torch, w, x, k, v, gate, valid, T):
    """The layer in 64 bits on the dequantised states."""
    N, n = valid.shape[0], x.shape[0]
    rms = lambda y, g: ref.normed(y, 1, g, None, 1e-6)[0]  # noqa: E731
    q = rms(x.double(), w["norm_in"]) @ w["q"].double().t()
    a = ref.attention(q.view(N, T, HEADS, D), k, v, D ** -0.5, valid)[0].reshape(n, HEADS * D)
    s = x.double() + gate.double().repeat_interleave(T, dim=0) * rms(a @ w["out"].double().t(), w["norm_post"])
    u = rms(s, w["norm_mlp"]) @ w["up"].double().t() + w["up_b"].double()
    return s + (u * torch.special.ndtr(u)) @ w["down"].double().t() + w["down_b"].double()


@pytest.mark.gpu
@pytest.mark.parametrize("code", [scl.SC_CODE_I8, scl.SC_CODE_E4M3])
@pytest.mark.parametrize("dtype", [scl.SC_F32, scl.SC_BF16])
def test_layer(sc, dtype, code):
    import torch
    bf16, N, H, W = dtype == scl.SC_BF16, 3, 21, 17
    Tk = H * W
    t = torch.bfloat16 if bf16 else torch.float32
    g = torch.Generator().manual_seed(1)
    w = make_weights(torch, dtype)
    k, v = (torch.randn(N, Tk, KEY_HEADS, D, generator=g).to(t).cuda() for _ in range(2))
    lens = [Tk, 100, 0]
    k[1, 100:], v[1, 100:] = math.nan, math.nan
    k_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cache = {n: torch.zeros(N, Tk, KEY_HEADS, D, dtype=torch.uint8, device="cuda") for n in "kv"}
    cache |= {n + "s": torch.zeros(N, KEY_HEADS, -(-Tk // BLOCK), device="cuda") for n in "kv"}
    sc.check(sc.kv_quantize_fwd((k, cache["k"], cache["ks"]), (v, cache["v"], cache["vs"]), N, Tk, KEY_HEADS, D, BLOCK, code, dtype,
                                k_len=k_len), "kv_quantize_fwd")
    as_code = torch.float8_e4m3fn if code == scl.SC_CODE_E4M3 else torch.int8
    kk, vv = (ref.dequantize(cache[n].view(as_code).double(), cache[n + "s"], BLOCK) for n in "kv")
    valid = torch.arange(Tk, device="cuda")[None] < k_len[:, None]
    # the cache is near the states: half a code's step of the block's largest value, or of the value itself
    for x, y in ((k, kk), (v, vv)):
        near = 2.0 ** -4 * x.double().abs() + x[valid].double().abs().max() * 2.0 ** -9 if code == scl.SC_CODE_E4M3 else \
            x[valid].double().abs().max() / 254 * (1 + 2.0 ** -7)
        assert ((x.double() - y).abs() <= near)[valid].all()
    gate = (1 + 0.3 * torch.randn(N, WIDTH, generator=g)).cuda()
    for T in (40, 1):   # a prompt, then a token
        x = torch.randn(N * T, WIDTH, generator=g).to(t).cuda()
        layer = Layer(torch, sc, w, N, T, dtype, code)
        y = layer.run(x, cache, gate, k_len).clone()
        sc.check(sc.sc_last_device_status())
        want = reference(torch, w, x, kk, vv, gate, valid, T)
        assert torch.isfinite(y.float()).all()
        # eight roundings of the stream and what feeds it, bf16's or fp32's with its sums, relative to the rows' size
        rel = ((y.double() - want).norm() / want.norm()).item()
        assert rel <= (8 * ref.UB if bf16 else 64 * ref.U * math.sqrt(MLP)), rel
        # each operator on the inputs that it was given
        n = N * T
        q = layer.q.double().view(N, T, HEADS, D)
        o, _, wabs, mag = ref.attention(q, kk, vv, D ** -0.5, valid)
        bound = wabs * (2 * ref.U * (6 * math.sqrt(D) + 32) * mag.transpose(1, 2)[..., None] + 2.0 ** -19 + (2 * ref.UB if bf16 else 0)) \
            + 2.0 ** -39 * vv.abs().sum(dim=1).repeat_interleave(HEADS // KEY_HEADS, dim=1)[:, None].nan_to_num()
        assert ((layer.a.double().view(N, T, HEADS, D) - o).abs() <= bound + 1e-30).all()
        assert (layer.a.view(N, T, -1)[2] == 0).all()       # the sequence without a state
        for src, wt, b, act, dst in ((layer.h, "q", None, 0, layer.q), (layer.a, "out", None, 0, layer.o),
                                     (layer.m, "up", "up_b", ref.ACT_GELU, layer.u)):
            want, mag, a = ref.linear(src, w[wt], None if b is None else w[b], None, act)
            assert ((dst.double() - want).abs() <= ref.linear_bound(want, mag, a, src.shape[1], bf16)).all(), wt
    # the token's layer in a graph, replayed on another token: the same bits as the calls
    x2 = torch.randn(N, WIDTH, generator=g).to(t).cuda()
    eager = layer.run(x2, cache, gate, k_len).clone()
    xin = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run(xin, cache, gate, k_len)
    xin.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(layer.s, eager)
    xin.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(layer.s, y)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 40, 700])
@pytest.mark.parametrize("dtype", [scl.SC_F32, scl.SC_BF16])
def test_calls_back_to_back_equal_calls_one_at_a_time(sc, dtype, rows):
    """Every operator reads what the call before has written, many times over and in place, with new inputs each time: the
    launches overlap their starts, and their temporary buffers are the ones that the last call has given back.  The same
    bits as with a wait behind every call."""
    import torch
    t = torch.bfloat16 if dtype == scl.SC_BF16 else torch.float32
    g = torch.Generator().manual_seed(5)
    Tk, C, TURNS = 416, HEADS * D, 25
    w = [(torch.randn(a, b, generator=g) * b ** -0.5).to(t).cuda() for a, b in ((C, C), (2 * KEY_HEADS * D, C), (MLP, C), (C, MLP))]
    bias, norm = torch.randn(MLP, generator=g).cuda(), (1 + 0.2 * torch.randn(C, generator=g)).cuda()
    xs = [torch.randn(rows, C, generator=g).to(t).cuda() for _ in range(TURNS)]
    states = [torch.randn(Tk, C, generator=g).to(t).cuda() for _ in range(TURNS)]

    def turns(wait):
        x, h, u, a = (torch.zeros(rows, n, dtype=t, device="cuda") for n in (C, C, MLP, C))
        kv = torch.zeros(Tk, 2, KEY_HEADS, D, dtype=t, device="cuda")
        codes = [torch.zeros(1, Tk, KEY_HEADS, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros(1, KEY_HEADS, Tk // BLOCK, device="cuda") for _ in range(2)]
        st = ((0, 2 * KEY_HEADS * D, D), None)
        outs = []

        def call(rc):
            sc.check(rc)
            if wait:
                torch.cuda.synchronize()

        for i in range(TURNS):
            x.add_(xs[i])
            call(sc.residual_norm_fwd(x, None, None, h, rows, C, pre=(sc.SC_NORM_RMS, norm, None, 1e-6), dtype=dtype))
            call(sc.linear_fwd(states[i], w[1], None, kv, Tk, C, 2 * KEY_HEADS * D, dtype=dtype))
            call(sc.kv_quantize_fwd((kv, codes[0], scales[0], *st), (kv[0, 1], codes[1], scales[1], *st), 1, Tk, KEY_HEADS, D, BLOCK,
                                    scl.SC_CODE_I8, dtype))
            call(sc.linear_fwd(h, w[0], None, a, rows, C, C, dtype=dtype))
            call(sc.cross_attention_q8_fwd(a, codes[0], scales[0], codes[1], scales[1], h, 1, rows, Tk, HEADS, KEY_HEADS, D, D ** -0.5,
                                           BLOCK, scl.SC_CODE_I8, dtype))
            call(sc.residual_norm_fwd(h, x, x, h, rows, C, pre=(sc.SC_NORM_RMS, norm, None, 1e-6), dtype=dtype))
            call(sc.linear_fwd(h, w[2], bias, u, rows, C, MLP, sc.SC_ACT_GELU, dtype))
            call(sc.linear_fwd(u, w[3], None, x, rows, MLP, C, dtype=dtype, residual=x))
            outs.append(x.clone())
        torch.cuda.synchronize()
        return outs

    want = turns(True)
    assert all(torch.isfinite(y.float()).all() for y in want)
    for _ in range(3):
        for i, (y, z) in enumerate(zip(turns(False), want)):
            assert torch.equal(y, z), f"turn {i}"


@pytest.mark.gpu
@pytest.mark.parametrize("code,near", [(scl.SC_CODE_I8, 127.0), (scl.SC_CODE_E4M3, 16.0)])
@pytest.mark.parametrize("dtype", [scl.SC_F32, scl.SC_BF16])
def test_example_with_states_in_8_bits(sc, dtype, code, near):
    """The feature-map example runs with its states in 8 bits, for points of interest and for a token, and gives what it
    gives without, but for the states' rounding: half a step of 1 / 127, or 1 / 16, of a block's largest value."""
    import torch
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import feature_map_attention as ex
    N, H, W = 2, 24, 40
    g = torch.Generator().manual_seed(3)
    images, w = torch.rand(N, H, W, generator=g).cuda(), ex.make_weights()
    valid = [(24, 31), (17, 40)]
    plain, held = ex.FeatureMap(images, w, valid, dtype), ex.FeatureMap(images, w, valid, dtype, code)
    t = torch.bfloat16 if dtype == scl.SC_BF16 else torch.float32
    for T in (9, 1):
        q = torch.randn(N, T, ex.HEADS, ex.D, generator=g).to(t).cuda()
        places = torch.stack([torch.randint(0, s, (N * T,), generator=g, dtype=torch.int32) for s in (H, W)]).cuda()
        a, b = plain.attend(q, places), held.attend(q, places)
        sc.check(sc.sc_last_device_status())
        assert held.k is None and held.cache is not None
        # a normalised key's element is off by at most 8 / (2 near), in length sqrt(64) times that, so a score by 1.5 * 8 of
        # it times 1 / 8 (|q| is 1.5 sqrt(64), the scale 1 / 8), weights by twice that, values by their own half step
        ds = 1.5 * 8 * 8 / (2 * near)
        size = plain.v.float().abs().amax()
        assert ((a.float() - b.float()).abs() <= size * (2 * min(1.0, ds) + 1 / (2 * near) + 2.0 ** -6)).all()
