"""What is measured of a decoder layer's operators over a feature map: cases, plain forms, exact values.

A decoder layer that attends to a feature map projects its tokens, attends to
the map's states, adds what comes back to its residual stream and norms the sum
for the next block.  The map's keys and values are made once and read at every
step, so they are held in 8 bits:

* ``linear``: y = act(x w^T + b) + residual.
* ``residual_norm``: s = scale * residual + gate * post(x), y = pre(s): the norm
  behind one block, its gate, the residual stream and the norm before the next
  block in one pass.
* ``kv_quantize``: states as 8-bit codes (integers, or floats of 4 exponent and
  3 mantissa bits) with one scale for each block of states and head.
* ``cross_attention_q8``: attention to states held that way, from one query to
  many, with lengths, masks and shared key heads.

``own`` False: elementary torch operations in 32 bits (64 where a value next to
a code's border has to fall on the right side).  ``own`` True: this library's
entry points.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
_CODES = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
_TOP = {"i8": 127.0, "e4m3": 448.0}   # a code's largest value
_EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _linear(name, dtype, rows, Cin, Cout, act, bias, residual):
    return dict(name=name, op="linear", dtype=dtype, rows=rows, Cin=Cin, Cout=Cout, act=act, bias=bias,
                residual=residual)


def _norm(name, dtype, N, T, C, post, pre, gate, scale):
    return dict(name=name, op="residual_norm", dtype=dtype, N=N, T=T, C=C, post=post, pre=pre, gate=gate, scale=scale)


def _quant(name, dtype, code, N, Tk, Hkv, D, block, valid="all"):
    return dict(name=name, op="kv_quantize", dtype=dtype, code=code, N=N, Tk=Tk, Hkv=Hkv, D=D, block=block, valid=valid)


def _attn(name, dtype, code, N, Tq, Tk, Hq, Hkv, D, block, valid="all", lse=False):
    return dict(name=name, op="cross_attention_q8", dtype=dtype, code=code, N=N, Tq=Tq, Tk=Tk, Hq=Hq, Hkv=Hkv, D=D,
                block=block, valid=valid, lse=lse)


def listed():
    return [
        # the output projection of one new token for each of four captions, 16 heads of 64: launch latency
        _linear("linear_step", "bf16", 4, 1024, 1024, "none", True, True),
        # one token of three captions in fp32 to the scores of an odd-sized vocabulary: reads the weights once
        _linear("linear_logits_fp32", "f32", 3, 512, 32001, "none", False, False),
        # the first MLP product of the states of four 1280 x 720 / 16 maps and one token, in fp32
        _linear("linear_states_fp32", "f32", 4 * 80 * 45 + 1, 1024, 4096, "silu", True, False),
        # the first MLP product of four images' 128 x 128 pixels: the arithmetic-bound case
        _linear("linear_pixels", "bf16", 4 * 128 * 128, 2048, 8192, "gelu", True, False),
        # a decode step of four captions, norm before the next block only: launch latency
        _norm("norm_step", "bf16", 4, 1, 1024, "none", "rms", False, 1.0),
        # four images' 128 x 128 pixels in fp32: norm, gate by image, scaled residual, layer norm
        _norm("norm_pixels", "f32", 4, 128 * 128, 2048, "rms", "layer", True, 0.5),
        # keys and values of one caption's 24 x 40 map: launch latency
        _quant("quantize_small_map", "bf16", "i8", 1, 24 * 40, 4, 64, 64),
        # 56 x 56 maps of 32 images of different valid lengths in fp32, as conv2d_fwd writes them
        _quant("quantize_maps", "f32", "e4m3", 32, 56 * 56, 8, 64, 32, valid="lengths"),
        # one new token for each of 32 captions, 56 x 56 maps of different valid lengths (one with none),
        # four query heads to a key head
        _attn("token_batch_lengths", "bf16", "i8", 32, 1, 56 * 56, 16, 4, 64, 64, valid="lengths"),
        # one token over every pixel of a 1280 x 720 map, one key head for four query heads
        _attn("token_whole_image", "bf16", "e4m3", 1, 1, 1280 * 720, 4, 1, 64, 128, lse=True),
        # an odd number of fp32 queries over padded 56 x 56 maps, four query heads to a key head
        _attn("prompt_masked_fp32", "f32", "i8", 8, 77, 56 * 56, 8, 2, 64, 32, valid="mask", lse=True),
        # 128 x 128 pixels of four images attending to the states of 1280 x 720 / 16: the arithmetic-bound case
        _attn("pixels_to_states", "bf16", "i8", 4, 128 * 128, 80 * 45, 16, 16, 128, 128),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_FLOPS_MAX = {"bf16": 1.5e12, "f32": 1.2e11}
_BYTES_MAX = 1.0e9


def draw(rng):
    op = rng.choice(["linear", "linear", "residual_norm", "kv_quantize", "cross_attention_q8", "cross_attention_q8"])
    dtype = rng.choice(["bf16", "f32"])
    while True:
        if op == "linear":
            rows = rng.choice([_logint(rng, 1, 16), _logint(rng, 1, 65536), _logint(rng, 17, 65536)])
            case = _linear("", dtype, rows, 8 * _logint(rng, 4, 1024), _logint(rng, 16, 33000),
                           rng.choice(["none", "relu", "gelu", "silu"]), rng.random() < 0.5, rng.random() < 0.5)
        elif op == "residual_norm":
            case = _norm("", dtype, _logint(rng, 1, 32), _logint(rng, 1, 16384), 8 * _logint(rng, 4, 1024),
                         rng.choice(["none", "rms", "layer"]), rng.choice(["rms", "layer"]), rng.random() < 0.5,
                         rng.choice([1.0, 0.5]))
        else:
            code, block = rng.choice(["i8", "e4m3"]), rng.choice([16, 32, 64, 128])
            D, Hkv = rng.choice([16, 32, 48, 64, 64, 80, 96, 128, 128]), rng.choice([1, 2, 3, 4, 8])
            N, Tk = _logint(rng, 1, 32), _logint(rng, 16, 1280 * 720)
            valid = rng.choice(["all", "lengths", "mask"])
            if op == "kv_quantize":
                case = _quant("", dtype, code, N, Tk, Hkv, D, block, valid)
            else:
                Tq = rng.choice([1, 1, _logint(rng, 2, 16), _logint(rng, 17, 16384)])
                case = _attn("", dtype, code, N, Tq, Tk, Hkv * rng.choice([1, 1, 2, 4, 5]), Hkv, D, block, valid,
                             rng.random() < 0.5)
                if 4.0 * N * Tq * case["Hq"] * Tk > 1.6e10:      # the plain form's scores
                    continue
        w = work(dict(case, valid="all"))
        if w["flops"] <= _FLOPS_MAX[dtype] and w["bytes"] <= _BYTES_MAX:
            break
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs, from the seed alone
# ---------------------------------------------------------------------------
def _lengths(case):
    """Valid lengths of the N sequences before they are shuffled: none for the
    first of several, the others spread from a quarter of Tk to all of it."""
    N, Tk = case["N"], case["Tk"]
    if N == 1:
        return [max(1, (3 * Tk) // 4)]
    return [0] + [max(1, Tk // 4 + (3 * Tk // 4) * (i + 1) // (N - 1)) if i < N - 2 else Tk for i in range(N - 1)]


def _map_sides(case):
    """The feature map's height and width (the factors of Tk nearest to a
    square) and each sequence's valid height and width before the shuffle."""
    N, Tk = case["N"], case["Tk"]
    h = next(d for d in range(int(math.isqrt(Tk)), 0, -1) if Tk % d == 0)
    w = Tk // h
    valid = [(max(1, h - (h * i) // (2 * N)), max(1, w - (w * (N - 1 - i)) // (2 * N))) for i in range(N)]
    return h, w, valid


def _blocks(case):
    return (case["Tk"] + case["block"] - 1) // case["block"]


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, gain=1.0, to=dt):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * gain).to(to)

    x = {}
    if case["op"] == "linear":
        M, K, C = case["rows"], case["Cin"], case["Cout"]
        x["x"], x["w"] = normal(M, K), normal(C, K, gain=K ** -0.5)
        x["b"] = normal(C, gain=0.1, to=torch.float32) if case["bias"] else None
        x["residual"] = normal(M, C) if case["residual"] else None
        return x
    if case["op"] == "residual_norm":
        N, T, C = case["N"], case["T"], case["C"]
        x["x"], x["residual"] = normal(N * T, C), normal(N * T, C, gain=2.0)
        x["gate"] = normal(N, C, gain=0.5, to=torch.float32) if case["gate"] else None
        for side in ("post", "pre"):
            # a norm's weight and, with the mean removed, its bias
            x[side + "_weight"] = 1.0 + normal(C, gain=0.2, to=torch.float32) if case[side] != "none" else None
            x[side + "_bias"] = normal(C, gain=0.1, to=torch.float32) if case[side] == "layer" else None
        return x
    N, Tk, Hkv, D = (case[n] for n in ("N", "Tk", "Hkv", "D"))
    order = torch.randperm(N, generator=torch.Generator().manual_seed(seed)).tolist()
    x["k_len"] = x["key_mask"] = None
    if case["valid"] == "lengths":
        lens = _lengths(case)
        x["k_len"] = torch.tensor([lens[i] for i in order], dtype=torch.int32, device=dev)
    elif case["valid"] == "mask":
        h, w, valid = _map_sides(case)
        hw = torch.tensor([valid[i] for i in order], device=dev)
        rows = torch.arange(h, device=dev).view(1, h, 1) < hw[:, 0].view(N, 1, 1)
        cols = torch.arange(w, device=dev).view(1, 1, w) < hw[:, 1].view(N, 1, 1)
        x["key_mask"] = (rows & cols).view(N, Tk).to(torch.uint8).contiguous()
    if case["op"] == "kv_quantize":
        x["k"], x["v"] = normal(N, Tk, Hkv, D), normal(N, Tk, Hkv, D, gain=0.5)
        return x
    x["q"] = normal(N, case["Tq"], case["Hq"], D, gain=2.0)
    for name, gain in (("k", 1.0), ("v", 0.5)):
        # codes as a block's largest value of some 3.5 standard deviations leaves them, scales a little uneven
        top = _TOP[case["code"]]
        y = torch.randn(N, Tk, Hkv, D, generator=g, device=dev) * (top / 3.5)
        y = y.clamp_(-top, top)
        x[name] = y.round_().to(torch.int8) if case["code"] == "i8" else y.to(torch.float8_e4m3fn)
        s = torch.rand(N, Hkv, _blocks(case), generator=g, device=dev)
        x[name + "_scale"] = (0.75 + 0.5 * s) * (3.5 * gain / top)
    return x


def prepare(case, seed):
    state = {"case": case, **_inputs(case, seed)}
    if case["op"] == "kv_quantize":
        # the cache: what a call leaves as it was is zero
        for name in ("k", "v"):
            state[name + "_codes"] = torch.zeros(state[name].shape, dtype=torch.int8, device="cuda")
            state[name + "_scales"] = torch.zeros(case["N"], case["Hkv"], _blocks(case), device="cuda")
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _valid(st):
    """[N][Tk] truth values, or None where every state is valid."""
    Tk = st["case"]["Tk"]
    if st["k_len"] is not None:
        return torch.arange(Tk, device=st["k"].device).view(1, Tk) < st["k_len"].view(-1, 1)
    return None if st["key_mask"] is None else st["key_mask"] != 0


def _plain_linear(st):
    c = st["case"]
    y = torch.matmul(st["x"].float(), st["w"].float().t())
    if st["b"] is not None:
        y += st["b"]
    if c["act"] == "relu":
        y.clamp_(min=0)
    elif c["act"] == "gelu":
        y *= 0.5 * (1.0 + torch.erf(y * math.sqrt(0.5)))
    elif c["act"] == "silu":
        y *= 1.0 / (1.0 + torch.exp(-y))
    if st["residual"] is not None:
        y += st["residual"].float()
    return {"y": y.to(st["x"].dtype)}


def _plain_normed(y, st, side):
    kind = st["case"][side]
    if kind == "none":
        return y
    if kind == "layer":
        y = y - y.mean(dim=-1, keepdim=True)
    y = y * torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + _EPS) * st[side + "_weight"]
    return y if st[side + "_bias"] is None else y + st[side + "_bias"]


def _plain_residual_norm(st):
    c = st["case"]
    t = _plain_normed(st["x"].float(), st, "post")
    if st["gate"] is not None:
        t = (t.view(c["N"], c["T"], c["C"]) * st["gate"].view(c["N"], 1, c["C"])).view(t.shape)
    s = c["scale"] * st["residual"].float() + t
    dt = st["x"].dtype
    return {"sum": s.to(dt), "y": _plain_normed(s, st, "pre").to(dt)}


def _to_code(y, code):
    """The code's value nearest to y (64 bits), ties to even."""
    if code == "i8":
        return y.round().to(torch.int8)
    # spacing of the codes at |y|: 2^-3 of its power of two, 2^-9 below 2^-6
    # (made of its bits: a power by pow may be off by a little)
    step = ((torch.frexp(y).exponent.clamp(min=-5).long() + 1019) << 52).view(torch.float64)
    return ((y / step).round() * step).float().to(torch.float8_e4m3fn)


def _plain_quantize(st):
    c = st["case"]
    N, Tk, Hkv, D, B = (c[n] for n in ("N", "Tk", "Hkv", "D", "block"))
    nb, valid, out = _blocks(c), _valid(st), {}
    for name in ("k", "v"):
        x = torch.zeros(N, nb * B, Hkv, D, dtype=torch.float64, device="cuda")
        x[:, :Tk] = st[name] if valid is None else torch.where(valid.view(N, Tk, 1, 1), st[name], torch.zeros_like(st[name]))
        x = x.view(N, nb, B, Hkv, D)
        top = x.abs().amax(dim=(2, 4), keepdim=True)
        y = x * _TOP[c["code"]] / torch.where(top > 0, top, torch.ones_like(top))
        out[name] = _to_code(y, c["code"]).view(N, nb * B, Hkv, D)[:, :Tk].contiguous()
        out[name + "_scale"] = (top.view(N, nb, Hkv).float() / _TOP[c["code"]]).transpose(1, 2).contiguous()
    return out


def _plain_attention(st):
    c = st["case"]
    N, Tq, Tk, Hq, Hkv, D, B = (c[n] for n in ("N", "Tq", "Tk", "Hq", "Hkv", "D", "block"))
    G = Hq // Hkv

    def states(name):
        s = st[name + "_scale"].transpose(1, 2).repeat_interleave(B, dim=1)[:, :Tk]
        return st[name].float().mul_(s.unsqueeze(-1))

    q = st["q"].float().view(N, Tq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(N, Hkv, G * Tq, D)
    s = torch.matmul(q, states("k").permute(0, 2, 3, 1)).mul_(D ** -0.5)
    valid = _valid(st)
    if valid is not None:
        s.masked_fill_(~valid.view(N, 1, 1, Tk), float("-inf"))
    top = s.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)   # rows with no valid key
    p = s.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, states("v").permute(0, 2, 1, 3)) / torch.where(total > 0, total, torch.ones_like(total))
    out = {"out": o.view(N, Hkv, G, Tq, D).permute(0, 3, 1, 2, 4).reshape(N, Tq, Hq, D).to(st["q"].dtype)}
    if c["lse"]:
        out["lse"] = (top + total.log()).view(N, Hq, Tq)
    return out


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own_pass(st):
    import stencil_conv2d_fwd_gb300 as sc
    c = st["case"]
    dt = sc.SC_BF16 if c["dtype"] == "bf16" else sc.SC_F32
    if c["op"] == "linear":
        act = {"none": sc.SC_ACT_NONE, "relu": sc.SC_ACT_RELU, "gelu": sc.SC_ACT_GELU, "silu": sc.SC_ACT_SILU}[c["act"]]
        y = torch.empty(c["rows"], c["Cout"], dtype=st["x"].dtype, device="cuda")
        sc.check(sc.linear_fwd(st["x"], st["w"], st["b"], y, c["rows"], c["Cin"], c["Cout"], act, dt,
                               residual=st["residual"]), "linear_fwd")
        return {"y": y}
    if c["op"] == "residual_norm":
        kinds = {"none": sc.SC_NORM_NONE, "rms": sc.SC_NORM_RMS, "layer": sc.SC_NORM_LAYER}
        post, pre = ((kinds[c[s]], st[s + "_weight"], st[s + "_bias"], _EPS) for s in ("post", "pre"))
        s, y = torch.empty_like(st["x"]), torch.empty_like(st["x"])
        sc.check(sc.residual_norm_fwd(st["x"], st["residual"], s, y, c["N"] * c["T"], c["C"], post=post, pre=pre,
                                      gate=st["gate"], gate_rows=c["T"], scale=c["scale"], dtype=dt), "residual_norm_fwd")
        return {"sum": s, "y": y}
    code = sc.SC_CODE_I8 if c["code"] == "i8" else sc.SC_CODE_E4M3
    N, Tk, Hkv, D = (c[n] for n in ("N", "Tk", "Hkv", "D"))
    if c["op"] == "kv_quantize":
        sc.check(sc.kv_quantize_fwd((st["k"], st["k_codes"], st["k_scales"]), (st["v"], st["v_codes"], st["v_scales"]),
                                    N, Tk, Hkv, D, c["block"], code, dt, k_len=st["k_len"], key_mask=st["key_mask"]),
                 "kv_quantize_fwd")
        return {"k": st["k_codes"].view(_CODES[c["code"]]), "k_scale": st["k_scales"],
                "v": st["v_codes"].view(_CODES[c["code"]]), "v_scale": st["v_scales"]}
    out = torch.empty_like(st["q"])
    lse = torch.empty(N, c["Hq"], c["Tq"], device="cuda") if c["lse"] else None
    sc.check(sc.cross_attention_q8_fwd(st["q"], st["k"], st["k_scale"], st["v"], st["v_scale"], out, N, c["Tq"], Tk,
                                       c["Hq"], Hkv, D, D ** -0.5, c["block"], code, dt, k_len=st["k_len"],
                                       key_mask=st["key_mask"], lse=lse), "cross_attention_q8_fwd")
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


def run(state):
    """Codes come as the values that they stand for before their block's scale, scales beside them."""
    if own:
        return _own_pass(state)
    return {"linear": _plain_linear, "residual_norm": _plain_residual_norm, "kv_quantize": _plain_quantize,
            "cross_attention_q8": _plain_attention}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its exact result
# ---------------------------------------------------------------------------
def work(case):
    e = _SIZE[case["dtype"]]
    if case["op"] == "linear":
        M, K, C = case["rows"], case["Cin"], case["Cout"]
        nbytes = e * (M * K + C * K + M * C * (2 if case["residual"] else 1)) + (4 * C if case["bias"] else 0)
        return {"bytes": nbytes, "flops": 2 * M * K * C}
    if case["op"] == "residual_norm":
        M, C = case["N"] * case["T"], case["C"]
        vectors = sum({"none": 0, "rms": 1, "layer": 2}[case[s]] for s in ("post", "pre"))
        return {"bytes": 4 * M * C * e + 4 * C * (vectors + (case["N"] if case["gate"] else 0)),
                "flops": M * C * (3 + 4 * vectors)}
    N, Tk, Hkv, D, B = (case[n] for n in ("N", "Tk", "Hkv", "D", "block"))
    keys, extra = N * Tk, 0
    blocks = N * _blocks(case)
    if case["valid"] == "lengths":
        lens = _lengths(case)
        keys, extra, blocks = sum(lens), 4 * N, sum((n + B - 1) // B for n in lens)
    elif case["valid"] == "mask":
        keys, extra = sum(h * w for h, w in _map_sides(case)[2]), N * Tk
    if case["op"] == "kv_quantize":
        return {"bytes": 2 * (keys * Hkv * D * (e + 1) + 4 * blocks * Hkv) + extra, "flops": 6 * keys * Hkv * D}
    Tq, Hq = case["Tq"], case["Hq"]
    nbytes = 2 * e * N * Tq * Hq * D + 2 * keys * Hkv * D + 8 * blocks * Hkv + extra + (4 * N * Hq * Tq if case["lse"] else 0)
    return {"bytes": nbytes, "flops": 4 * Tq * Hq * D * keys}


def _exact_linear(case, x):
    y = x["x"].double() @ x["w"].double().t()
    if case["bias"]:
        y += x["b"].double()
    if case["act"] == "relu":
        y = torch.where(y > 0, y, torch.zeros_like(y))
    elif case["act"] == "gelu":
        y *= torch.special.ndtr(y)
    elif case["act"] == "silu":
        y *= torch.sigmoid(y)
    return {"y": y + x["residual"].double() if case["residual"] else y}


def _exact_residual_norm(case, x):
    def norm(v, side):
        if case[side] == "none":
            return v
        if case[side] == "layer":
            var, mean = torch.var_mean(v, dim=-1, correction=0, keepdim=True)
            return (v - mean) / torch.sqrt(var + _EPS) * x[side + "_weight"].double() + x[side + "_bias"].double()
        return v / torch.sqrt(v.pow(2).sum(dim=-1, keepdim=True) / case["C"] + _EPS) * x[side + "_weight"].double()

    t = norm(x["x"].double(), "post")
    if case["gate"]:
        t = t * x["gate"].double().repeat_interleave(case["T"], dim=0)
    s = x["residual"].double() * case["scale"] + t
    return {"sum": s, "y": norm(s, "pre")}


def _exact_quantize(case, x):
    """Block by block of states; codes by comparison with the borders between them."""
    N, Tk, Hkv, D, B = (case[n] for n in ("N", "Tk", "Hkv", "D", "block"))
    dev = x["k"].device
    if case["code"] == "i8":
        values = torch.arange(0, 128, dtype=torch.float64, device=dev)
    else:
        values = torch.arange(0, 127, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn).double()
    borders = (values[1:] + values[:-1]) / 2
    keep = torch.ones(N, Tk, dtype=torch.bool, device=dev)
    if x["k_len"] is not None:
        keep = torch.arange(Tk, device=dev)[None, :] < x["k_len"][:, None]
    if x["key_mask"] is not None:
        keep = x["key_mask"].bool()
    out = {}
    for name in ("k", "v"):
        codes = torch.zeros(N, Tk, Hkv, D, dtype=torch.float64, device=dev)
        scale = torch.zeros(N, Hkv, _blocks(case), dtype=torch.float64, device=dev)
        step = B * max(1, int(4e7 // (N * B * Hkv * D)))
        for t in range(0, Tk, step):
            y = x[name][:, t:t + step].double() * keep[:, t:t + step, None, None]
            n = y.shape[1]
            rows = torch.arange(n, device=dev) // B
            top = torch.zeros(N, int(rows[-1]) + 1, Hkv, dtype=torch.float64, device=dev)
            top.scatter_reduce_(1, rows.view(1, n, 1).expand(N, n, Hkv), y.abs().amax(dim=3), "amax")
            scale[:, :, t // B:t // B + top.shape[1]] = top.transpose(1, 2) / values[-1]
            size = y.abs() * values[-1] / torch.where(top > 0, top, torch.ones_like(top))[:, rows].unsqueeze(-1)
            at = torch.bucketize(size, borders)                       # borders below
            tie = (at < borders.numel()) & (size == borders[at.clamp(max=borders.numel() - 1)]) & (at % 2 == 1)
            codes[:, t:t + step] = values[at + tie] * torch.sign(y)
        out[name] = codes.to(torch.int8) if case["code"] == "i8" else codes
        out[name + "_scale"] = scale
    return out


def _exact_attention(case, x):
    """Sequence by sequence and head by head, keys gathered before the products."""
    N, Tq, Tk, Hq, Hkv, D = (case[n] for n in ("N", "Tq", "Tk", "Hq", "Hkv", "D"))
    out = torch.zeros(N, Tq, Hq, D, dtype=torch.float64, device=x["q"].device)
    lse = torch.full((N, Hq, Tq), float("-inf"), dtype=torch.float64, device=out.device)
    for n in range(N):
        keep = torch.arange(Tk, device=out.device)
        if x["k_len"] is not None:
            keep = keep[:int(x["k_len"][n])]
        if x["key_mask"] is not None:
            keep = keep[x["key_mask"][n].bool()]
        if keep.numel() == 0:
            continue
        step = max(1, int(2.5e8 // keep.numel()))
        for h in range(Hq):
            g = h * Hkv // Hq
            k = x["k"][n, :, g].double()[keep] * x["k_scale"][n, g].double()[keep // case["block"], None]
            v = x["v"][n, :, g].double()[keep] * x["v_scale"][n, g].double()[keep // case["block"], None]
            for t in range(0, Tq, step):
                s = x["q"][n, t:t + step, h].double() @ k.t() / math.sqrt(D)
                z = torch.logsumexp(s, dim=1)
                out[n, t:t + step, h] = torch.exp(s - z[:, None]) @ v
                lse[n, h, t:t + step] = z
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def exact(case, seed):
    x = _inputs(case, seed)
    return {"linear": _exact_linear, "residual_norm": _exact_residual_norm, "kv_quantize": _exact_quantize,
            "cross_attention_q8": _exact_attention}[case["op"]](case, x)
