"""What is measured of the attention operators: cases, their plain form and their exact values.

A convolutional encoder's NHWC feature map [N][H][W][C] is, without moving a
byte, a sequence of H * W states of C = heads * D channels; 1x1 convolutions
of it are keys and values.  The operators here let a decoder's tokens attend
to such states:

* ``cross_attention``: out = softmax(scale * q k^T over the valid keys) v, with
  shared key heads, a length or a byte mask for each sequence's states, from
  one query to many.
* ``qk_norm_rotary``: RMS norm of each head of the queries and keys and the
  position rotation, in one pass.
* ``rotary``: the position rotation alone, both pair layouts, part of the
  head, one position axis or two (row and column of a feature map), scaled
  frequencies.

``own`` False: elementary torch operations in 32 bits.  ``own`` True: this
library's entry points.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attn(name, dtype, N, Tq, Tk, Hq, Hkv, D, valid="all", lse=False):
    return dict(name=name, op="cross_attention", dtype=dtype, N=N, Tq=Tq, Tk=Tk, Hq=Hq, Hkv=Hkv, D=D, valid=valid,
                lse=lse)


def _norm(name, dtype, Mq, Mk, Hq, Hkv, D, rot, mode, axes, side, rule="none", factor=1.0):
    return dict(name=name, op="qk_norm_rotary", dtype=dtype, Mq=Mq, Mk=Mk, Hq=Hq, Hkv=Hkv, D=D, rot=rot, mode=mode,
                axes=axes, side=side, rule=rule, factor=factor)


def _rot(name, dtype, M, heads, D, rot, mode, axes, side, rule="none", factor=1.0):
    return dict(name=name, op="rotary", dtype=dtype, M=M, heads=heads, D=D, rot=rot, mode=mode, axes=axes, side=side,
                rule=rule, factor=factor)


def listed():
    return [
        # one token of one caption over a small 24 x 40 map: launch latency
        _attn("token_small_map", "bf16", 1, 1, 24 * 40, 4, 4, 64),
        # one new token for each of 32 captions, 56 x 56 maps of different valid lengths (one with none),
        # four query heads to a key head
        _attn("token_batch_lengths", "bf16", 32, 1, 56 * 56, 16, 4, 64, valid="lengths"),
        # one token over every pixel of a 1280 x 720 map, one key head for four query heads
        _attn("token_whole_image", "bf16", 1, 1, 1280 * 720, 4, 1, 64, lse=True),
        # three tokens (a short draft) over 128 x 128 maps in fp32, as conv2d_fwd writes them
        _attn("draft_fp32", "f32", 8, 3, 128 * 128, 4, 4, 32),
        # 77-token prompts over 56 x 56 maps, each padded to the batch's size on the right and below
        _attn("prompt_masked_maps", "bf16", 32, 77, 56 * 56, 8, 8, 64, valid="mask"),
        # 128 x 128 pixels of four images attending to the states of 1280 x 720 / 16: the arithmetic-bound case
        _attn("pixels_to_states", "bf16", 4, 128 * 128, 80 * 45, 16, 16, 128),
        # an odd number of fp32 queries over 56 x 56 maps, four query heads to a key head
        _attn("prompt_fp32", "f32", 2, 1001, 56 * 56, 8, 2, 64, lse=True),
        # the decode step's queries and keys of four sequences: launch latency
        _norm("norm_rotary_step", "bf16", 4, 4, 16, 4, 64, 64, "half", 1, 4096),
        # prompts' queries and 56 x 56 maps' keys, rows and columns as the two position axes
        _norm("norm_rotary_maps", "bf16", 32 * 77, 32 * 56 * 56, 8, 8, 64, 64, "half", 2, 56),
        # a large fp32 batch, interleaved pairs, half of the head rotated
        _norm("norm_rotary_fp32", "f32", 4 * 128 * 128, 4 * 80 * 45, 16, 16, 128, 64, "interleaved", 1, 16384),
        # part of an 80-wide head, a 77-token prompt
        _rot("rotary_prompt", "bf16", 77, 12, 80, 32, "interleaved", 1, 128),
        # a long context with frequencies scaled by 8 in bands
        _rot("rotary_long", "bf16", 131072, 8, 128, 128, "half", 1, 131072, rule="bands", factor=8.0),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_ATTN_FLOPS_MAX = {"bf16": 1.5e12, "f32": 2.0e11}
_ATTN_BYTES_MAX = 4e8
_ROW_BYTES_MAX = 8e8


def draw(rng):
    op = rng.choice(["cross_attention", "cross_attention", "qk_norm_rotary", "rotary"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "cross_attention":
        while True:
            D = rng.choice([24, 32, 40, 64, 64, 80, 96, 128, 128])
            Hkv = rng.choice([1, 2, 3, 4, 8])
            Hq = Hkv * rng.choice([1, 1, 2, 4, 5])
            N = _logint(rng, 1, 32)
            Tq = rng.choice([1, 1, _logint(rng, 2, 16), _logint(rng, 17, 16384), _logint(rng, 17, 16384)])
            Tk = _logint(rng, 16, 1280 * 720)
            case = _attn("", dtype, N, Tq, Tk, Hq, Hkv, D, valid=rng.choice(["all", "lengths", "mask"]),
                         lse=rng.random() < 0.5)
            w = work(dict(case, valid="all"))
            if w["flops"] <= _ATTN_FLOPS_MAX[dtype] and w["bytes"] <= _ATTN_BYTES_MAX:
                break
    else:
        while True:
            D = rng.choice([32, 64, 64, 80, 96, 128, 128, 256])
            axes = rng.choice([1, 1, 2])
            rot = 8 * axes * rng.randint(1, D // (8 * axes))
            rot = rng.choice([rot, D // (8 * axes) * 8 * axes])
            mode = rng.choice(["half", "interleaved"])
            rule = rng.choice(["none", "linear", "ntk", "bands"]) if axes == 1 and rot > 8 else "none"
            factor = 1.0 if rule == "none" else rng.choice([2.0, 4.0, 8.0])
            side = _logint(rng, 16, 131072) if axes == 1 else _logint(rng, 8, 1280)
            heads = rng.choice([1, 2, 3, 4, 8, 12, 16, 32])
            if op == "rotary":
                case = _rot("", dtype, _logint(rng, 1, 200000), heads, D, rot, mode, axes, side, rule, factor)
            else:
                kv = rng.choice([h for h in (1, 2, 3, 4, 8) if heads % h == 0])
                case = _norm("", dtype, _logint(rng, 1, 100000), _logint(rng, 1, 100000), heads, kv, D, rot, mode,
                             axes, side, rule, factor)
            if work(case)["bytes"] <= _ROW_BYTES_MAX:
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


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, gain=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * gain).to(dt)

    x = {}
    if case["op"] == "cross_attention":
        N, Tq, Tk, Hq, Hkv, D = (case[n] for n in ("N", "Tq", "Tk", "Hq", "Hkv", "D"))
        # normalised heads, the queries' learned gain making the weights uneven
        x["q"] = normal(N, Tq, Hq, D, gain=2.0)
        x["k"] = normal(N, Tk, Hkv, D)
        x["v"] = normal(N, Tk, Hkv, D)
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
        return x
    parts = [("q", case["Mq"], case["Hq"]), ("k", case["Mk"], case["Hkv"])] if case["op"] == "qk_norm_rotary" else \
        [("x", case["M"], case["heads"])]
    for name, M, heads in parts:
        x[name] = normal(M, heads, case["D"], gain=1.5)
        # one axis: a position for each token; two: the row and the column of a side x side map
        x[name + "_pos"] = torch.randint(0, case["side"], (case["axes"], M), generator=g, device=dev,
                                         dtype=torch.int32)
        if case["op"] == "qk_norm_rotary":
            x[name + "_weight"] = 1.0 + 0.2 * torch.randn(case["D"], generator=g, device=dev)
    return x


_BASE = 10000.0
_EPS = 1e-6
_LOW_TURNS, _HIGH_TURNS = 1.0, 32.0


def _frequencies(case):
    """The rotation's radians per position of each pair of one axis, in 64
    bits, and the factor on cos and sin (the scaling rules' definitions)."""
    pairs = case["rot"] // (2 * case["axes"])
    base, s = _BASE, case["factor"]
    if case["rule"] == "ntk":
        base = base * s ** (pairs / (pairs - 1.0))
    f = torch.tensor([base ** (-i / pairs) for i in range(pairs)], dtype=torch.float64)
    magnitude = 1.0
    if case["rule"] == "linear":
        f = f / s
    elif case["rule"] == "bands":
        # pairs that turn often over the original length keep their frequency,
        # those that turn less than once are stretched
        turns = case["side"] / s * f / (2.0 * math.pi)
        keep = ((turns - _LOW_TURNS) / (_HIGH_TURNS - _LOW_TURNS)).clamp(0.0, 1.0)
        f = f * keep + f / s * (1.0 - keep)
        magnitude = 0.1 * math.log(s) + 1.0
    return f, magnitude


def prepare(case, seed):
    state = {"case": case}
    state.update(_inputs(case, seed))
    dev = torch.device("cuda")
    if case["op"] == "cross_attention":
        state["scale"] = case["D"] ** -0.5
        if own:
            state["out"] = torch.empty_like(state["q"])
            state["lse"] = torch.empty(case["N"], case["Hq"], case["Tq"], device=dev) if case["lse"] else None
    else:
        pairs = case["rot"] // (2 * case["axes"])
        if own:
            import stencil_conv2d_fwd_gb300 as sc
            rule = {"none": sc.SC_ROT_SCALE_NONE, "linear": sc.SC_ROT_SCALE_LINEAR, "ntk": sc.SC_ROT_SCALE_NTK,
                    "bands": sc.SC_ROT_SCALE_BANDS}[case["rule"]]
            state["table"] = torch.empty(case["side"], pairs, 2, device=dev)
            sc.check(sc.rotary_table_fwd(state["table"], case["side"], pairs, _BASE, rule, case["factor"],
                                         case["side"] / case["factor"]), "rotary_table_fwd")
            for name in ("q", "k", "x"):
                if name in state:
                    state[name + "_out"] = torch.empty_like(state[name])
        else:
            f, magnitude = _frequencies(case)
            angle = torch.arange(case["side"], dtype=torch.float64, device=dev).view(-1, 1) * f.to(dev)
            state["cos"] = (angle.cos() * magnitude).float()
            state["sin"] = (angle.sin() * magnitude).float()
    if own:
        import stencil_conv2d_fwd_gb300 as sc
        sc.load()
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plain_attention(st):
    c = st["case"]
    N, Tq, Tk, Hq, Hkv, D = (c[n] for n in ("N", "Tq", "Tk", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    valid = None
    if st["k_len"] is not None:
        valid = torch.arange(Tk, device=st["q"].device).view(1, Tk) < st["k_len"].view(N, 1)
    elif st["key_mask"] is not None:
        valid = st["key_mask"] != 0
    out = torch.empty_like(st["q"])
    lse = torch.empty(N, Hq, Tq, device=out.device)
    # as many sequences, then as many queries, as keep the scores under 4 GB
    nb = max(1, min(N, int(1e9 // max(1, Hq * Tq * Tk))))
    tb = max(1, min(Tq, int(1e9 // (nb * Hq * Tk))))
    for n in range(0, N, nb):
        k = st["k"][n:n + nb].float().permute(0, 2, 3, 1)                     # [n][Hkv][D][Tk]
        v = st["v"][n:n + nb].float().permute(0, 2, 1, 3)                     # [n][Hkv][Tk][D]
        b = k.shape[0]
        for t in range(0, Tq, tb):
            q = st["q"][n:n + nb, t:t + tb].float()
            m = q.shape[1]
            q = q.view(b, m, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(b, Hkv, G * m, D)
            s = torch.matmul(q, k).mul_(st["scale"])
            if valid is not None:
                s.masked_fill_(~valid[n:n + nb].view(b, 1, 1, Tk), float("-inf"))
            top = s.amax(dim=-1, keepdim=True)
            top = torch.where(torch.isinf(top), torch.zeros_like(top), top)   # rows with no valid key
            p = s.sub_(top).exp_()
            total = p.sum(dim=-1, keepdim=True)
            o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
            out[n:n + nb, t:t + tb] = o.view(b, Hkv, G, m, D).permute(0, 3, 1, 2, 4).reshape(b, m, Hq, D).to(out.dtype)
            lse[n:n + nb, :, t:t + tb] = (top + total.log()).view(b, Hq, m)
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


def _plain_rotate(y, pos, st):
    """y [M][heads][D] in 32 bits, rotated by the tables' rows at pos [axes][M]."""
    c = st["case"]
    rot = c["rot"]
    cos = torch.cat([st["cos"][p] for p in pos.long()], dim=-1).unsqueeze(1)   # [M][1][rot / 2]
    sin = torch.cat([st["sin"][p] for p in pos.long()], dim=-1).unsqueeze(1)
    if c["mode"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], dim=-1)


def run(state):
    c = state["case"]
    if own:
        import stencil_conv2d_fwd_gb300 as sc
        dt = sc.SC_BF16 if c["dtype"] == "bf16" else sc.SC_F32
        if c["op"] == "cross_attention":
            sc.check(sc.cross_attention_fwd(state["q"], state["k"], state["v"], state["out"], c["N"], c["Tq"], c["Tk"],
                                            c["Hq"], c["Hkv"], c["D"], state["scale"], dt, k_len=state["k_len"],
                                            key_mask=state["key_mask"], lse=state["lse"]), "cross_attention_fwd")
            return {"out": state["out"], "lse": state["lse"]} if c["lse"] else {"out": state["out"]}
        mode = sc.SC_ROT_HALF if c["mode"] == "half" else sc.SC_ROT_INTERLEAVED
        if c["op"] == "rotary":
            sc.check(sc.rotary_fwd(state["x"], state["x_out"], state["table"], state["x_pos"], c["M"], c["heads"],
                                   c["D"], c["rot"], c["side"], mode, c["axes"], dtype=dt), "rotary_fwd")
            return {"x": state["x_out"]}
        sc.check(sc.qk_norm_rotary_fwd(
            (state["q"], state["q_out"], state["q_weight"], state["q_pos"], c["Mq"], c["Hq"]),
            (state["k"], state["k_out"], state["k_weight"], state["k_pos"], c["Mk"], c["Hkv"]),
            state["table"], c["D"], c["rot"], c["side"], _EPS, mode, c["axes"], dtype=dt), "qk_norm_rotary_fwd")
        return {"q": state["q_out"], "k": state["k_out"]}
    if c["op"] == "cross_attention":
        return _plain_attention(state)
    if c["op"] == "rotary":
        return {"x": _plain_rotate(state["x"].float(), state["x_pos"], state).to(state["x"].dtype)}
    out = {}
    for n in ("q", "k"):
        x = state[n].float()
        y = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + _EPS) * state[n + "_weight"]
        out[n] = _plain_rotate(y, state[n + "_pos"], state).to(state[n].dtype)
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its exact result
# ---------------------------------------------------------------------------
def work(case):
    e = _SIZE[case["dtype"]]
    if case["op"] == "cross_attention":
        N, Tq, Tk, Hq, Hkv, D = (case[n] for n in ("N", "Tq", "Tk", "Hq", "Hkv", "D"))
        keys, extra = N * Tk, 0
        if case["valid"] == "lengths":
            keys, extra = sum(_lengths(case)), 4 * N
        elif case["valid"] == "mask":
            keys, extra = sum(h * w for h, w in _map_sides(case)[2]), N * Tk
        nbytes = e * D * (2 * N * Tq * Hq + 2 * keys * Hkv) + extra + (4 * N * Hq * Tq if case["lse"] else 0)
        return {"bytes": nbytes, "flops": 4 * Tq * Hq * D * keys}
    parts = [(case["Mq"], case["Hq"]), (case["Mk"], case["Hkv"])] if case["op"] == "qk_norm_rotary" else \
        [(case["M"], case["heads"])]
    nbytes = flops = 0
    norm = case["op"] == "qk_norm_rotary"
    for M, heads in parts:
        # rows of the table: each is read at least once where the tokens cover it
        rows = min(M * case["axes"], case["side"])
        nbytes += M * (2 * heads * case["D"] * e + 4 * case["axes"]) + (4 * case["D"] if norm else 0)
        nbytes += rows * 8 * (case["rot"] // (2 * case["axes"])) // len(parts)
        flops += M * heads * (3 * case["rot"] + (4 * case["D"] if norm else 0))
    return {"bytes": nbytes, "flops": flops}


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
            k = x["k"][n, keep, h * Hkv // Hq].double()
            v = x["v"][n, keep, h * Hkv // Hq].double()
            for t in range(0, Tq, step):
                s = x["q"][n, t:t + step, h].double() @ k.t() / math.sqrt(D)
                z = torch.logsumexp(s, dim=1)
                out[n, t:t + step, h] = torch.exp(s - z[:, None]) @ v
                lse[n, h, t:t + step] = z
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _exact_rows(case, v, pos, weight):
    """Pairs as complex numbers, turned by e^(i angle)."""
    v = v.double()
    if weight is not None:
        v = v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / case["D"] + _EPS) * weight.double()
    rot, half = case["rot"], case["rot"] // 2
    f, magnitude = _frequencies(case)
    f = f.to(v.device)
    angle = torch.cat([pos[a].double()[:, None] * f[None, :] for a in range(case["axes"])], dim=1)
    turn = torch.polar(torch.full_like(angle, magnitude), angle)[:, None, :]
    if case["mode"] == "half":
        z = torch.complex(v[:, :, :half].contiguous(), v[:, :, half:rot].contiguous()) * turn
        v[:, :, :half], v[:, :, half:rot] = z.real, z.imag
    else:
        z = torch.view_as_complex(v[:, :, :rot].reshape(v.shape[0], v.shape[1], half, 2).contiguous()) * turn
        v[:, :, :rot] = torch.view_as_real(z).reshape(v.shape[0], v.shape[1], rot)
    return v


def exact(case, seed):
    x = _inputs(case, seed)
    if case["op"] == "cross_attention":
        return _exact_attention(case, x)
    if case["op"] == "rotary":
        return {"x": _exact_rows(case, x["x"].clone(), x["x_pos"], None)}
    return {n: _exact_rows(case, x[n].clone(), x[n + "_pos"], x[n + "_weight"]) for n in ("q", "k")}
