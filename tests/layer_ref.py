"""Plain 64-bit forms of the decoder layer's operators (torch, float64) and the bounds their tests use.

U = 2^-24 is fp32's unit roundoff, UB = 2^-8 bf16's.  Sums of n terms rounded to
nearest are bounded by 6 sqrt(n) U (errors of random sign, six standard
deviations); sums inside the tensor cores are cut short, each by up to 2 U of the
running sum."""
import math

import torch

U = 2.0 ** -24
UB = 2.0 ** -8
ACT_NONE, ACT_RELU, ACT_GELU, ACT_SILU = range(4)


def activate(v, act):
    if act == ACT_RELU:
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == ACT_GELU:
        return v * torch.special.ndtr(v)
    return v * torch.sigmoid(v) if act == ACT_SILU else v


def linear(x, w, b, residual, act):
    """Returns y, and for the bound the sum of |x w| + |b| of each element and |act(v)|."""
    x, w = x.double(), w.double()
    v, mag = x @ w.t(), x.abs() @ w.abs().t()
    if b is not None:
        v, mag = v + b.double(), mag + b.double().abs()
    a = activate(v, act)
    return (a if residual is None else a + residual.double()), mag, a.abs()


def linear_bound(y, mag, a, K, bf16):
    """The product's error: fp32 in tiles of at most 256 elements of K summed on
    the tensor cores (16 products at a time) and these to nearest, bf16 the whole of
    K on the tensor cores.  An activation passes it on times 1.13 at most (the largest
    slope of gelu and silu), and is itself good to 8 U of its value and, where 1 + erf
    cancels, of U times its argument's size."""
    steps = min(K, 256) / 16 if not bf16 else K / 16
    e = 1.13 * mag * U * (2 * steps + 6 * math.sqrt(K) + 8) + U * (8 * a + 2 * mag + 2 * y.abs()) + 1e-37
    return e + UB * y.abs() if bf16 else e


def normed(v, kind, weight, bias, eps):
    """Returns the norm of the rows of v and, for the bound, the size of its terms."""
    if kind == 0:
        return v, v.abs()
    mag = v.abs()
    if kind == 2:
        mean = v.mean(dim=-1, keepdim=True)
        mag = mag + v.abs().mean(dim=-1, keepdim=True)
        v = v - mean
    r = 1 / torch.sqrt(v.pow(2).mean(dim=-1, keepdim=True) + eps)
    v, mag = v * r, mag * r
    if weight is not None:
        v, mag = v * weight.double(), mag * weight.double().abs()
    if bias is not None:
        v, mag = v + bias.double(), mag + bias.double().abs()
    return v, mag


def quantize(x, valid, block, e4m3):
    """x [N][T][H][D] (any float type), valid [N][T] bool: codes as float64 values, scales [N][H][blocks]
    (NaN where a block has no valid state, codes NaN where a state is not valid)."""
    N, T, H, D = x.shape
    top = 448.0 if e4m3 else 127.0
    nb = -(-T // block)
    y = torch.zeros(N, nb * block, H, D, dtype=torch.float64, device=x.device)
    ok = torch.zeros(N, nb * block, dtype=torch.bool, device=x.device)
    y[:, :T] = torch.where(valid[:, :, None, None], x.double(), torch.zeros((), dtype=torch.float64, device=x.device))
    ok[:, :T] = valid
    y = y.view(N, nb, block, H, D)
    a = y.abs().amax(dim=(2, 4))                                         # [N][nb][H]
    a = torch.where(y.isfinite().all(dim=4).all(dim=2), a, torch.full_like(a, math.nan))
    scale = (a / top).float().double()   # rounded once
    q = y * top / torch.where(a > 0, a, torch.ones_like(a))[:, :, None, :, None]
    if e4m3:
        # spacing of the codes at |q|, 2^(exponent - 4), made of its bits (a power by pow may be off by a little)
        step = ((torch.frexp(q).exponent.clamp(min=-5).long() + 1019) << 52).view(torch.float64)
        code = (q / step).round() * step
    else:
        code = q.round()
    code = torch.where(a.isnan()[:, :, None, :, None], torch.zeros_like(code), code).view(N, nb * block, H, D)[:, :T]
    code = torch.where(valid[:, :, None, None], code, torch.full_like(code, math.nan))
    any_valid = ok.view(N, nb, block).any(dim=2)
    none = torch.full_like(scale, math.inf)   # inf: left as it was
    scale = torch.where(any_valid[:, :, None], scale, none)
    return code, scale.transpose(1, 2).contiguous()


def dequantize(codes, scale, block):
    """codes [N][T][H][D] as values, scale [N][H][blocks] -> float64 states."""
    T = codes.shape[1]
    s = scale.double().transpose(1, 2).repeat_interleave(block, dim=1)[:, :T]
    return codes.double() * s.unsqueeze(-1)


def attention(q, k, v, scale, valid):
    """q [N][Tq][Hq][D], k and v [N][Tk][Hkv][D] in float64, valid [N][Tk] bool: out, lse,
    sum_j p_j |v_j| / sum p and the largest sum of |scale q k| of each row."""
    N, Tq, Hq, D = q.shape
    G = Hq // k.shape[2]
    kk, vv = (torch.where(valid[:, :, None, None], t, torch.zeros_like(t)).repeat_interleave(G, dim=2).transpose(1, 2)
              for t in (k, v))
    s = scale * (q.transpose(1, 2) @ kk.transpose(2, 3))
    mag = scale * (q.abs().transpose(1, 2) @ kk.abs().transpose(2, 3)).amax(dim=-1)
    s = s.masked_fill(~valid[:, None, None, :], -math.inf)
    lse = torch.logsumexp(s, dim=-1)
    p = torch.exp(s - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[..., None])
    out, wabs = (p @ vv).transpose(1, 2), (p @ vv.abs()).transpose(1, 2)
    return out, lse, wabs, mag
