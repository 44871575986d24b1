"""The feature-map example end to end against the plain 64-bit forms."""
import os
import sys

import numpy as np
import pytest

import attention_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
@pytest.mark.parametrize("bf16", [False, True])
def test_feature_map_attention(sc, oracle_mod, bf16):
    import torch
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import feature_map_attention as ex
    N, H, W, T = 2, 24, 40, 9
    g = torch.Generator().manual_seed(3)
    images = torch.rand(N, H, W, generator=g)
    valid = [(24, 31), (17, 40)]
    weights = ex.make_weights()
    dtype, t = (sc.SC_BF16, torch.bfloat16) if bf16 else (sc.SC_F32, torch.float32)
    fmap = ex.FeatureMap(images.cuda(), weights, valid, dtype)
    # the keys and values as the convolutions wrote them, from the oracle
    w = {k: v.cpu().numpy() for k, v in weights.items()}
    x, _ = oracle_mod.conv2d_nchw(images.numpy()[:, None], w["conv1"], w["bias"][:32], 1)
    y, _ = oracle_mod.conv2d_nchw(x.astype(np.float32), w["conv2"], w["bias"][:32], 1)
    for name, got in (("key", fmap.k), ("value", fmap.v)):
        want, _ = oracle_mod.conv2d_nchw(y.astype(np.float32), w[name], w["bias"][:128], 0)
        want = want.transpose(0, 2, 3, 1)
        err = np.abs(got.float().cpu().numpy() - want).max()
        assert err <= (2.0 ** -6 if bf16 else 1e-4) * np.abs(want).max()
    k0, v0 = (a.float().cpu().numpy().astype(np.float64).reshape(N, H * W, ex.KEY_HEADS, ex.D) for a in (fmap.k, fmap.v))
    f, _ = ref.frequencies(ex.D // 4, 100.0)
    mask = fmap.mask.cpu().numpy().reshape(N, H * W) != 0
    assert mask.sum(axis=1).tolist() == [24 * 31, 17 * 40]
    pos = fmap.pos.cpu().numpy()
    k, _ = ref.rotate(ref.rms_norm(k0, w["key_norm"].astype(np.float64), 1e-6).reshape(-1, ex.KEY_HEADS, ex.D), pos, ex.D, 0,
                      2, f)
    for step, n in enumerate((T, 1)):      # the second step keeps the keys
        q = torch.randn(N, n, ex.HEADS, ex.D, generator=g).to(t)
        places = torch.stack([torch.randint(0, s, (N * n,), generator=g, dtype=torch.int32) for s in (H, W)])
        out = fmap.attend(q.cuda(), places.cuda())
        sc.check(sc.sc_last_device_status())
        qn, _ = ref.rotate(ref.rms_norm(q.double().numpy(), w["query_norm"].astype(np.float64), 1e-6)
                           .reshape(-1, ex.HEADS, ex.D), places.numpy(), ex.D, 0, 2, f)
        want, _, wabs, _ = ref.attention(qn.reshape(N, n, ex.HEADS, ex.D), k.reshape(N, H * W, ex.KEY_HEADS, ex.D), v0,
                                         ex.D ** -0.5, mask)
        # bf16: rounded queries and keys move a score by 2^-8 of its size (up to 12 here) twice over, on top of the
        # weights' and the output's rounding; fp32: the scores' own bound
        rel = 2 * 2 * 12 * 2.0 ** -8 / 4 + 2 * 2.0 ** -8 if bf16 else 1e-4
        assert (np.abs(out.float().cpu().numpy() - want) <= rel * wabs + 1e-6).all()
