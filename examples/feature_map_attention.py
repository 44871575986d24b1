#!/usr/bin/env python3
"""Queries that look at an image: convolutions, heads, attention.

A small convolutional encoder turns an image into a feature map; two 1x1
convolutions of the map are the keys and values of its H * W states, used as
they lie in memory ([N][H][W][heads * D] is [N][H * W][heads][D]).  Queries
(tokens of a decoder, or points of interest, each with a place in the image)
and keys are normalised per head and rotated by their row and column, and the
queries attend to the map.  A later step with new queries keeps the map's keys
and values.

    python examples/feature_map_attention.py [--dtype bf16] [--size 720x1280]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import stencil_conv2d_fwd_gb300 as sc  # noqa: E402

HEADS, KEY_HEADS, D = 8, 2, 64      # four query heads share a key head
FEATURES = 32


def make_weights(seed=0, device="cuda"):
    g = torch.Generator().manual_seed(seed)

    def conv(cout, cin, k):
        return (torch.randn(cout, cin, k, k, generator=g) * (2.0 / (cin * k * k)) ** 0.5).to(device)

    return {
        "conv1": conv(FEATURES, 1, 5), "conv2": conv(FEATURES, FEATURES, 3),
        "key": conv(KEY_HEADS * D, FEATURES, 1), "value": conv(KEY_HEADS * D, FEATURES, 1),
        "bias": torch.zeros(max(FEATURES, KEY_HEADS * D), device=device),
        "query_norm": torch.ones(D, device=device) * 1.5, "key_norm": torch.ones(D, device=device),
    }


class FeatureMap:
    """Keys and values of N images [N][H][W] (fp32), padded to one size: valid[n] = (height, width)."""

    def __init__(self, images, weights, valid=None, dtype=sc.SC_F32):
        N, H, W = images.shape
        dev, t = images.device, torch.bfloat16 if dtype == sc.SC_BF16 else torch.float32
        self.N, self.H, self.W, self.dtype, self.weights = N, H, W, dtype, weights
        w, b = weights, weights["bias"]
        x = torch.empty(N, H, W, FEATURES, device=dev)
        y = torch.empty_like(x)
        sc.check(sc.conv2d_fwd(images, w["conv1"], b, x, N, H, W, 1, FEATURES, 5, 5, act=sc.SC_ACT_RELU), "conv1")
        sc.check(sc.conv2d_fwd(x, w["conv2"], b, y, N, H, W, FEATURES, FEATURES, 3, 3, act=sc.SC_ACT_RELU), "conv2")
        self.k, self.v = (torch.empty(N, H, W, KEY_HEADS * D, device=dev, dtype=t) for _ in range(2))
        if dtype == sc.SC_BF16:
            y = y.bfloat16()
        for out, name in ((self.k, "key"), (self.v, "value")):
            if dtype == sc.SC_BF16:
                rc = sc.conv2d_fwd_tc_bf16(y, w[name], b, out, N, H, W, FEATURES, KEY_HEADS * D, 1, 1)
            else:
                rc = sc.conv2d_fwd(y, w[name], b, out, N, H, W, FEATURES, KEY_HEADS * D, 1, 1)
            sc.check(rc, name)
        # a pixel's two positions, and the rotation's table of the longer side
        side = max(H, W)
        rows = torch.arange(H, device=dev, dtype=torch.int32).view(H, 1).expand(H, W)
        cols = torch.arange(W, device=dev, dtype=torch.int32).view(1, W).expand(H, W)
        self.pos = torch.stack([p.reshape(1, H * W).expand(N, -1).reshape(-1) for p in (rows, cols)]).contiguous()
        self.side, self.table = side, torch.empty(side, D // 4, 2, device=dev)
        sc.check(sc.rotary_table_fwd(self.table, side, D // 4, base=100.0), "rotary_table_fwd")
        self.mask = None
        if valid is not None:
            hw = torch.tensor(valid, device=dev)
            inside = (rows < hw[:, :1, None]) & (cols < hw[:, 1:, None])
            self.mask = inside.to(torch.uint8).contiguous()
        self._keys_ready = False

    def attend(self, q, places):
        """q [N][T][HEADS][D] (left as it is), places [2][N * T] int32: (row, column) of each query."""
        N, T = q.shape[:2]
        qn, out = torch.empty_like(q), torch.empty_like(q)
        states = self.N * self.H * self.W
        w = self.weights
        queries = (q, qn, w["query_norm"], places, N * T, HEADS)
        # the keys once, in place, in the first queries' launch
        keys = None if self._keys_ready else (self.k, self.k, w["key_norm"], self.pos, states, KEY_HEADS)
        sc.check(sc.qk_norm_rotary_fwd(queries, keys, self.table, D, D, self.side, 1e-6, sc.SC_ROT_HALF, axes=2,
                                       dtype=self.dtype), "qk_norm_rotary_fwd")
        self._keys_ready = True
        sc.check(sc.cross_attention_fwd(qn, self.k, self.v, out, N, T, self.H * self.W, HEADS, KEY_HEADS, D, D ** -0.5,
                                        self.dtype, key_mask=self.mask), "cross_attention_fwd")
        return out


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--dtype", choices=["f32", "bf16"], default="f32")
    ap.add_argument("--size", default="360x640")
    ap.add_argument("--images", type=int, default=2)
    ap.add_argument("--queries", type=int, default=100)
    args = ap.parse_args()
    H, W = (int(s) for s in args.size.split("x"))
    dtype = sc.SC_BF16 if args.dtype == "bf16" else sc.SC_F32
    t = torch.bfloat16 if dtype == sc.SC_BF16 else torch.float32
    g = torch.Generator(device="cuda").manual_seed(1)
    images = torch.rand(args.images, H, W, device="cuda", generator=g)
    valid = [(H - 8 * i, W - 16 * i) for i in range(args.images)]
    fmap = FeatureMap(images, make_weights(), valid, dtype)
    for T in (args.queries, 1, 1):      # points of interest, then single tokens
        q = torch.randn(args.images, T, HEADS, D, device="cuda", generator=g).to(t)
        places = torch.stack([torch.randint(0, s, (args.images * T,), device="cuda", generator=g, dtype=torch.int32)
                              for s in (H, W)])
        out = fmap.attend(q, places)
        sc.check(sc.sc_last_device_status(), "device status")
        print(f"{T} queries an image over {H} x {W} states: out {tuple(out.shape)}, rms {out.float().pow(2).mean().sqrt():.4f}")


if __name__ == "__main__":
    main()
