"""Attention over the pixels of a deformable layer's feature maps, trained for a
few steps, then a short sequence of new tokens read from the maps.

    python examples/feature_map_attention.py [--steps 20]

Two images of different size go through a modulated deformable convolution
each; their pixels become the tokens of one packed batch. A linear layer makes
queries, keys and values in one tensor, whose slices are normed per head and
rotated by the pixels' rows and columns, and attend within their image. The
gradients run back through all of it, and the linear layers, the norms' weights
and the convolution's weight take plain gradient steps towards a random target.
At the end one new token at a time attends to the pixels of its image and to the
tokens before it, kept in a cache with room for more.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import modulated_deformable_convolution_gb300 as mdcn  # noqa: E402

CHANNELS, Q_HEADS, K_HEADS, DIM = 64, 4, 2, 64
SIZES = [(32, 32), (20, 28)]
SECTIONS = (16, 16)  # half of each head's pairs turn with the row, half with the column


class Model:
    def __init__(self, seed=0, dtype=torch.bfloat16):
        g = torch.Generator().manual_seed(seed)
        new = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(dtype).cuda()  # noqa: E731
        self.images = [new(1, CHANNELS, h, w) for h, w in SIZES]
        self.offsets = [new(1, 18, h, w) for h, w in SIZES]
        self.masks = [torch.sigmoid(new(1, 9, h, w)) for h, w in SIZES]
        heads = Q_HEADS + 2 * K_HEADS
        self.p = {"conv": new(CHANNELS, CHANNELS, 3, 3, scale=(CHANNELS * 9) ** -0.5),
                  "qkv": new(CHANNELS, heads * DIM, scale=CHANNELS**-0.5),
                  "proj": new(Q_HEADS * DIM, CHANNELS, scale=(Q_HEADS * DIM) ** -0.5),
                  "q_norm": torch.ones(DIM, dtype=dtype, device="cuda"),
                  "k_norm": torch.ones(DIM, dtype=dtype, device="cuda")}
        lengths = [h * w for h, w in SIZES]
        self.starts = mdcn.sequence_starts(lengths)
        self.positions = torch.cat([torch.cartesian_prod(torch.arange(h), torch.arange(w)) for h, w in SIZES]).int().cuda()
        self.freq = mdcn.rotary_frequencies(SECTIONS)
        self.target = new(sum(lengths), CHANNELS)

    def rotary_args(self):
        return dict(norm=True, q_weight=self.p["q_norm"], k_weight=self.p["k_norm"])

    def forward(self):
        """Outputs of every step that the gradients need."""
        maps = [mdcn.forward(x, o, m, self.p["conv"], padding=1) for x, o, m in zip(self.images, self.offsets, self.masks)]
        tokens = torch.cat([y[0].flatten(1).T for y in maps])
        qkv = (tokens @ self.p["qkv"]).view(len(tokens), -1, DIM)
        q, k, v = qkv.split([Q_HEADS, K_HEADS, K_HEADS], 1)
        qr, kr = mdcn.rotary(q, k, self.positions, self.freq, SECTIONS, **self.rotary_args())
        out, lse = mdcn.attention(qr, kr, v, self.starts, self.starts)
        return dict(tokens=tokens, q=q, k=k, v=v, qr=qr, kr=kr, out=out, lse=lse, y=out.flatten(1) @ self.p["proj"])

    def backward(self, s):
        """Gradients of mean((y - target)^2) / 2."""
        gy = ((s["y"].float() - self.target.float()) / s["y"].numel()).to(s["y"].dtype) * 1024  # kept in range, undone below
        g = {"proj": s["out"].flatten(1).T @ gy}
        ga = mdcn.attention_backward((gy @ self.p["proj"].T).view_as(s["out"]), s["qr"], s["kr"], s["v"], s["out"], s["lse"], self.starts, self.starts)
        gr = mdcn.rotary_backward(ga["q"], ga["k"], s["q"], s["k"], self.positions, self.freq, SECTIONS, **self.rotary_args())
        g["q_norm"], g["k_norm"] = gr["q_weight"], gr["k_weight"]
        gqkv = torch.cat([gr["q"], gr["k"], ga["v"]], 1).flatten(1)
        g["qkv"] = s["tokens"].T @ gqkv
        gtokens = gqkv @ self.p["qkv"].T
        g["conv"], at = 0, 0
        for x, o, m in zip(self.images, self.offsets, self.masks):
            h, w = x.shape[2:]
            gmap = gtokens[at:at + h * w].T.reshape(1, CHANNELS, h, w).contiguous()
            g["conv"] = g["conv"] + mdcn.backward(x, o, m, self.p["conv"], gmap, with_bias=False, padding=1)["weight"]
            at += h * w
        return {n: t.float() / 1024 for n, t in g.items()}

    def step(self, rate):
        s = self.forward()
        loss = float((s["y"].float() - self.target.float()).square().mean()) / 2
        for n, g in self.backward(s).items():
            self.p[n] = (self.p[n].float() - rate * g).to(self.p[n].dtype)
        return loss

    def read(self, count):
        """`count` new tokens for each image, one at a time."""
        s = self.forward()
        room = max(h * w for h, w in SIZES) + count
        k = torch.zeros(len(SIZES) * room, K_HEADS, DIM, dtype=s["kr"].dtype, device="cuda")
        v, lengths = torch.zeros_like(k), [h * w for h, w in SIZES]
        for b, n in enumerate(lengths):
            first = int(self.starts[b])
            k[b * room:b * room + n], v[b * room:b * room + n] = s["kr"][first:first + n], s["v"][first:first + n]
        starts, ones = mdcn.sequence_starts([room] * len(SIZES)), mdcn.sequence_starts([1] * len(SIZES))
        token, outs = torch.stack([s["y"][int(self.starts[b])] for b in range(len(SIZES))]), []
        for i in range(count):
            q, kn, vn = (token @ self.p["qkv"]).view(len(SIZES), -1, DIM).split([Q_HEADS, K_HEADS, K_HEADS], 1)
            place = torch.tensor([[h, i] for h, _ in SIZES], dtype=torch.int32, device="cuda")  # a line below the image
            qr, kr = mdcn.rotary(q, kn, place, self.freq, SECTIONS, **self.rotary_args())
            at = torch.tensor([b * room + n + i for b, n in enumerate(lengths)], device="cuda")
            k[at], v[at] = kr, vn
            used = torch.tensor([n + i + 1 for n in lengths], dtype=torch.int32, device="cuda")
            out, _ = mdcn.attention(qr, k, v, ones, starts, k_lengths=used, causal=True)
            token = out.flatten(1) @ self.p["proj"]
            outs.append(token)
        return torch.stack(outs, 1)


def main(steps=20, rate=50.0):
    model = Model()
    losses = [model.step(rate) for _ in range(steps)]
    tokens = model.read(4)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps; new tokens {tuple(tokens.shape)}")
    return losses, tokens


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    main(ap.parse_args().steps)
