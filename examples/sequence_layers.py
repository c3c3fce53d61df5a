"""A small sequence model from the framework's operators: trained, then decoded token by token.

Two layers, each a residual block over x [B, L, D]:

  convolution layer  q, k, v = x Wq^T, x Wk^T, x Wv^T;  x += (HyenaConv(q, k, v, h)) Wo^T
  recurrence layer   [q k v g] = x W^T + b (one projection, its column slices go in as they are);
                     x += (GatedScan(q, k, v, g)) Wo^T

between an embedding and a readout.  The task is next-token prediction of a
sequence whose second half repeats its first.  Decoding keeps a ring cache of
past rows for the convolution and one state row for the recurrence; a step is a
fixed set of launches, captured once in a HIP graph and replayed for each token.

    python examples/sequence_layers.py [--steps 200] [--width 256]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_convolution_sequence_amd as hc  # noqa: E402

GROUP, TAPS, VOCAB = 16, 24, 32


class Model(torch.nn.Module):
    def __init__(self, width: int, dtype=torch.bfloat16, device="cuda", seed: int = 0):
        super().__init__()
        gen = torch.Generator().manual_seed(seed)

        def new(*shape, scale):
            return torch.nn.Parameter((scale * torch.randn(*shape, generator=gen)).to(device, dtype))

        D = self.width = width
        self.embed = new(VOCAB, D, scale=1.0)
        self.conv_in = torch.nn.ParameterList(new(D, D, scale=D ** -0.5) for _ in range(3))
        self.taps = new(D // GROUP, TAPS, scale=TAPS ** -0.5)
        self.conv_out = new(D, D, scale=D ** -0.5)
        self.scan_in = new(4 * D, D, scale=D ** -0.5)
        bias = torch.zeros(4 * D)
        bias[3 * D:] = torch.linspace(1.0, 6.0, D)  # memories from a few rows to some hundreds
        self.scan_bias = torch.nn.Parameter(bias.to(device, dtype))
        self.scan_out = new(D, D, scale=D ** -0.5)
        self.readout = new(VOCAB, D, scale=0.1 * D ** -0.5)

    def forward(self, tokens):
        """Logits [B, L, VOCAB] of tokens [B, L], with gradients."""
        D, lin = self.width, hc.LinearAct.apply
        x = self.embed[tokens]
        q, k, v = (lin(x, w, None, None, "none") for w in self.conv_in)
        x = lin(hc.HyenaConv.apply(q, k, v, self.taps, GROUP), self.conv_out, None, x, "none")
        z = lin(x, self.scan_in, self.scan_bias, None, "none")
        y, _ = hc.GatedScan.apply(*(z[..., i * D:(i + 1) * D] for i in range(4)))
        x = lin(y, self.scan_out, None, x, "none")
        return lin(x, self.readout, None, None, "none")


class Decoder:
    """The model one token at a time for B sequences."""

    def __init__(self, model: Model, B: int):
        D, dev, dt = model.width, model.embed.device, model.embed.dtype
        self.m, self.B = model, B
        self.ring = torch.zeros(B, TAPS, D, dtype=dt, device=dev)
        self.state = torch.zeros(B, D, device=dev)
        self.pos = torch.zeros(B, dtype=torch.int64, device=dev)
        self.token = torch.zeros(B, dtype=torch.int64, device=dev)
        self.logits = torch.zeros(B, VOCAB, dtype=dt, device=dev)
        self.graph = None

    @torch.no_grad()
    def prefill(self, tokens):
        """Logits of a prompt [B, L]; its last rows and state stay for the steps."""
        m, D = self.m, self.m.width
        lin = lambda x, w, **kw: hc.linear_fwd(x, w, **kw)[0]  # noqa: E731
        x = m.embed[tokens]
        q, k, v = (lin(x, w) for w in m.conv_in)
        hc.conv_cache_fill(k, v, self.ring)
        x = lin(hc.conv_fwd(q, k, v, m.taps, GROUP), m.conv_out, residual=x)
        z = lin(x, m.scan_in, bias=m.scan_bias)
        y, last, _ = hc.scan_fwd(*(z[..., i * D:(i + 1) * D] for i in range(4)))
        self.state.copy_(last)
        self.pos.fill_(tokens.shape[1])
        return lin(lin(y, m.scan_out, residual=x), m.readout)

    def _step(self):
        m, D = self.m, self.m.width
        lin = lambda x, w, **kw: hc.linear_fwd(x, w, **kw)[0]  # noqa: E731
        x = m.embed[self.token]
        q, k, v = (lin(x, w) for w in m.conv_in)
        y = hc.conv_step(q, k, v, m.taps, self.ring, self.pos, GROUP)
        x = lin(y, m.conv_out, residual=x)
        z = lin(x, m.scan_in, bias=m.scan_bias)
        y = hc.scan_step(*(z[:, i * D:(i + 1) * D] for i in range(4)), self.state)
        hc.linear_fwd(lin(y, m.scan_out, residual=x), m.readout, out=self.logits)
        self.pos += 1

    @torch.no_grad()
    def step(self, token):
        """Logits [B, VOCAB] after one more token [B] (the buffer of the next step too)."""
        self.token.copy_(token)
        if self.graph is None:  # capture once, with what the warm-up moved put back
            kept = [t.clone() for t in (self.ring, self.state, self.pos)]
            self._step()
            torch.cuda.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self._step()
            for t, old in zip((self.ring, self.state, self.pos), kept):
                t.copy_(old)
        self.graph.replay()
        return self.logits


def batch(B: int, half: int, gen):
    """Sequences of 2 half tokens whose second half repeats the first."""
    first = torch.randint(0, VOCAB, (B, half), generator=gen)
    return torch.cat([first, first], dim=1)


def train(model: Model, steps: int, B: int = 64, half: int = 8, lr: float = 3e-3, seed: int = 1, log=print):
    gen = torch.Generator().manual_seed(seed)
    # fp32 copies of the weights take the updates
    params = list(model.parameters())
    master = [p.detach().float().clone().requires_grad_(True) for p in params]
    opt = torch.optim.Adam(master, lr=lr)
    losses = []
    for step in range(steps):
        opt.param_groups[0]["lr"] = lr * (1 - step / steps)
        tokens = batch(B, half, gen).to(model.embed.device)
        logits = model(tokens[:, :-1])
        # what can be known: the repeated half
        loss = torch.nn.functional.cross_entropy(logits[:, half - 1:].float().flatten(0, 1),
                                                 tokens[:, half:].flatten())
        model.zero_grad(set_to_none=True)
        loss.backward()
        for m, p in zip(master, params):
            m.grad = p.grad.float()
        torch.nn.utils.clip_grad_norm_(master, 1.0)
        opt.step()
        with torch.no_grad():
            for m, p in zip(master, params):
                p.copy_(m)
        losses.append(loss.item())
        if step % 50 == 0 or step == steps - 1:
            log("step %d loss %.4f" % (step, losses[-1]))
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--width", type=int, default=256)
    args = ap.parse_args()
    model = Model(args.width)
    train(model, args.steps)
    half, B = 8, 16
    tokens = batch(B, half, torch.Generator().manual_seed(99)).cuda()
    dec = Decoder(model, B)
    token = dec.prefill(tokens[:, :half])[:, -1].argmax(-1)
    right = (token == tokens[:, half]).float().mean().item()
    for t in range(half, 2 * half - 1):
        token = dec.step(tokens[:, t]).argmax(-1)
        right += (token == tokens[:, t + 1]).float().mean().item()
    print("decoded tokens right: %.1f%%" % (100 * right / half))


if __name__ == "__main__":
    main()
