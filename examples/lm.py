"""A small language model of selective-scan layers, trained and generating with
the library's operators.

    python examples/lm.py [--steps 200]

Each layer adds to a residual stream kept in fp32:

    y, stream = layer_norm(h, residual=stream)      # the addition and its norm
    x, z, ... = projections of y                    # plain matrix products
    u = causal_conv(x)                              # short convolution + silu
    h = out_proj(selective_scan(u, delta, A, B, C, D, z))

and the model ends in linear_cross_entropy against the embedding, whose logits
are never kept.  Generation runs the prompt once (conv_fwd and scan_fwd return
their states) and then single tokens (norm_fwd, conv_step, decode_step), which
reproduce the prompt pass.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_fwd_gb300 as S  # noqa: E402

BF16 = torch.bfloat16


class Layer(torch.nn.Module):
    def __init__(self, dim: int, inner: int, dstate: int, width: int):
        super().__init__()
        self.inner, self.dstate = inner, dstate

        def weight(rows, cols):
            return torch.nn.Parameter((torch.randn(rows, cols) / cols ** 0.5).to(BF16))

        self.norm_w = torch.nn.Parameter(torch.ones(dim))
        self.in_w = weight(2 * inner, dim)                       # x and the gate z
        self.conv_w = torch.nn.Parameter((torch.rand(inner, width) * 2 - 1) / width ** 0.5)
        self.conv_b = torch.nn.Parameter(torch.zeros(inner))
        self.bc_w = weight(2 * dstate, inner)
        self.dt_w = weight(inner, inner)
        self.dt_b = torch.nn.Parameter(torch.log(torch.expm1(torch.empty(inner).uniform_(1e-3, 1e-1))))
        self.a_log = torch.nn.Parameter(torch.log(torch.arange(1.0, dstate + 1)).repeat(inner, 1))
        self.d = torch.nn.Parameter(torch.ones(inner))
        self.out_w = weight(dim, inner)

    def scan_inputs(self, u):
        """delta, A, B, C of the scan from the convolution's output."""
        delta = F.softplus((u @ self.dt_w.T).float() + self.dt_b).to(BF16)
        b, c = (u @ self.bc_w.T).split(self.dstate, dim=-1)
        return delta, -torch.exp(self.a_log), b.contiguous(), c.contiguous()

    def forward(self, h, stream):
        y, stream = S.layer_norm(h, self.norm_w, residual=stream, rms=True)
        xz = y @ self.in_w.T
        x, z = xz.split(self.inner, dim=-1)                      # x is read in place, strided
        u = S.causal_conv(x, self.conv_w, self.conv_b)
        delta, a, b, c = self.scan_inputs(u)
        h = S.selective_scan(u, delta, a, b, c, self.d, z.contiguous(), chunk_len=64)
        return h @ self.out_w.T, stream

    def prompt(self, h, stream):
        """As forward, keeping the states to generate from."""
        y, stream, _ = S.norm_fwd(h, self.norm_w, residual=stream, rms=True)
        x, z = (y @ self.in_w.T).split(self.inner, dim=-1)
        u, conv_state = S.conv_fwd(x, self.conv_w, self.conv_b, want_final=True)
        delta, a, b, c = self.scan_inputs(u)
        h, _, scan_state = S.scan_fwd(u, delta, a, b, c, self.d, z.contiguous(), want_final=True)
        return h @ self.out_w.T, stream, (conv_state, scan_state)

    def step(self, h, stream, state):
        """One token per sequence; the states and the stream are updated in place."""
        y, stream, _ = S.norm_fwd(h, self.norm_w, residual=stream, rms=True, out_r=stream)
        x, z = (y @ self.in_w.T).split(self.inner, dim=-1)
        u = S.conv_step(x, self.conv_w, self.conv_b, state=state[0])
        delta, a, b, c = self.scan_inputs(u)
        h = S.decode_step(u, delta, a, b, c, self.d, z.contiguous(), state=state[1])
        return h @ self.out_w.T, stream


class Model(torch.nn.Module):
    def __init__(self, vocab=1000, dim=128, layers=2, inner=256, dstate=16, width=4):
        super().__init__()
        self.embed = torch.nn.Parameter((torch.randn(vocab, dim) * 0.05).to(BF16))
        self.layers = torch.nn.ModuleList(Layer(dim, inner, dstate, width) for _ in range(layers))
        self.norm_w = torch.nn.Parameter(torch.ones(dim))

    def start(self, tokens):
        h = F.embedding(tokens, self.embed)
        return h, torch.zeros(h.shape, dtype=torch.float32, device=h.device)

    def loss(self, tokens, targets):
        """The mean cross entropy of targets (-100: no target) after tokens."""
        h, stream = self.start(tokens)
        for layer in self.layers:
            h, stream = layer(h, stream)
        y, _ = S.layer_norm(h, self.norm_w, residual=stream, rms=True)
        return S.linear_cross_entropy(y, self.embed, targets)

    def head(self, h, stream):
        y, _, _ = S.norm_fwd(h, self.norm_w, residual=stream, rms=True)
        return (y @ self.embed.T).float()

    @torch.no_grad()
    def prompt(self, tokens):
        """The logits after every token of the prompt, and the states."""
        h, stream = self.start(tokens)
        states = []
        for layer in self.layers:
            h, stream, state = layer.prompt(h, stream)
            states.append(state)
        return self.head(h, stream), states

    @torch.no_grad()
    def step(self, token, states):
        h, stream = self.start(token)
        for layer, state in zip(self.layers, states):
            h, stream = layer.step(h, stream, state)
        return self.head(h, stream)

    def generate(self, tokens, count):
        logits, states = self.prompt(tokens)
        out = []
        for _ in range(count):
            out.append(logits[:, -1].argmax(-1) if logits.dim() == 3 else logits.argmax(-1))
            logits = self.step(out[-1], states)
        return torch.stack(out, 1)


def batch(rng, rows, length, vocab, device):
    """Sequences that count upward by a step of their own: learnable from context.
    The first targets, which no context determines, are left out of the loss."""
    start = torch.randint(0, vocab, (rows, 1), generator=rng)
    step = torch.randint(1, 4, (rows, 1), generator=rng)
    seq = (start + step * torch.arange(length + 1)) % vocab
    targets = seq[:, 1:].clone()
    targets[:, 0] = -100
    return seq[:, :-1].to(device), targets.to(device)


def train(model, steps, rows=8, length=96, lr=3e-3, seed=0, report=None):
    device = model.embed.device
    rng = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=lr, weight_decay=0.0)
    losses = []
    for i in range(steps):
        tokens, targets = batch(rng, rows, length, model.embed.shape[0], device)
        loss = model.loss(tokens, targets)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if report and (i + 1) % report == 0:
            print(f"step {i + 1}: loss {loss.item():.3f}")
    S.check_device_errors()
    return [v.item() for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=300)
    a = ap.parse_args()
    torch.manual_seed(0)
    model = Model(vocab=200).cuda()
    train(model, a.steps, report=50)
    prompt = torch.tensor([[10, 12, 14, 16, 18, 20], [50, 51, 52, 53, 54, 55]], device="cuda")
    print("prompt", prompt.tolist(), "->", model.generate(prompt, 6).tolist())


if __name__ == "__main__":
    main()
