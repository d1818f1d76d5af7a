"""A small state-space decoder run end to end on the library's operators.

Packed prompts of unequal lengths go through a stack of layers (residual norm in
8 bits, input projection, causal convolution, selective scan, output
projection); the log probabilities read off the last logits choose the next
token, and further tokens are decoded one at a time from the layers' states.
The projections are plain matrix products (torch).

    python examples/state_space_decoder.py [--steps 8]
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bidirectional_lstm_stack_gb300 import binding  # noqa: E402


@dataclass(frozen=True)
class Sizes:
    vocab: int = 1000
    width: int = 256
    channels: int = 512   # of a layer, twice its width
    states: int = 16
    rank: int = 16        # of the step sizes' projection
    taps: int = 4
    layers: int = 4


class Decoder:
    """Random weights; `slots` sequences' states a layer."""

    def __init__(self, sizes: Sizes = Sizes(), slots: int = 8, seed: int = 0,
                 dtype=torch.bfloat16, device: str = "cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        s = sizes

        def normal(*shape, scale=1.0):
            return torch.randn(shape, generator=g, device=device) * scale

        def uniform(*shape):
            return torch.rand(shape, generator=g, device=device)

        self.sizes, self.dtype = sizes, dtype
        self.embedding = normal(s.vocab, s.width).to(dtype)
        self.head = normal(s.width, s.vocab, scale=2.0 * s.width ** -0.5).to(dtype)
        self.final_norm = 0.5 + uniform(s.width)
        self.layers = []
        for _ in range(s.layers):
            step = torch.exp(uniform(s.channels) * 4.6 - 6.9)  # 0.001 to 0.1
            self.layers.append({
                "norm": 0.5 + uniform(s.width),
                "in": normal(s.width, 2 * s.channels, scale=s.width ** -0.5).to(dtype),
                "taps": normal(s.channels, s.taps, scale=s.taps ** -0.5),
                "taps_bias": normal(s.channels, scale=0.1),
                "x": normal(s.channels, s.rank + 2 * s.states, scale=s.channels ** -0.5).to(dtype),
                "dt": normal(s.rank, s.channels, scale=s.rank ** -0.5).to(dtype),
                "dt_bias": step + torch.log(-torch.expm1(-step)),
                "a": -torch.arange(1.0, s.states + 1, device=device).repeat(s.channels, 1),
                "skip": torch.ones(s.channels, device=device),
                "out": normal(s.channels, s.width, scale=s.channels ** -0.5).to(dtype),
                # what the sequences leave for their next tokens
                "conv_state": torch.zeros(slots, s.taps - 1, s.channels, dtype=dtype, device=device),
                "scan_state": torch.zeros(slots, s.channels, s.states, device=device),
            })

    def _through(self, tokens, conv, scan):
        """Logits of the tokens; `conv` and `scan` run a layer's two operators."""
        s = self.sizes
        hidden = self.embedding[tokens]
        residual = torch.zeros_like(hidden)
        for layer in self.layers:
            # the residual stream grows by the layer before; its norm in 8 bits
            q, scales, residual = binding.lstm_residual_rms_norm(
                hidden, layer["norm"], 1e-5, residual=residual, residual_out=residual,
                quantize=True)
            xz = (q.to(self.dtype) @ layer["in"]) * scales.to(self.dtype)
            x = conv(layer, xz[:, :s.channels])
            small = x @ layer["x"]
            dt = small[:, :s.rank] @ layer["dt"]
            y = scan(layer, x, dt, small[:, s.rank:s.rank + s.states],
                     small[:, s.rank + s.states:], xz[:, s.channels:])
            hidden = y @ layer["out"]
        y, _, _ = binding.lstm_residual_rms_norm(hidden, self.final_norm, 1e-5, residual=residual)
        return y @ self.head

    def prompts(self, tokens, offsets, slots, resume=None):
        """Logits [tokens, vocab] of packed prompts; their states go to `slots`."""
        where = dict(offsets=offsets, slots=slots, resume=resume)
        return self._through(
            tokens,
            lambda l, x: binding.lstm_causal_conv(x, l["taps"], l["taps_bias"],
                                                  state=l["conv_state"], **where),
            lambda l, x, dt, b, c, z: binding.lstm_selective_scan(
                x, dt, l["a"], b, c, skip=l["skip"], z=z, dt_bias=l["dt_bias"],
                state=l["scan_state"], **where))

    def step(self, tokens, slots):
        """Logits [sequences, vocab] of the sequences' next tokens."""
        return self._through(
            tokens,
            lambda l, x: binding.lstm_causal_conv_step(x, l["taps"], l["taps_bias"],
                                                       l["conv_state"], slots=slots),
            lambda l, x, dt, b, c, z: binding.lstm_selective_scan_step(
                x, dt, l["a"], b, c, l["scan_state"], skip=l["skip"], z=z, dt_bias=l["dt_bias"],
                slots=slots))

    def generate(self, tokens, offsets, slots, steps: int, top: int = 5):
        """The likeliest next tokens of packed prompts (of one token at least),
        one at a time.  Returns
        (tokens, log probabilities, entropies, alternatives), [steps, sequences]
        each ([steps, sequences, top] the last)."""
        logits = self.prompts(tokens, offsets, slots)[offsets[1:].long() - 1]
        out = []
        for k in range(steps):
            _, entropy, top_logp, top_ids = binding.lstm_token_logprobs(logits, top=top)
            out.append((top_ids[:, 0], top_logp[:, 0], entropy, top_ids))
            if k + 1 < steps:
                logits = self.step(top_ids[:, 0], slots)
        return tuple(torch.stack(v) for v in zip(*out))


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    decoder = Decoder()
    lengths = [5, 130, 1, 42]
    offsets = torch.tensor([0, 5, 135, 136, 178], dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, 0, 7, 5], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    prompt = torch.randint(decoder.sizes.vocab, (sum(lengths),), generator=g, device="cuda")
    tokens, logp, entropy, _ = decoder.generate(prompt, offsets, slots, a.steps)
    for n, length in enumerate(lengths):
        print(f"prompt of {length}:", " ".join(f"{t}({p:.2f}, H {h:.2f})" for t, p, h in zip(
            tokens[:, n].tolist(), logp[:, n].tolist(), entropy[:, n].tolist())))


if __name__ == "__main__":
    main()
