"""A small decoder of linear-attention layers run end to end on the library's operators.

Packed prompts of unequal lengths go through a stack of layers (residual norm, one dense
product to queries, keys, values and a gate, linear attention with a decay for each head,
a dense product back, and a two-product block with an activation); the log probabilities
read off the last logits choose the next token, and further tokens are decoded one at a
time from the layers' states.

    python examples/linear_attention_decoder.py [--steps 8]
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
    heads: int = 4
    shared: int = 2       # heads of keys and values
    keys: int = 32
    values: int = 64
    inner: int = 512      # of the block behind a layer
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

        def weight(out, n_in):
            return normal(out, n_in, scale=n_in ** -0.5).to(dtype)

        self.sizes, self.dtype = sizes, dtype
        self.widths = [s.heads * s.keys, s.shared * s.keys, s.shared * s.values]
        self.embedding = normal(s.vocab, s.width).to(dtype)
        self.head = normal(s.vocab, s.width, scale=2.0 * s.width ** -0.5).to(dtype)
        self.final_norm = 0.5 + torch.rand(s.width, generator=g, device=device)
        # memories of 8 to 256 tokens
        self.log_decay = torch.log1p(-torch.exp2(-torch.linspace(3.0, 8.0, s.heads, device=device)))
        self.layers = [{
            "norm": torch.ones(s.width, device=device),
            "in": weight(sum(self.widths), s.width),
            "out": weight(s.width, s.heads * s.values),
            "norm2": torch.ones(s.width, device=device),
            "up": weight(s.inner, s.width),
            "up_bias": normal(s.inner, scale=0.1),
            "down": weight(s.width, s.inner),
            # what the sequences leave for their next tokens
            "state": torch.zeros(slots, s.heads, s.keys, s.values, device=device),
        } for _ in range(s.layers)]

    def _through(self, tokens, attention):
        """Logits of the tokens; `attention` runs a layer's."""
        s = self.sizes
        hidden = self.embedding[tokens]
        for layer in self.layers:
            x, _, _ = binding.lstm_residual_rms_norm(hidden, layer["norm"], 1e-5)
            q, k, v = binding.lstm_dense(x, layer["in"]).split(self.widths, 1)
            y = attention(layer, q.unflatten(1, (s.heads, s.keys)), k.unflatten(1, (s.shared, s.keys)),
                          v.unflatten(1, (s.shared, s.values)))
            hidden = binding.lstm_dense(y.flatten(1), layer["out"], residual=hidden)
            x, _, _ = binding.lstm_residual_rms_norm(hidden, layer["norm2"], 1e-5)
            x = binding.lstm_dense(x, layer["up"], layer["up_bias"], activation="silu")
            hidden = binding.lstm_dense(x, layer["down"], residual=hidden)
        x, _, _ = binding.lstm_residual_rms_norm(hidden, self.final_norm, 1e-5)
        return binding.lstm_dense(x, self.head)

    def prompts(self, tokens, offsets, slots, resume=None):
        """Logits [tokens, vocab] of packed prompts; their states go to `slots`."""
        return self._through(tokens, lambda l, q, k, v: binding.lstm_linear_attention(
            q, k, v, self.log_decay, scale=self.sizes.keys ** -0.5, sequences=slots.numel(),
            offsets=offsets, state=l["state"], slots=slots, resume=resume))

    def step(self, tokens, slots):
        """Logits [sequences, vocab] of the sequences' next tokens."""
        return self._through(tokens, lambda l, q, k, v: binding.lstm_linear_attention_step(
            q, k, v, self.log_decay, l["state"], scale=self.sizes.keys ** -0.5, slots=slots))

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
