"""A small language model's head, trained and then used: the norm before the head, the fused loss
with clipped gradients and an orthogonalised update, the norm's output and the head's weight in
8-bit integers, and a beam search over its logits.

    python examples/train_and_decode.py

The model is one recurrent cell over token embeddings with a head over the vocabulary. It learns
sequences that count up by a step given at their start, and then continues such sequences with
four beams; the training's loss falls and most continuations are right (all 64, where it was
tried). Takes seconds on one GPU.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from linear_cross_entropy_vocab_gb300 import (  # noqa: E402
    beam_reorder_, beam_select, clip_grad_norm_, fused_linear_cross_entropy, int8_linear,
    orthogonalize, quantize_rows, rms_norm, rms_norm_quantize)

VOCAB, HIDDEN, STEPS, LENGTH = 1000, 256, 300, 24
BEAMS, PROMPT, END = 4, 4, 0  # token 0 ends a sequence


def sequences(n, generator):
    """start, start + step, ... with a step of 1 to 9; the last token is END."""
    start = torch.randint(1, 500, (n, 1), generator=generator, device="cuda")
    step = torch.randint(1, 10, (n, 1), generator=generator, device="cuda")
    tokens = start + step * torch.arange(LENGTH, device="cuda")
    tokens[:, -1] = END
    return tokens


class Model(torch.nn.Module):
    """A token's embedding and that of its difference to the one before, and a hidden layer."""

    def __init__(self):
        super().__init__()
        self.token = torch.nn.Embedding(VOCAB, HIDDEN)
        self.change = torch.nn.Embedding(2 * VOCAB, HIDDEN)
        self.place = torch.nn.Embedding(LENGTH, HIDDEN)
        self.mix = torch.nn.Linear(HIDDEN, HIDDEN)
        self.norm = torch.nn.Parameter(torch.ones(HIDDEN))
        self.head = torch.nn.Parameter(torch.randn(VOCAB, HIDDEN) * HIDDEN ** -0.5)

    def hidden(self, token, before, place):
        """What the layer adds, in 16 bits, and the stream it is added to, in 32."""
        x = self.token(token) + self.change(token - before + VOCAB) + self.place(place)
        return torch.nn.functional.gelu(self.mix(x)).bfloat16(), x


def train(model, generator):
    # the layer's matrix is updated by its orthogonalised momentum, everything else by AdamW
    mix = model.mix.weight
    optimizer = torch.optim.AdamW([p for p in model.parameters() if p is not mix], lr=1e-2,
                                  weight_decay=0.0)
    momentum = torch.zeros_like(mix)
    losses = []
    for _ in range(STEPS):
        tokens = sequences(256, generator)
        before = torch.cat([tokens[:, :1], tokens[:, :-1]], 1)
        place = torch.arange(LENGTH, device="cuda").expand_as(tokens)
        added, stream = model.hidden(tokens, before, place)
        hidden, _ = rms_norm(added, model.norm, residual=stream)
        loss = fused_linear_cross_entropy(hidden[:, 1:-1], model.head.bfloat16(),
                                          tokens[:, 2:], reduction="mean")
        model.zero_grad()
        loss.backward()
        clip_grad_norm_(model.parameters(), 1.0)
        optimizer.step()
        with torch.no_grad():
            momentum.mul_(0.95).add_(mix.grad)
            mix.add_(orthogonalize(momentum), alpha=-0.02)
        losses.append(loss.detach())
    return float(losses[0]), float(losses[-1])


@torch.no_grad()
def decode(model, prompts):
    """[B, LENGTH] continuations of prompts [B, PROMPT], the best of BEAMS beams each."""
    batch = prompts.shape[0]
    weight, weight_scale = quantize_rows(model.head.bfloat16())
    # what is kept for each beam: its tokens, and here no cache
    history = torch.zeros(batch * BEAMS, LENGTH, dtype=torch.int64, device="cuda")
    history[:, :PROMPT] = prompts.repeat_interleave(BEAMS, 0)
    # one beam to start with: the others are copies of it
    scores = torch.full((batch, BEAMS), -torch.inf, device="cuda")
    scores[:, 0] = 0.0
    finished = torch.zeros(batch, BEAMS, dtype=torch.bool, device="cuda")
    for at in range(PROMPT, LENGTH):
        added, stream = model.hidden(history[:, at - 1], history[:, at - 2],
                                     torch.full((batch * BEAMS,), at - 1, device="cuda"))
        hidden, scale, _ = rms_norm_quantize(added, model.norm, residual=stream)
        logits = int8_linear(hidden, weight, weight_scale, x_scale=scale)
        chosen = beam_select(logits.view(batch, BEAMS, VOCAB), scores, finished=finished,
                             pad_token=END)
        flags = finished.view(-1, 1)
        beam_reorder_([history, flags], chosen.parents)
        history[:, at] = chosen.tokens.view(-1)
        scores = chosen.scores
        finished = flags.view(batch, BEAMS) | (chosen.tokens == END)
    return history.view(batch, BEAMS, LENGTH)[:, 0]


def main():
    torch.manual_seed(0)
    generator = torch.Generator("cuda").manual_seed(0)
    model = Model().cuda()
    first, last = train(model, generator)
    wanted = sequences(64, generator)
    got = decode(model, wanted[:, :PROMPT])
    right = float((got == wanted).all(1).float().mean())
    print(f"loss {first:.3f} -> {last:.3f}; {100 * right:.0f} % of the continuations are right")
    return first, last, right


if __name__ == "__main__":
    main()
