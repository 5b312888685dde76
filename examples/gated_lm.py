"""A small language model of gated linear recurrences on the library: embedding,
layers y + gated(y W), logits, token log probabilities.

    python examples/gated_lm.py [--steps 150]

Trains on a synthetic text by gradient descent with the global norm clipped and
then continues prompts with drafted tokens: drafts are looked up in the text so
far, one pass over them gives the model's logits at every position, they are
verified with given random numbers, and each layer's state is taken back to the
last token that stands.  Every step of the model runs in the library's kernels
(embed_fwd, input_proj, gated_fwd / gated_step, token_logprobs, verify_drafts,
clip_grads) and so do their gradients; those of the projections' weights are
plain matrix products.  float32 throughout.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gru_recurrence_amd as g  # noqa: E402


class GatedLM:
    """y = E[ids]; y += gated(y W_l) for each layer; logits = y Wout."""

    def __init__(self, vocab=64, width=128, layers=2, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.V, self.H, self.L, self.dev = vocab, width, layers, device

        def randn(*shape, std):
            return torch.randn(shape, generator=gen, device=device) * std
        self.p = {"E": randn(vocab, width, std=1.0), "Wout": randn(width, vocab, std=width ** -0.5)}
        # gates that start with memories from 1 to 64 tokens over the channels
        span = torch.linspace(0.0, 4.2, width, device=device)
        for i in range(layers):
            self.p["W%d" % i] = randn(width, 2 * width, std=width ** -0.5)
            self.p["b%d" % i] = torch.cat([span, torch.zeros_like(span)])

    def _layers(self, y, states=None):
        """Runs the layers: the last y, each layer's (input, f, x, h), new states."""
        kept, new = [], []
        for i in range(self.L):
            f, x = g.input_proj(y, self.p["W%d" % i], self.p["b%d" % i]).split(self.H, -1)
            h0 = None if states is None else states[i]
            if y.shape[0] == 1 and h0 is not None:
                h, hT = g.gated_step(f, x, h0, h_out=torch.empty_like(h0))
            else:
                h, hT = g.gated_fwd(f, x, h0)
            kept.append((y, f, x, h))
            new.append(hT)
            y = y + h
        return y, kept, new

    def forward(self, ids, states=None):
        """ids [T,B] -> logits [T,B,V], what the backward needs, the new states."""
        y, kept, new = self._layers(g.embed_fwd(ids, self.p["E"]), states)
        return g.input_proj(y, self.p["Wout"]), (y, kept), new

    def gradients(self, ids, targets):
        """Mean negative log probability of the targets and its gradients."""
        logits, (y, kept), _ = self.forward(ids)
        r = g.token_logprobs(logits, targets)
        n = (targets >= 0).sum()
        dlogp = (-1.0 / n).expand(targets.shape).contiguous()
        dl = g.token_logprobs_bwd(logits, targets, r["lse"], dlogp=dlogp, out=logits)
        rows = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        d = {"Wout": rows(y).t() @ rows(dl)}
        dy = dl @ self.p["Wout"].t()
        for i in reversed(range(self.L)):
            y, f, x, h = kept[i]
            dfx = torch.empty((*f.shape[:2], 2 * self.H), device=self.dev)
            df, dx = dfx.split(self.H, -1)
            g.gated_bwd(f, x, h, dy, out={"df": df, "dx": dx})
            d["W%d" % i], d["b%d" % i] = rows(y).t() @ rows(dfx), rows(dfx).sum(0)
            dy = dy + dfx @ self.p["W%d" % i].t()
        d["E"] = g.embed_bwd(ids, dy, self.V)
        return -(r["logp"].sum() / n), d

    def train(self, ids, targets, steps, lr=0.5, clip=1.0):
        losses = []
        for _ in range(steps):
            loss, d = self.gradients(ids, targets)
            g.clip_grads(list(d.values()), clip)
            for n, t in d.items():
                self.p[n] -= lr * t
            losses.append(loss)
        return [float(x) for x in losses]

    def generate(self, prompt, n):
        """Continue prompt [T,B] greedily, a token at a time: ids [n,B]."""
        logits, _, states = self.forward(prompt)
        ids = []
        for _ in range(n):
            ids.append(logits[-1:].argmax(-1))
            logits, _, states = self.forward(ids[-1], states)
        return torch.cat(ids)

    def continue_drafted(self, prompt, n, drafts=4, temperature=0.0, seed=0):
        """The same with drafted tokens: a list of at least n ids for each
        sequence, and the passes it took.  temperature 0 is greedy."""
        gen = torch.Generator(device=self.dev).manual_seed(seed)
        B, K = prompt.shape[1], drafts
        texts = prompt.t().tolist()
        start = [len(t) for t in texts]
        temp = torch.full((B,), float(temperature), device=self.dev)
        _, _, states = self.forward(prompt[:-1])
        passes = 0
        while min(len(t) - s for t, s in zip(texts, start)) < n:
            found = [_lookup(t, K) for t in texts]
            num = torch.tensor([len(x) for x in found], dtype=torch.int32, device=self.dev)
            rows = [[t[-1]] + x + [0] * (K - len(x)) for t, x in zip(texts, found)]
            ids = torch.tensor(rows, device=self.dev).t()  # [K+1, B]: the last token, the drafts
            logits, (_, kept), _ = self.forward(ids, states)
            u = torch.rand((K + 1, B), generator=gen, device=self.dev)
            tokens, accepted = g.verify_drafts(logits, ids[1:], u, temperature=temp, n_drafts=num)
            # the states behind the last token that stands
            states = [g.gated_fwd(f, x, s, lens=accepted + 1)[1]
                      for (_, f, x, _), s in zip(kept, states)]
            for t, new, k in zip(texts, tokens.t().tolist(), accepted.tolist()):
                t += new[:k + 1]
            passes += 1
        return [t[s:] for t, s in zip(texts, start)], passes


def _lookup(text, most):
    """What followed the last two tokens when they last stood in the text."""
    for i in range(len(text) - 3, -1, -1):
        if text[i:i + 2] == text[-2:]:
            return text[i + 2:i + 2 + most]
    return []


def text(T, B, vocab, device="cuda", seed=1):
    """Sequences that repeat a random phrase of 5 to 8 tokens of their own."""
    gen = torch.Generator().manual_seed(seed)
    cols = []
    for i in range(B):
        phrase = torch.randint(0, vocab, (5 + i % 4,), generator=gen)
        cols.append(phrase.repeat(T // len(phrase) + 2)[:T + 1])
    t = torch.stack(cols, 1).to(device)
    return t[:-1].contiguous(), t[1:].contiguous()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=150)
    a = ap.parse_args()
    m = GatedLM()
    ids, targets = text(96, 8, m.V)
    losses = m.train(ids, targets, a.steps)
    for i in range(0, len(losses), max(1, len(losses) // 6)):
        print("step %3d  loss %.4f" % (i, losses[i]))
    print("step %3d  loss %.4f" % (len(losses) - 1, losses[-1]))
    out, passes = m.continue_drafted(ids[:40], 32)
    want = targets[39:71].t().tolist()
    right = sum(a == b for t, w in zip(out, want) for a, b in zip(t, w)) / (32 * len(out))
    print("continued right: %.0f%%, %d tokens a sequence in %d passes"
          % (100 * right, min(len(t) for t in out), passes))


if __name__ == "__main__":
    main()
