"""A small recurrent language model on the library: embedding, one LSTM layer,
linear attention with a decay for each head, logits, token log probabilities.

    python examples/recurrent_lm.py [--steps 60]

Trains by plain gradient descent on a synthetic text and then continues a
prompt token by token.  Every step of the model runs in the library's kernels
(embed_fwd, lstm_fwd, input_proj, linattn_fwd / linattn_step, token_logprobs)
and so do their gradients; the gradients of the two projections' weights are
plain matrix products.  float32 throughout.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gru_recurrence_amd as g  # noqa: E402


class RecurrentLM:
    """x = E[ids]; h = LSTM(x); y = h + linear_attention(h Wqkv); logits = y Wout."""

    def __init__(self, vocab=64, heads=4, head_dim=32, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        H = heads * head_dim
        self.V, self.NH, self.Dh, self.H, self.dev = vocab, heads, head_dim, H, device

        def randn(*shape, std):
            return torch.randn(shape, generator=gen, device=device) * std
        self.p = {"E": randn(vocab, H, std=1.0), "W": randn(H, 4 * H, std=H ** -0.5),
                  "R": randn(heads, head_dim, 4 * head_dim, std=head_dim ** -0.5),
                  "b": torch.zeros(4 * H, device=device),
                  "Wqkv": randn(H, 3 * H, std=H ** -0.5), "Wout": randn(H, vocab, std=H ** -0.5)}
        # log decays: half-lives from 2 to 64 tokens over the heads
        half = torch.exp2(torch.linspace(1.0, 6.0, heads, device=device))
        self.decay = -torch.log(torch.tensor(2.0, device=device)) / half

    def _qkv(self, h):
        qkv = g.input_proj(h, self.p["Wqkv"])
        return [t.unflatten(-1, (self.NH, self.Dh)) for t in qkv.split(self.H, -1)]

    def forward(self, ids, state=None):
        """ids [T,B] -> logits [T,B,V], what the backward needs, the new state."""
        p = self.p
        h0, c0, S0 = state if state is not None else (None, None, None)
        x = g.embed_fwd(ids, p["E"])
        h, c, hT, cT = g.lstm_fwd(x, p["W"], p["R"], p["b"], h0, c0)
        q, k, v = self._qkv(h)
        if ids.shape[0] == 1 and S0 is not None:
            o, ST = g.linattn_step(q, k, v, self.decay, S0)
        else:
            o, ST = g.linattn_fwd(q, k, v, self.decay, S0)
        y = h + o.flatten(2)
        return g.input_proj(y, p["Wout"]), (x, h, c, q, k, v, y), (hT, cT, ST)

    def gradients(self, ids, targets):
        """Mean negative log probability of the targets and its gradients."""
        p = self.p
        logits, (x, h, c, q, k, v, y), _ = self.forward(ids)
        r = g.token_logprobs(logits, targets)
        n = (targets >= 0).sum()
        dlogp = (-1.0 / n).expand(targets.shape).contiguous()
        dl = g.token_logprobs_bwd(logits, targets, r["lse"], dlogp=dlogp, out=logits)
        rows = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        d = {"Wout": rows(y).t() @ rows(dl)}
        dy = dl @ p["Wout"].t()
        a = g.linattn_bwd(q, k, v, self.decay, dy.unflatten(-1, (self.NH, self.Dh)))
        dqkv = torch.cat([a[n_].flatten(2) for n_ in ("dq", "dk", "dv")], -1)
        d["Wqkv"] = rows(h).t() @ rows(dqkv)
        dh = dy + dqkv @ p["Wqkv"].t()
        b = g.lstm_bwd(x, p["W"], p["R"], p["b"], None, None, h, c, dh)
        d.update(W=b["dW"], R=b["dR"], b=b["db"], E=g.embed_bwd(ids, b["dx"], self.V))
        return -(r["logp"].sum() / n), d

    def train(self, ids, targets, steps, lr=0.5, clip=1.0):
        losses = []
        for _ in range(steps):
            loss, d = self.gradients(ids, targets)
            norm = torch.stack([t.norm() for t in d.values()]).norm()
            scale = lr * torch.clamp(clip / norm, max=1.0)
            for n, t in d.items():
                self.p[n] -= scale * t
            losses.append(loss)
        return [float(x) for x in losses]

    def generate(self, prompt, n, top=3):
        """Continue prompt [T,B] greedily: ids [n,B], their log probabilities."""
        logits, _, state = self.forward(prompt)
        ids, lps = [], []
        for _ in range(n):
            last = logits[-1:]
            r = g.token_logprobs(last, torch.full(last.shape[:2], -1, device=self.dev), top=top)
            nxt = r["top_id"][..., 0].contiguous()
            ids.append(nxt)
            lps.append(r["top_logp"][..., 0])
            logits, _, state = self.forward(nxt, state)
        return torch.cat(ids), torch.cat(lps)


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
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    m = RecurrentLM()
    ids, targets = text(96, 8, m.V)
    losses = m.train(ids, targets, a.steps)
    for i in range(0, len(losses), max(1, len(losses) // 6)):
        print("step %3d  loss %.4f" % (i, losses[i]))
    print("step %3d  loss %.4f" % (len(losses) - 1, losses[-1]))
    out, lp = m.generate(ids[:40], 20)
    print("continued right: %.0f%%, mean log probability %.3f"
          % (100 * (out == targets[39:59]).float().mean().item(), lp.mean().item()))


if __name__ == "__main__":
    main()
