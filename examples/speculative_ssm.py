"""Speculative decoding on one state space layer: packed prompts, drafted runs, verification, commit.

A toy language model with random weights - embedding, projection, short convolution, selective
scan, head - whose drafts come from a table of next-token probabilities.  The prompts go through
``conv_fwd`` and ``ssm_fwd``, which leave each sequence's convolution inputs and state in the pools.
Every step then runs the last token and its drafts without commit, lets ``verify_draft`` decide,
and commits as many tokens of each run as were emitted (``used=n_out``): nothing of a step waits
for the host until its tokens are printed.

    python examples/speculative_ssm.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_serving_chunk_gb300 as kda  # noqa: E402


class Layer:
    """Weights of the toy model, and its two forms."""

    def __init__(self, vocab=512, width=128, H=4, P=64, G=1, N=64, W=4, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.H, self.P, self.G, self.N, self.W, self.vocab = H, P, G, N, W, vocab
        self.conv_dim = H * P + 2 * G * N
        self.embed = rnd(vocab, width).bfloat16()
        # z | x B C | dt, as one projection
        self.proj = (rnd(width, H * P + self.conv_dim + 8) / width ** 0.5).bfloat16()
        self.conv_w = (rnd(self.conv_dim, W) / W ** 0.5).bfloat16()
        self.conv_b = (0.1 * rnd(self.conv_dim)).bfloat16()
        self.A, self.D = -torch.arange(1, H + 1, device="cuda").float(), torch.ones(H, device="cuda")
        self.dt_bias = torch.full((H,), -3.0, device="cuda")
        self.head = (4 * rnd(H * P, vocab) / (H * P) ** 0.5).bfloat16()

    def _split(self, tokens):
        h = self.embed[tokens.long()] @ self.proj
        hp = self.H * self.P
        return h[:, :hp].unflatten(1, (self.H, self.P)), h[:, hp:hp + self.conv_dim], \
            h[:, hp + self.conv_dim:hp + self.conv_dim + self.H]

    def _scan_args(self, c, dt, z):
        hp, gn = self.H * self.P, self.G * self.N
        return dict(x=c[:, :hp].unflatten(1, (self.H, self.P)), dt=dt, A=self.A,
                    B=c[:, hp:hp + gn].unflatten(1, (self.G, self.N)),
                    C=c[:, hp + gn:].unflatten(1, (self.G, self.N)), D=self.D, z=z, dt_bias=self.dt_bias)

    def probs(self, o):
        return torch.softmax((o.flatten(1) @ self.head).float(), 1)

    def prompts(self, tokens, cu):
        """Outputs of packed prompts, and what each leaves behind: (o, conv inputs, states)."""
        n = cu.numel() - 1
        z, xbc, dt = self._split(tokens)
        conv = torch.empty(n, self.W - 1, self.conv_dim, dtype=torch.bfloat16, device="cuda")
        state = torch.empty(n, self.H, self.N, self.P, device="cuda")
        c = kda.conv_fwd(xbc, self.conv_w, self.conv_b, cu_seqlens=cu, conv_final=conv)
        o = kda.ssm_fwd(cu_seqlens=cu, S_final=state, **self._scan_args(c, dt, z))
        return o, conv, state

    def verify_and_commit(self, tokens, cu, draft_probs, u, conv_pool, state_pool):
        """One speculative step of all runs: (emitted tokens, how many of each run)."""
        z, xbc, dt = self._split(tokens)
        c = kda.conv_tokens(xbc, self.conv_w, self.conv_b, conv_pool, cu_seqlens=cu, commit=False)
        scan = self._scan_args(c, dt, z)
        o = kda.ssm_tokens(state_pool=state_pool, cu_seqlens=cu, commit=False, **scan)
        out, n_out = kda.verify_draft(self.probs(o), tokens, u, cu, draft=draft_probs)
        kda.conv_tokens(xbc, self.conv_w, self.conv_b, conv_pool, cu_seqlens=cu, used=n_out, o=False)
        kda.ssm_tokens(state_pool=state_pool, cu_seqlens=cu, used=n_out, o=False, **scan)
        return out, n_out


def run(n=4, drafts=3, steps=12, seed=0):
    """Generates from n prompts.  Returns (tokens of each sequence, accepted share of the drafts,
    largest difference between the pools and the states of the same tokens as one prompt)."""
    torch.manual_seed(seed)
    m = Layer()
    lens = [5 + 37 * b for b in range(n)]
    texts = [torch.randint(0, m.vocab, (L,)).tolist() for L in lens]
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    tokens = torch.tensor(sum(texts, []), dtype=torch.int32, device="cuda")
    # the last token of a prompt is the first of its first run: it is not in the states yet
    keep = torch.ones(len(tokens), dtype=torch.bool, device="cuda")
    keep[cu[1:].long() - 1] = False
    cu0 = cu - torch.arange(n + 1, device="cuda", dtype=torch.int32)
    _, conv_pool, state_pool = m.prompts(tokens[keep], cu0)
    # the draft model: the target's first-token distribution, smoothed
    first, _, _ = m.prompts(torch.arange(m.vocab, device="cuda", dtype=torch.int32),
                            torch.arange(m.vocab + 1, device="cuda", dtype=torch.int32))
    table = 0.8 * m.probs(first) + 0.2 / m.vocab
    run_cu = torch.arange(0, n * (drafts + 1) + 1, drafts + 1, device="cuda", dtype=torch.int32)
    last = tokens[cu[1:].long() - 1]
    accepted = 0
    for _ in range(steps):
        rows, q = [last], []
        for _ in range(drafts):
            q.append(table[rows[-1].long()])
            rows.append(torch.multinomial(q[-1], 1)[:, 0].int())
        batch = torch.stack(rows, 1).reshape(-1)
        out, n_out = m.verify_and_commit(batch, run_cu, torch.stack(q, 1).flatten(0, 1),
                                         torch.rand(len(batch), device="cuda"), conv_pool, state_pool)
        new, count = out.view(n, -1).tolist(), n_out.tolist()
        for b in range(n):
            texts[b] += new[b][:count[b]]
        accepted += sum(count) - n
        last = torch.tensor([t[-1] for t in texts], dtype=torch.int32, device="cuda")
    # the same tokens as prompts end in the same states (the last token of each is still to come)
    packed = torch.tensor(sum((t[:-1] for t in texts), []), dtype=torch.int32, device="cuda")
    ends = torch.tensor([0] + [len(t) - 1 for t in texts], device="cuda").cumsum(0).int()
    _, conv, state = m.prompts(packed, ends)
    apart = max(float((conv.float() - conv_pool.float()).abs().max()),
                float((state - state_pool).abs().max() / state.abs().max()))
    if kda.device_status() != 0:
        raise RuntimeError("device status word set")
    return texts, accepted / (steps * n * drafts), apart


if __name__ == "__main__":
    texts, share, apart = run()
    for t in texts:
        print(len(t), "tokens, the last:", t[-8:])
    print(f"drafts accepted: {share:.2f}; pools against one prompt of the same tokens: {apart:.1e}")
