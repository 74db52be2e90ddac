"""Serving a layer of the gated delta rule: a prompt shared by many sequences,
its state kept in 8 bits, and generation with drafted tokens.

    python examples/delta_serving.py [--batch 8] [--prompt 700] [--new 48] [--draft 4]

A toy language model of one layer with random weights: token embeddings give
queries, keys, values, decays and strengths; the layer's output against the
embeddings gives the next token's logits.  The draft is the same model with a
cheaper readout.  What the library does:

  prompt      DeltaDevice       the chunked forward, up to the prompt's last state
  prefix      StateCache        that state put away once and read into every sequence
  drafted     DeltaStepDevice   outputs of the drafted tokens, states left alone
  verified    verify_draft      which of them the target keeps, and the token after
  advanced    DeltaStepDevice   the states moved on by the kept tokens only

and, for what was generated, the readout in 8 bits:

  scored      AddNormDevice     the outputs as int8 codes of their normed rows
              Linear8           against the embeddings in int8: the logits
              LogProbsDevice    the next tokens' log probabilities, entropies, alternatives
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mamba_selective_state_gb300 import runner  # noqa: E402


class Layer:
    """Random weights of the toy layer, and its maps from tokens to the delta
    rule's inputs and from its outputs to probabilities."""

    def __init__(self, vocab=512, width=256, nheads=8, headdim=64, dstate=64, ngroups=2, seed=0,
                 device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=gen, device=device) * s[0] ** -0.5  # noqa: E731
        self.H, self.P, self.N, self.G = nheads, headdim, dstate, ngroups
        self.embed = torch.randn(vocab, width, generator=gen, device=device)
        self.wq, self.wk = r(width, ngroups * dstate), r(width, ngroups * dstate)
        self.wv, self.wg, self.wb = r(width, nheads * headdim), r(width, nheads), r(width, nheads)
        self.wo = r(nheads * headdim, width)

    def inputs(self, tokens):
        """q, k, v, g, beta of tokens (b, L)."""
        b, L = tokens.shape
        x = self.embed[tokens.long()]
        f = torch.nn.functional
        unit = lambda w: f.normalize((x @ w).view(b, L, self.G, self.N), dim=-1).bfloat16()  # noqa: E731
        g = (-0.2 * f.softplus(x @ self.wg)).bfloat16()
        return (unit(self.wq), unit(self.wk), (x @ self.wv).view(b, L, self.H, self.P).bfloat16(), g,
                torch.sigmoid(x @ self.wb).bfloat16())

    def probs(self, y, temperature=1.0):
        """The next token's probabilities after outputs y (b, L, H, P)."""
        h = y.float().flatten(2) @ self.wo
        return torch.softmax(h @ self.embed.T / temperature, -1)


def generate(layer, prompt, batch, new, draft, seed=1):
    """Continue one prompt (L,) in `batch` sequences by at least `new` tokens
    each; returns the sequences' tokens (lists), the pool of states after all
    but each sequence's last token, and how many drafted tokens were kept."""
    dev = prompt.device
    gen = torch.Generator(device=dev).manual_seed(seed)
    # the prompt's state, but for its last token: that is the first one fed to the loop
    cache = runner.StateCache(1, layer.H, layer.P, layer.N, "int8", device=dev)
    if len(prompt) > 1:
        pre = runner.DeltaDevice(*layer.inputs(prompt[None, :-1]))
        pre.fwd()
        cache.store(pre.final)
    else:
        cache.store(torch.zeros(1, layer.H, layer.P, layer.N, device=dev))
    states = torch.empty(batch, layer.H, layer.P, layer.N, device=dev)
    cache.load(torch.zeros(batch, dtype=torch.int32, device=dev), states)  # one slot, many sequences
    pool = runner.DeltaStepDevice(states)
    last = prompt[-1].int().expand(batch).clone()
    out, kept = [[] for _ in range(batch)], 0
    while min(len(o) for o in out) < new:
        # the draft: token by token on a copy of the states, with a flatter readout
        scratch = runner.DeltaStepDevice(pool.states.clone())
        fed, q = [last], []
        for _ in range(draft):
            p = layer.probs(scratch.step(*layer.inputs(fed[-1][:, None])), temperature=1.3)[:, 0]
            q.append(p)
            race = torch.empty_like(p).exponential_(generator=gen)
            fed.append((p / race).argmax(-1).int())
        tokens = torch.stack(fed, 1)
        # the target over all of them at once; the states stay where they are
        ins = layer.inputs(tokens)
        p = layer.probs(pool.step(*ins, update=False))
        uniform = torch.rand(batch, draft, generator=gen, device=dev)
        noise = torch.empty(batch, p.shape[-1], device=dev).exponential_(generator=gen)
        chosen, n = runner.verify_draft(p, torch.stack(q, 1) if q else None, tokens[:, 1:].contiguous(),
                                        uniform, noise)
        # move on by the token that was fed and the drafted ones that were kept
        pool.step(*ins, lengths=n + 1, outputs=False)
        last = chosen.gather(1, n[:, None].long())[:, 0]
        for o, row, m in zip(out, chosen.tolist(), n.tolist()):
            o.extend(row[:m + 1])
            kept += m
    return out, pool.states, kept


def score(layer, tokens, top=3):
    """The log probability of each token of a sequence (L,) after those before it,
    with the entropies and the top alternatives (L - 1 rows): the model's readout
    with outputs and embeddings in 8 bits."""
    pre = runner.DeltaDevice(*layer.inputs(tokens[None, :-1]))
    pre.fwd()
    h = (pre.y[0].float().flatten(1) @ layer.wo).bfloat16()
    eps = 1e-5
    norm = runner.AddNormDevice(h, torch.ones(h.shape[1], device=h.device), eps=eps, form="int8")
    norm.fwd()
    # this readout takes its input as it is: the rows' sizes go back into their scales
    size = (h.float().square().mean(-1) + eps).sqrt()
    readout = runner.Linear8.from_weight(layer.embed, out_dtype=torch.float32)
    answer = runner.LogProbsDevice(readout(norm.codes, norm.scales * size), tokens[1:].clone(), ntop=top)
    answer.fwd()
    return answer


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=700)
    ap.add_argument("--new", type=int, default=48)
    ap.add_argument("--draft", type=int, default=4)
    a = ap.parse_args()
    layer = Layer()
    prompt = torch.randint(0, layer.embed.shape[0], (a.prompt,), device="cuda", dtype=torch.int32,
                           generator=torch.Generator(device="cuda").manual_seed(2))
    out, _, kept = generate(layer, prompt, a.batch, a.new, a.draft)
    total = sum(len(o) for o in out)
    print(f"{total} tokens in {a.batch} sequences, {kept} of them drafted and kept")
    for i, o in enumerate(out[:4]):
        got = score(layer, torch.cat((prompt, torch.tensor(o, device="cuda", dtype=torch.int32))))
        print(f"  sequence {i}: {o[:12]} ... mean log probability {got.logprobs[-len(o):].mean():.2f}, "
              f"entropy {got.entropy[-len(o):].mean():.2f}")


if __name__ == "__main__":
    main()
