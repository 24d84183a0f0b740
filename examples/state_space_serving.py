"""A small state space model served the way an engine serves it, on the library's layer
operators: prompts of mixed lengths in one packed call per layer, one prompt answered
several ways by forking its slots, decoding, and compaction when requests end.

The model is random: a few layers of projection, short convolution, selective scan
(one decay per channel and state element) and projection, with residuals. The run checks
itself: the scores that the packed, forked and compacted run gives the tokens are those of
every request run alone from its first token on, but for bf16 roundings.

    python examples/state_space_serving.py [--layers 4] [--dim 512] [--tokens 24]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_update_ssu_amd as ssu  # noqa: E402

DSTATE, WIDTH, VOCAB = 16, 4, 1000


class Layer:
    """x -> x + W_out scan(conv(W_in x)), with its slot caches."""

    def __init__(self, g, dim, slots, device):
        inner, rank = 2 * dim, max(8, dim // 16)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g) * cols ** -0.5).to(device, torch.bfloat16)

        self.inner, self.rank = inner, rank
        self.w_in, self.w_out = weight(2 * inner, dim), weight(dim, inner)
        self.w_x, self.w_dt = weight(rank + 2 * DSTATE, inner), weight(inner, rank)
        self.conv_w = (torch.rand(inner, WIDTH, generator=g) - 0.5).to(device, torch.bfloat16)
        self.conv_b = torch.zeros(inner, dtype=torch.bfloat16, device=device)
        self.A = -torch.arange(1, DSTATE + 1, dtype=torch.float32).repeat(inner, 1).to(device)
        self.D = torch.ones(inner, device=device)
        self.dt_bias = torch.log(torch.expm1(
            torch.exp(torch.rand(inner, generator=g) * 4.6 - 6.9))).to(device)
        self.conv_state = torch.zeros(slots, WIDTH - 1, inner, dtype=torch.bfloat16, device=device)
        self.state = torch.zeros(slots, inner, DSTATE, device=device)

    def __call__(self, x, slots, cu=None):
        xz = x @ self.w_in.t()
        u, z = xz[:, :self.inner], xz[:, self.inner:]
        if cu is None:
            u = ssu.causal_conv1d_update(self.conv_state, u, self.conv_w, bias=self.conv_b,
                                         state_batch_indices=slots)
        else:
            u = ssu.causal_conv1d_varlen(self.conv_state, u, self.conv_w, cu, bias=self.conv_b,
                                         state_batch_indices=slots)
        dbc = u @ self.w_x.t()
        dt = dbc[:, :self.rank] @ self.w_dt.t()
        B = dbc[:, self.rank:self.rank + DSTATE].unflatten(1, (1, DSTATE))
        C = dbc[:, self.rank + DSTATE:].unflatten(1, (1, DSTATE))
        common = dict(D=self.D, z=z, dt_bias=self.dt_bias, dt_softplus=True,
                      state_batch_indices=slots)
        if cu is None:
            y = ssu.selective_scan_update(self.state, u, dt, self.A, B, C, **common)
        else:
            y = ssu.selective_scan_varlen(self.state, u, dt, self.A, B, C, cu, **common)
        return x + y @ self.w_out.t()


class Model:
    def __init__(self, layers, dim, slots, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.embed = (torch.randn(VOCAB, dim, generator=g)).to(device, torch.bfloat16)
        self.layers = [Layer(g, dim, slots, device) for _ in range(layers)]
        self.caches = [c for layer in self.layers for c in (layer.conv_state, layer.state)]
        self.refcount = torch.zeros(slots, dtype=torch.int32, device=device)

    def __call__(self, tokens, slots, cu=None):
        """Next-token scores after each row."""
        x = self.embed[tokens]
        for layer in self.layers:
            x = layer(x, slots, cu)
        return (x @ self.embed.t()).float()


def serve(model, prompts, ways, tokens, choose):
    """Every prompt answered `ways` ways; after half of the tokens every second answer ends.
    choose(request, step, scores) picks a token; returns {request: tokens}."""
    device = model.refcount.device
    slots = ssu.cache_alloc(model.refcount, len(prompts))
    cu = torch.tensor([0] + [len(p) for p in prompts], device=device).cumsum(0).to(torch.int32)
    scores = model(torch.cat(prompts), slots, cu)[(cu[1:] - 1).long()]
    # The prompt's own slot serves its first answer, forks the others.
    requests = [(p, w) for w in range(ways) for p in range(len(prompts))]
    forks = ssu.cache_fork(model.caches, model.refcount, slots.repeat(ways - 1))
    slots, scores = torch.cat([slots, forks]), scores.repeat(ways, 1)
    answers = {r: [] for r in requests}
    for step in range(tokens):
        picked = [choose(r, step, s) for r, s in zip(requests, scores)]
        for r, t in zip(requests, picked):
            answers[r].append(t)
        if step == tokens // 2:
            stay = [i for i, r in enumerate(requests) if r[1] % 2 == 0]
            over = [i for i, r in enumerate(requests) if r[1] % 2 == 1]
            ssu.cache_free(model.refcount, slots[over])
            remap = ssu.cache_compact(model.caches, model.refcount)
            slots = remap[slots[stay].long()]
            requests, picked = [requests[i] for i in stay], [picked[i] for i in stay]
        scores = model(torch.tensor(picked, device=device), slots)
    ssu.cache_free(model.refcount, slots)
    return answers


def alone(model, prompt, answer):
    """The scores before each token of an answer, from one request's own run."""
    device = model.refcount.device
    slot = ssu.cache_alloc(model.refcount, 1)
    cu = torch.tensor([0, len(prompt)], dtype=torch.int32, device=device)
    scores = [model(prompt, slot, cu)[-1]]
    for t in answer[:-1]:
        scores.append(model(torch.tensor([t], device=device), slot)[0])
    ssu.cache_free(model.refcount, slot)
    return torch.stack(scores)


def main(layers=4, dim=512, tokens=24, lengths=(5, 130, 1, 64, 300), ways=4):
    model = Model(layers, dim, slots=len(lengths) * ways + 3)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(VOCAB, (n,), generator=g).cuda() for n in lengths]
    seen = {}

    def choose(request, step, scores):
        # The way-th best token, so that the answers differ.
        seen[request, step] = scores
        return int(scores.topk(request[1] + 1).indices[-1])

    answers = serve(model, prompts, ways, tokens, choose)
    worst = 0.0
    for (p, w), answer in answers.items():
        ref = alone(model, prompts[p], answer)
        got = torch.stack([seen[(p, w), i] for i in range(len(answer))])
        worst = max(worst, float((got - ref).abs().max() / ref.abs().max()))
    assert not bool((model.refcount != 0).any())
    print(f"{len(answers)} answers of up to {tokens} tokens to {len(prompts)} prompts; largest "
          f"difference of a score from a request run alone: {worst:.1e} of the largest score")
    return worst


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--dim", type=int, default=512)
    ap.add_argument("--tokens", type=int, default=24)
    a = ap.parse_args()
    sys.exit(0 if main(a.layers, a.dim, a.tokens) < 0.05 else 1)
