"""A one-layer decoder trained and served with the library's operators.

Training: the embedding is a gather whose gradient is a fixed-order row
scatter-add, the attention scores get the learned relative position bias, and the
loss is taken from token log probabilities -- so two runs end in the same weights,
bit for bit.  Serving: each new token attends to a paged key-value cache with the
same bias table, and its log probability is reported with the alternatives; what
a sequence gets does not depend on the batch it is served in.

    python examples/reproducible_decoder.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from deterministic_floating_point_gb300 import _build, autograd, det  # noqa: E402

VOCAB, HEADS, DIM, BUCKETS, REACH = 1000, 4, 64, 32, 128
WIDTH = HEADS * DIM
PAGE = 16


def make_weights(seed: int) -> dict:
    g = torch.Generator().manual_seed(seed)

    def draw(*shape, scale):
        return (torch.randn(*shape, generator=g) * scale).cuda().requires_grad_(True)

    w = {name: draw(WIDTH, WIDTH, scale=WIDTH ** -0.5) for name in ("query", "key", "value", "mix")}
    w["embed"] = draw(VOCAB, WIDTH, scale=1.0)
    w["head"] = draw(WIDTH, VOCAB, scale=WIDTH ** -0.5)
    w["bias"] = draw(BUCKETS, HEADS, scale=0.1)
    return w


def make_batch(seed: int, batch: int, length: int) -> torch.Tensor:
    """Sequences that repeat a short random phrase: what comes next stands some tokens back."""
    g = torch.Generator().manual_seed(seed)
    phrase = torch.randint(0, VOCAB, (batch, 12), generator=g)
    return phrase.repeat(1, length // 12 + 1)[:, :length].to(torch.int32).cuda()


def forward(w: dict, tokens: torch.Tensor, bounds: torch.Tensor) -> torch.Tensor:
    """Logits [batch, length, VOCAB] of a batch of whole sequences."""
    batch, length = tokens.shape
    x = autograd.gather(w["embed"], tokens.reshape(-1)).view(batch, length, WIDTH)
    q, k, v = ((x @ w[n]).view(batch, length, HEADS, DIM).transpose(1, 2) for n in ("query", "key", "value"))
    scores = q @ k.transpose(2, 3) * DIM ** -0.5
    scores = scores + autograd.relative_bias(w["bias"], bounds, length, length, batch=batch)
    later = torch.ones(length, length, dtype=torch.bool, device="cuda").triu(1)
    mixed = torch.softmax(scores.masked_fill(later, float("-inf")), -1) @ v
    return (x + mixed.transpose(1, 2).reshape(batch, length, WIDTH) @ w["mix"]) @ w["head"]


def train(steps: int, seed: int = 0, batch: int = 8, length: int = 96):
    """(weights, losses) after plain gradient descent."""
    w, bounds = make_weights(seed), det.det_relative_bounds(BUCKETS, REACH)
    losses = []
    for step in range(steps):
        tokens = make_batch(1000 * seed + step % 4, batch, length)
        targets = torch.cat([tokens[:, 1:], tokens.new_full((batch, 1), -1)], 1).contiguous()   # -1: nothing to predict
        logprob, _ = autograd.token_logprobs(forward(w, tokens, bounds), targets)
        loss = -logprob.sum() / (targets >= 0).sum()
        grads = torch.autograd.grad(loss, list(w.values()))
        with torch.no_grad():
            for p, g in zip(w.values(), grads):
                p -= 0.5 * g
        losses.append(loss.item())
    return w, losses


class Server:
    """Sequences served a token at a time from a paged cache."""

    def __init__(self, w: dict, batch: int, most_tokens: int):
        self.w = {n: t.detach() for n, t in w.items()}
        self.bounds = det.det_relative_bounds(BUCKETS, REACH)
        pages = -(-most_tokens // PAGE)
        self.k = torch.empty(batch * pages, PAGE, HEADS, DIM, dtype=torch.bfloat16, device="cuda")
        self.v = torch.empty_like(self.k)
        # the pages of a sequence lie anywhere in the pool
        self.table = torch.randperm(batch * pages, generator=torch.Generator().manual_seed(3)).to(torch.int32).view(
            batch, pages).cuda()
        self.lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def step(self, tokens: torch.Tensor, top_k: int = 5):
        """Take one token of each sequence; (logits, alternatives, attention) for the next."""
        w, at = self.w, self.lengths.long()
        x = det.det_gather_rows(w["embed"], tokens)
        q, k, v = ((x @ w[n]).view(-1, HEADS, DIM).bfloat16() for n in ("query", "key", "value"))
        page = self.table.gather(1, (at // PAGE)[:, None])[:, 0].long()
        self.k[page, at % PAGE], self.v[page, at % PAGE] = k, v
        self.lengths += 1
        mixed = det.det_paged_attention(q, self.k, self.v, self.table, self.lengths, bias_table=w["bias"],
                                        bias_bounds=self.bounds)
        logits = (x + mixed.out.float().reshape(-1, WIDTH) @ w["mix"]) @ w["head"]
        return logits, det.det_token_logprobs(logits, top_k=top_k), (q, mixed)


def main(steps: int = 60) -> dict:
    first, losses = train(steps)
    second, _ = train(steps)
    same_weights = all(torch.equal(first[n], second[n]) for n in first)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {steps} steps; two runs end in the same bits: {same_weights}")

    batch, length = 3, 60
    tokens = make_batch(99, batch, length)
    server = Server(first, batch, length)
    served = []
    same_alone = True
    for t in range(length):
        logits, alternatives, (q, mixed) = server.step(tokens[:, t].contiguous())
        if t + 1 < length:
            served.append(det.det_token_logprobs(logits, tokens[:, t + 1].contiguous()).logprob)
        if t % 13 == 0:
            for b in range(batch):
                alone = det.det_paged_attention(q[b:b + 1], server.k, server.v, server.table[b:b + 1],
                                                server.lengths[b:b + 1], bias_table=server.w["bias"],
                                                bias_bounds=server.bounds)
                one = det.det_token_logprobs(logits[b:b + 1], top_k=5)
                same_alone &= torch.equal(alone.out[0], mixed.out[b]) and torch.equal(one.top_logprob[0],
                                                                                    alternatives.top_logprob[b])
    served = torch.stack(served, 1)
    targets = torch.cat([tokens[:, 1:], tokens.new_full((batch, 1), -1)], 1).contiguous()
    with torch.no_grad():
        whole = det.det_token_logprobs(forward(first, tokens, server.bounds), targets).logprob[:, :-1]
    apart = float((served - whole).abs().max())
    print(f"served log probabilities against the training pass: at most {apart:.3f} apart (16-bit cache)")
    print(f"a sequence alone and in the batch: same bits {same_alone}")
    print("alternatives for the first sequence's next token:",
          [(int(i), round(float(p), 2)) for i, p in zip(alternatives.top_index[0], alternatives.top_logprob[0])])
    return {"losses": losses, "same_weights": same_weights, "same_alone": bool(same_alone), "apart": apart}


if __name__ == "__main__":
    _build.build()
    main()
