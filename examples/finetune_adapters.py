"""Fine-tune and serve low-rank adapters over frozen 2:4 layers, end to end.

A small residual language model: an embedding, `LAYERS` blocks of

    x + W_nm norm(x) + (the request's adapter of norm(x)),

a final norm and a dense head.  The 2:4 weights are packed once and stay
frozen; the adapters, the norms and the head learn, two tasks in one batch, each
with its own adapter.  Every step runs

    nm_layernorm -> nm_adapter_spmm -> ... -> nm_xent
    nm_xent_bwd -> nm_layernorm_bwd -> nm_adapter_spmm_bwd -> ...

and then both tasks are served together, a token at a time, each request naming
its adapter.

    python examples/finetune_adapters.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import structured_sparse_gemm_nm_amd as nm

WIDTH, VOCAB, LAYERS, RANK = 512, 1000, 2, 16
REQUESTS, LENGTH = 8, 48          # a batch: requests of so many tokens
BF16 = torch.bfloat16


class Model:
    def __init__(self, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *shape, s: torch.randn(*shape, generator=g, device=device) * s
        self.embedding = normal(VOCAB, WIDTH, s=1.0).to(BF16)
        self.packed = [nm.nm_compress(normal(WIDTH, WIDTH, s=WIDTH ** -0.5).to(BF16)) for _ in range(LAYERS)]
        self.scale = torch.full((2,), 2.0, device=device)         # of the two adapters
        # what learns, in fp32; the operators take bf16 copies
        self.params = {"head": normal(VOCAB, WIDTH, s=WIDTH ** -0.5), "norm": torch.ones(WIDTH, device=device),
                       "norm_bias": torch.zeros(WIDTH, device=device)}
        for i in range(LAYERS):
            self.params[f"A{i}"] = normal(2, RANK, WIDTH, s=WIDTH ** -0.5)
            self.params[f"B{i}"] = torch.zeros(2, WIDTH, RANK, device=device)   # the adapters start out silent
            self.params[f"norm{i}"] = torch.ones(WIDTH, device=device)
            self.params[f"norm{i}_bias"] = torch.zeros(WIDTH, device=device)

    def rounded(self):
        return {k: v.to(BF16) for k, v in self.params.items()}

    def hidden(self, p, tokens, adapter):
        """The final norm's output and what the backward pass needs of each layer."""
        x = self.embedding[tokens]
        saved = []
        for i, (values, idx) in enumerate(self.packed):
            h, mean, rstd = nm.nm_layernorm(x, p[f"norm{i}"], p[f"norm{i}_bias"], stats=True)
            y, xa = nm.nm_adapter_spmm(values, idx, h, adapter, p[f"A{i}"], p[f"B{i}"], self.scale, WIDTH,
                                       out_dtype=BF16)
            saved.append((x, mean, rstd, h, xa))
            x = x + y
        out, mean, rstd = nm.nm_layernorm(x, p["norm"], p["norm_bias"], stats=True)
        return out, (x, mean, rstd), saved

    def step(self, tokens, adapter, labels, rate):
        """One step of gradient descent; returns the mean loss before it (a device scalar)."""
        p = self.rounded()
        out, (x, mean, rstd), saved = self.hidden(p, tokens, adapter)
        loss, lse = nm.nm_xent(out, p["head"], labels)
        count = (labels >= 0).sum()
        grads = {}
        weight = (1.0 / count).expand(labels.shape[0]).contiguous()
        d, grads["head"] = nm.nm_xent_bwd(out, p["head"], labels, lse, weight)
        d, grads["norm"], grads["norm_bias"] = nm.nm_layernorm_bwd(d.to(BF16), x, mean, rstd, p["norm"])
        for i in reversed(range(LAYERS)):
            x, mean, rstd, h, xa = saved[i]
            values, idx = self.packed[i]
            dh, grads[f"A{i}"], grads[f"B{i}"] = nm.nm_adapter_spmm_bwd(
                values, idx, d, h, xa, adapter, p[f"A{i}"], p[f"B{i}"], self.scale, WIDTH, out_dtype=BF16)
            dx, grads[f"norm{i}"], grads[f"norm{i}_bias"] = nm.nm_layernorm_bwd(dh, x, mean, rstd, p[f"norm{i}"])
            d = d + dx                       # the residual's and the block's
        for k, g in grads.items():
            self.params[k] -= rate * g
        return loss.sum() / count

    def next_tokens(self, tokens, adapter):
        """Serve one token of every request: the most likely next ones."""
        p = self.rounded()
        out, _, _ = self.hidden(p, tokens, adapter)
        return (out.float() @ p["head"].float().t()).argmax(dim=1)


def tasks(device="cuda", seed=1):
    """Each task follows its own permutation of the vocabulary: token t is followed by next[task][t]."""
    g = torch.Generator(device=device).manual_seed(seed)
    return torch.stack([torch.randperm(VOCAB, generator=g, device=device) for _ in range(2)])


def batch(follow, seed):
    """Requests in turn from both tasks; the last token of each has no label."""
    device = follow.device
    g = torch.Generator(device=device).manual_seed(seed)
    adapter = (torch.arange(REQUESTS, device=device) % 2).repeat_interleave(LENGTH)
    tokens = torch.randint(0, VOCAB, (REQUESTS * LENGTH,), generator=g, device=device)
    labels = follow[adapter, tokens]
    labels[LENGTH - 1::LENGTH] = -100
    return tokens, adapter.to(torch.int32), labels.to(torch.int32)


def main(steps=300, rate=2.0):
    model, follow = Model(), tasks()
    losses = [model.step(*batch(follow, 100 + i), rate) for i in range(steps)]
    losses = torch.stack(losses).cpu()
    # serve: 16 requests, both tasks side by side, one token each
    tokens = torch.arange(16, device="cuda") * 7
    adapter = (torch.arange(16, device="cuda") % 2).to(torch.int32)
    right = (model.next_tokens(tokens, adapter) == follow[adapter.long(), tokens]).float().mean().item()
    return losses, right


if __name__ == "__main__":
    n = int(sys.argv[1]) if len(sys.argv) > 1 else 300
    losses, right = main(n)
    for i in range(0, n, max(n // 10, 1)):
        print(f"step {i:4d}  loss {losses[i]:.3f}")
    print(f"step {n:4d}  loss {losses[-1]:.3f}; {right:.0%} of 16 served tokens right")
