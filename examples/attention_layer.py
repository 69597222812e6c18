"""One attention layer on the library, trained on a pack and served from a paged cache.

    python examples/attention_layer.py

Training: the projection's fused output is rotated where it was written and attended sample by
sample; the gradients flow back through both.  Serving: the same layer takes its prompts in
chunks and then token by token, appending to a paged cache (the rotation on the way) and
attending over it; its outputs are compared with the training form's on the whole prompts.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import packed_varlen_rope_gb300 as pr  # noqa: E402
from packed_varlen_rope_gb300 import build  # noqa: E402
from packed_varlen_rope_gb300 import workloads as wl  # noqa: E402


class AttentionLayer(torch.nn.Module):
    def __init__(self, width, n_q_heads, n_kv_heads, head_dim, theta, device):
        super().__init__()
        self.hq, self.hkv, self.d = n_q_heads, n_kv_heads, head_dim
        kw = dict(bias=False, dtype=torch.bfloat16, device=device)
        self.qkv = torch.nn.Linear(width, (n_q_heads + 2 * n_kv_heads) * head_dim, **kw)
        self.out = torch.nn.Linear(n_q_heads * head_dim, width, **kw)
        self.rope = pr.RotaryEmbedding(head_dim, theta)

    def project(self, x):
        return self.qkv(x).view(x.shape[0], self.hq + 2 * self.hkv, self.d).split([self.hq, self.hkv, self.hkv], dim=1)

    def forward(self, x, cu_seqlens):
        """x [tokens, width] of a pack."""
        q, k, v = self.project(x)
        q, k = self.rope(q.clone(), k.clone(), cu_seqlens=cu_seqlens)      # clones: autograd keeps the views apart
        return self.out(pr.apply_attn(q, k, v, cu_seqlens).flatten(1))

    @torch.no_grad()
    def step(self, x, cache, page_table, kv_lens, cu_seqlens):
        """x: the new tokens of every sequence; kv_lens counts them in."""
        q, k, v = self.project(x)
        q = pr.rope_kv_append(q, k, v, cache, page_table, kv_lens, cu_seqlens, self.rope.theta)
        return self.out(pr.attn_paged(q, cache, page_table, kv_lens, cu_seqlens).flatten(1))


def offsets(lengths, device):
    return torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device=device)


def main():
    build.build()
    device = torch.device("cuda:0")
    torch.manual_seed(0)
    w = wl.WORKLOADS[1]
    layer = AttentionLayer(256, 8, 2, 64, w.theta, device)
    lengths = [300, 1, 77, 512]
    x = torch.randn(sum(lengths), 256, device=device).to(torch.bfloat16)
    target = torch.randn_like(x)
    cu = offsets(lengths, device)

    optimiser = torch.optim.Adam(layer.parameters(), lr=1e-2)
    losses = []
    for _ in range(5):
        optimiser.zero_grad()
        loss = (layer(x, cu).float() - target.float()).square().mean()
        loss.backward()
        optimiser.step()
        losses.append(loss.item())
    print("training losses: " + " ".join("%.4f" % v for v in losses))
    assert losses[-1] < losses[0]

    with torch.no_grad():
        whole = layer(x, cu)
    page = 16
    need = [-(-n // page) for n in lengths]
    cache = pr.new_paged_kv_cache(sum(need), page, layer.hkv, layer.d, device=device)
    table = torch.zeros((len(lengths), max(need)), dtype=torch.int32, device=device)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = torch.arange(at, at + n, device=device)
        at += n
    served = torch.empty_like(whole)
    done, starts = [0] * len(lengths), [0, *torch.tensor(lengths).cumsum(0).tolist()[:-1]]
    chunk, steps = 256, 0
    while done != lengths:
        # long prompts come in chunks, the last tokens one at a time
        new = [min(chunk, max(1, n - a - 4)) if a < n else 0 for a, n in zip(done, lengths)]
        rows = torch.cat([torch.arange(b + a, b + a + c, device=device) for a, b, c in zip(done, starts, new)])
        done = [a + c for a, c in zip(done, new)]
        lens = torch.tensor(done, dtype=torch.int32, device=device)
        served[rows] = layer.step(x[rows], cache, table, lens, offsets(new, device))
        steps += 1
    error = float((served.float() - whole.float()).norm() / whole.float().norm())
    print("served in %d steps; difference from the whole prompts: %.2e" % (steps, error))
    assert error < 1e-2 and not pr.attn_fault()


if __name__ == "__main__":
    main()
