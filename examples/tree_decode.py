"""Speculative decoding with trees of drafted tokens over a paged cache, end to end.

A small target model with random weights (a residual stream of token embeddings,
a few attention layers with grouped heads and rotary positions, an LM head)
decodes several prompts greedily.  Every turn

  1. drafts a tree: a spine of the drafter's best tokens and, at each step, its
     next best as siblings (dfl2_topk over the drafter's logits; the drafter is
     the target without its attention, so it is often right and not always),
  2. takes pages for the tree's nodes (dfl2_cache_reserve) and works out what each
     node sees (dfl2_tree_mask),
  3. runs the target over all nodes at once: per layer the nodes' keys and values
     go into the cache (dfl2_cache_write) and the nodes attend over it
     (dfl2_tree_attn); the LM head's best token per node comes from dfl2_lmhead_topk,
  4. follows the target's tokens through the tree (dfl2_tree_accept) and keeps the
     accepted rows of the cache (dfl2_cache_compact).

Sequence 0's prompt is shared: its continuations are forks (dfl2_cache_fork), and
all sequences are given back at the end (dfl2_cache_free).  PyTorch does the dense
projections and holds the memory.

  python examples/tree_decode.py --turns 12 --check
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import draft_selection_gb300 as dfl2  # noqa: E402
from draft_selection_gb300 import build  # noqa: E402


class Target:
    def __init__(self, V=2048, d=512, layers=3, q_heads=8, kv_heads=2, head_dim=128, mix=0.35,
                 seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s: (torch.randn(*s, generator=g, device="cuda") / math.sqrt(s[-1])).bfloat16()
        self.V, self.d, self.layers = V, d, layers
        self.q_heads, self.kv_heads, self.head_dim, self.mix = q_heads, kv_heads, head_dim, mix
        self.E = torch.randn(V, d, generator=g, device="cuda").bfloat16()
        self.W_qkv = [w((q_heads + 2 * kv_heads) * head_dim, d) for _ in range(layers)]
        self.W_o = [w(d, q_heads * head_dim) for _ in range(layers)]
        self.W_lm = w(V, d)
        self.freq = 10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda") / head_dim)

    def rotate(self, x, pos):
        a = pos[..., None, None].float() * self.freq
        c, s = torch.cos(a), torch.sin(a)
        u, v = x[..., 0::2].float(), x[..., 1::2].float()
        return torch.stack((u * c - v * s, u * s + v * c), -1).flatten(-2).to(x.dtype)

    def run(self, tokens, cache, rows, length, depth, mask, ws):
        """tokens [B,T] behind `length` positions -> hidden [B,T,d]; their keys and values
        are in the cache afterwards."""
        B, T = tokens.shape
        H, K, D = self.q_heads, self.kv_heads, self.head_dim
        pos = length[:, None] + depth
        x = self.E[tokens.long()]
        out = torch.empty(B, T, H, D, dtype=x.dtype, device="cuda")
        for layer in range(self.layers):
            qkv = (x @ self.W_qkv[layer].T).view(B, T, H + 2 * K, D)
            q = self.rotate(qkv[:, :, :H], pos)
            k = self.rotate(qkv[:, :, H:H + K], pos)
            v = qkv[:, :, H + K:].contiguous()
            dfl2.dfl2_cache_write(cache, k, v, length, rows=rows, layer=layer)
            dfl2.dfl2_tree_attn(q, cache, layer, length, mask, out, ws, rows=rows)
            x = x + self.mix * (out.view(B, T, H * D) @ self.W_o[layer].T)
        return x

    def best(self, hidden, ws):
        """The LM head's token per row of hidden [B,T,d]: int32 [B,T] (and its logit)."""
        B, T, _ = hidden.shape
        idx = torch.empty(B, T, 16, dtype=torch.int32, device="cuda")
        val = torch.empty(B, T, 16, dtype=torch.float32, device="cuda")
        dfl2.dfl2_lmhead_topk(hidden.contiguous(), self.W_lm, idx, val, ws)
        return idx[:, :, 0].contiguous(), val


def draft(target, root, spine, siblings, ws):
    """A tree behind the tokens root [B]: `spine` steps, each with the drafter's
    `siblings` next best tokens beside it.  tokens, parents int32 [B, T]."""
    B = root.shape[0]
    tokens, parents, at, cur = [root], [torch.full_like(root, -1)], 0, root
    idx = torch.empty(B, 1, 16, dtype=torch.int32, device="cuda")
    val = torch.empty(B, 1, 16, dtype=torch.float32, device="cuda")
    for _ in range(spine):
        logits = (target.E[cur.long()] @ target.W_lm.T)[:, None].contiguous()
        dfl2.dfl2_topk(logits, idx, val, ws)
        step = len(tokens)
        for z in range(1 + siblings):
            tokens.append(idx[:, 0, z])
            parents.append(torch.full_like(root, at))
        at, cur = step, idx[:, 0, 0].clone()
        tokens[step] = cur
    return torch.stack(tokens, 1).contiguous(), torch.stack(parents, 1).contiguous()


def decode(batch=6, turns=12, prompt=45, spine=6, siblings=2, page=16, seed=0):
    """Returns the target, the emitted tokens of each sequence (prompt first), how many
    each turn kept, and the cache."""
    dev = dict(dtype=torch.int32, device="cuda")
    target = Target(seed=seed)
    V = target.V
    T = 1 + spine * (1 + siblings)
    cols = -(-(prompt + turns * (spine + 1) + T) // page)
    cache = dfl2.cache(target.layers, batch * cols, target.kv_heads, page, target.head_dim, batch,
                       cols, torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    text = torch.randint(0, V, (prompt,), generator=g, **dev)

    # the prompt, all but its last token, as one chain in row 0; the others fork it
    served = torch.zeros(batch, **dev)
    length = torch.zeros(batch, **dev)
    one = slice(0, 1)
    n = prompt - 1
    dfl2.dfl2_cache_reserve(cache, length[one], n, served[one])
    attn_ws = dfl2.workspace(max(
        dfl2.dfl2_tree_attn_workspace_size(b, t, target.q_heads, target.kv_heads, target.head_dim,
                                           torch.bfloat16) for b, t in ((1, n), (batch, T))))
    target.run(text[None, :n].contiguous(), cache, None, length[one],
               torch.arange(n, **dev)[None], None, attn_ws)
    length.fill_(n)
    if batch > 1:
        dfl2.dfl2_cache_fork(cache, torch.zeros(batch - 1, **dev), torch.arange(1, batch, **dev),
                             length[1:].clone(), served[1:].clone())
    # different last tokens make different continuations
    root = (text[-1] + 17 * torch.arange(batch, **dev)) % V

    lm_ws = dfl2.workspace(dfl2.dfl2_lmhead_topk_workspace_size(batch, T, V, target.d))
    top_ws = dfl2.workspace(dfl2.dfl2_topk_workspace_size(batch, 1, V))
    mask = torch.empty(batch, T, (T + 31) // 32, **dev)
    depth, path = torch.empty(batch, T, **dev), torch.empty(batch, T, **dev)
    n_path, next_token = torch.empty(batch, **dev), torch.empty(batch, **dev)
    emitted = [text[:n].tolist() + [int(r)] for r in root]
    kept = []
    for _ in range(turns):
        tokens, parents = draft(target, root, spine, siblings, top_ws)
        dfl2.dfl2_cache_reserve(cache, length, T, served)
        dfl2.dfl2_tree_mask(parents, mask, depth)
        hidden = target.run(tokens, cache, None, length, depth, mask, attn_ws)
        choice, _ = target.best(hidden, lm_ws)
        dfl2.dfl2_tree_accept(tokens, parents, choice, path, n_path, next_token)
        dfl2.dfl2_cache_compact(cache, length, T, path, n_path, length)
        if not bool(served.all()):
            raise RuntimeError("the cache ran out of pages")
        kept.append(n_path.tolist())
        for b in range(batch):  # (only to print the text; a server would read less often)
            p = path[b, 1:int(n_path[b])].long()
            emitted[b] += tokens[b, p].tolist() + [int(next_token[b])]
        root = next_token.clone()
    return target, emitted, kept, cache, length


def check(target, emitted):
    """Every emitted token is the target's own choice after the ones before it, taken
    from one pass over the whole text in a fresh cache: equal, or level with it to the
    rounding of bf16 activations.  Yields each text, the gaps of its tokens' logits to
    the best ones, and the logits' spread."""
    dev = dict(dtype=torch.int32, device="cuda")
    for text in emitted:
        T = len(text) - 1
        cache = dfl2.cache(target.layers, -(-T // 64), target.kv_heads, 64, target.head_dim, 1,
                           -(-T // 64), torch.bfloat16)
        zero, served = torch.zeros(1, **dev), torch.zeros(1, **dev)
        dfl2.dfl2_cache_reserve(cache, zero, T, served)
        ws = dfl2.workspace(dfl2.dfl2_tree_attn_workspace_size(
            1, T, target.q_heads, target.kv_heads, target.head_dim, torch.bfloat16))
        hidden = target.run(torch.tensor([text[:T]], **dev), cache, None, zero,
                            torch.arange(T, **dev)[None], None, ws)
        logits = hidden[0].float() @ target.W_lm.float().T
        want = torch.tensor(text[1:], device="cuda")
        got = logits.gather(1, want[:, None])[:, 0]
        gap = logits.max(1).values - got
        yield text, gap, logits.std()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=6)
    ap.add_argument("--turns", type=int, default=12)
    ap.add_argument("--prompt", type=int, default=45)
    ap.add_argument("--check", action="store_true", help="verify the text against a plain pass")
    a = ap.parse_args()
    build.build()
    target, emitted, kept, cache, length = decode(a.batch, a.turns, a.prompt)
    per_turn = sum(map(sum, kept)) / (len(kept) * a.batch)
    print(f"{a.batch} sequences, {a.turns} turns: {per_turn:.2f} tokens a turn; pages in use "
          f"{int((cache.refs > 0).sum())} of {cache.refs.numel()}")
    if a.check:
        worst = 0.0
        for text, gap, spread in check(target, emitted):
            worst = max(worst, float(gap[a.prompt - 1:].max() / spread))
        print(f"largest gap of an emitted token to the best logit: {worst:.4f} of their spread")
        if worst > 0.1:
            raise SystemExit("the emitted text is not the target's")
    dfl2.dfl2_cache_free(cache, torch.arange(a.batch, dtype=torch.int32, device="cuda"))
    if int((cache.refs != 0).sum()) or dfl2.dfl2_device_error():
        raise SystemExit("pages are left, or a kernel recorded an error")


if __name__ == "__main__":
    main()
