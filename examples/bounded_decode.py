"""Sampled speculative decoding of long texts in a cache of bounded size, end to end.

The target of tree_decode.py, its first layer with a window (and a few first tokens that
stay visible), decodes several texts by sampling.  Every turn

  1. drafts a tree: at each node of a spine, children drawn without replacement from the
     drafter's 16 best tokens,
  2. runs the target over the tree (dfl2_cache_reserve, dfl2_tree_mask, dfl2_cache_write,
     dfl2_window_attn in the first layer, dfl2_tree_attn in the others),
  3. accepts or replaces the drafted tokens so that the text follows the target's own
     distribution (dfl2_tree_verify), and keeps the accepted rows (dfl2_cache_compact),
  4. adds up the attention that every cached position received from the accepted tokens
     (dfl2_cache_weigh) and, past the budget, gives up those that received least
     (dfl2_cache_evict).  The first layer's window and first tokens are among what stays in any
     case, so that its window is one of the text's positions.

  python examples/bounded_decode.py --turns 60 --keep 96
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from tree_decode import Target, build, dfl2  # noqa: E402


class Windowed(Target):
    """The first layer's tokens see `window` positions and the first `sinks`.  After run(),
    q and lse hold the other layers' queries and the logarithms of their sums."""

    def __init__(self, window, sinks, **kw):
        super().__init__(**kw)
        self.window, self.sinks = window, sinks

    def run(self, tokens, cache, length, pos, depth, mask, ws):
        """tokens [B,T] at text positions pos [B,T], behind `length` cached ones."""
        B, T = tokens.shape
        H, K, D = self.q_heads, self.kv_heads, self.head_dim
        x = self.E[tokens.long()]
        out = torch.empty(B, T, H, D, dtype=x.dtype, device="cuda")
        self.q, self.lse = [], []
        for layer in range(self.layers):
            qkv = (x @ self.W_qkv[layer].T).view(B, T, H + 2 * K, D)
            q, k = self.rotate(qkv[:, :, :H], pos), self.rotate(qkv[:, :, H:H + K], pos)
            dfl2.dfl2_cache_write(cache, k, qkv[:, :, H + K:].contiguous(), length, layer=layer)
            lse = torch.empty(B, T, H, device="cuda")
            if layer == 0:
                dfl2.dfl2_window_attn(q, cache, layer, length, mask, depth, self.sinks, self.window,
                                      out, ws)
            else:
                dfl2.dfl2_tree_attn(q, cache, layer, length, mask, out, ws, lse=lse)
            self.q.append(q)
            self.lse.append(lse)
            x = x + self.mix * (out.view(B, T, H * D) @ self.W_o[layer].T)
        return x


def draft(target, root, spine, children, ws, g, temperature):
    """A tree behind the tokens root [B]: tokens, parents int32 [B,T], and what each node's
    children were drawn from: cand int32 [B,T,16], q float32 [B,T,16]."""
    B, T = root.shape[0], 1 + spine * children
    dev = dict(dtype=torch.int32, device="cuda")
    tokens, parents = torch.zeros(B, T, **dev), torch.full((B, T), -1, **dev)
    cand = torch.arange(16, **dev).expand(B, T, 16).contiguous()
    q = torch.zeros(B, T, 16, device="cuda")
    idx, val = torch.empty(B, 1, 16, **dev), torch.empty(B, 1, 16, device="cuda")
    tokens[:, 0], at = root, 0
    for step in range(spine):
        logits = (target.E[tokens[:, at].long()] @ target.W_lm.T)[:, None].contiguous()
        dfl2.dfl2_topk(logits, idx, val, ws)
        cand[:, at], q[:, at] = idx[:, 0], torch.softmax(val[:, 0] / temperature, 1)
        # the largest of log q plus Gumbel noise: draws without replacement, in order
        noise = -torch.log(-torch.log(torch.rand(B, 16, generator=g, device="cuda").clamp(min=1e-20)))
        order = torch.topk(torch.log(q[:, at]) + noise, children, dim=1).indices
        first = 1 + step * children
        tokens[:, first:first + children] = torch.gather(cand[:, at], 1, order)
        parents[:, first:first + children] = at
        at = first
    return tokens, parents, cand, q


def decode(batch=4, turns=40, keep=96, spine=5, children=3, page=16, window=None, sinks=4, recent=24,
           temperature=0.2, seed=0):
    """window: the first layer's, at most recent + 1, its default.  Returns the emitted tokens of
    each text, the cached lengths, the cache, and how many positions each turn gave up."""
    window = recent + 1 if window is None else window
    if window > recent + 1:  # its last window - 1 cached positions would not be the text's
        raise ValueError(f"window={window} is more than recent + 1 = {recent + 1}")
    dev = dict(dtype=torch.int32, device="cuda")
    target = Windowed(window, sinks, seed=seed)
    V, T = target.V, 1 + spine * children
    cols = -(-(keep + 2 * T) // page) + 1
    cache = dfl2.cache(target.layers, batch * cols, target.kv_heads, page, target.head_dim, batch,
                       cols, torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    length, before, served = torch.zeros(batch, **dev), torch.zeros(batch, **dev), torch.zeros(batch, **dev)
    text = torch.zeros(batch, **dev)  # tokens of each text whose rows have been cached
    root = 17 * torch.arange(1, batch + 1, **dev) % V
    mask = torch.empty(batch, T, (T + 31) // 32, **dev)
    depth, path = torch.empty(batch, T, **dev), torch.empty(batch, T, **dev)
    n_path, next_token = torch.empty(batch, **dev), torch.empty(batch, **dev)
    kept = torch.empty(batch, keep, **dev)
    weight = torch.zeros(batch, cols * page, device="cuda")
    attn_ws = dfl2.workspace(dfl2.dfl2_tree_attn_workspace_size(
        batch, T, target.q_heads, target.kv_heads, target.head_dim, torch.bfloat16))
    top_ws = dfl2.workspace(dfl2.dfl2_topk_workspace_size(batch, 1, V))
    weigh_ws = dfl2.workspace(dfl2.dfl2_cache_weigh_workspace_size())
    evict_ws = dfl2.workspace(dfl2.dfl2_cache_evict_workspace_size(batch, keep))
    emitted = [[int(r)] for r in root]
    gone = []
    for _ in range(turns):
        tokens, parents, cand, q = draft(target, root, spine, children, top_ws, g, temperature)
        dfl2.dfl2_cache_reserve(cache, length, T, served)
        if not bool(served.all()):
            raise RuntimeError("the cache ran out of pages")
        dfl2.dfl2_tree_mask(parents, mask, depth)
        hidden = target.run(tokens, cache, length, text[:, None] + depth, depth, mask, attn_ws)
        p = torch.softmax((hidden @ target.W_lm.T).float() / temperature, 2)
        u = torch.rand(batch, T, generator=g, device="cuda")
        dfl2.dfl2_tree_verify(p, tokens, parents, cand, q, u, path, n_path, next_token)
        before.copy_(length)
        dfl2.dfl2_cache_compact(cache, length, T, path, n_path, length)
        for layer in range(1, target.layers):
            dfl2.dfl2_cache_weigh(target.q[layer], target.lse[layer], cache, layer, before, weight,
                                  weigh_ws, path=path, n_path=n_path, first=layer == 1)
        text += n_path
        long = length.clone()
        dfl2.dfl2_cache_evict(cache, long, keep, sinks, recent, weight, kept, length, served, evict_ws)
        gone.append((long - length).tolist())
        for b in range(batch):  # (only to print the text; a server would read less often)
            at = path[b, 1:int(n_path[b])].long()
            emitted[b] += tokens[b, at].tolist() + [int(next_token[b])]
        root = next_token.clone()
    return emitted, length, cache, gone


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--turns", type=int, default=60)
    ap.add_argument("--keep", type=int, default=96, help="positions that a text may keep")
    a = ap.parse_args()
    build.build()
    emitted, length, cache, gone = decode(a.batch, a.turns, a.keep)
    total = sum(len(t) - 1 for t in emitted)
    print(f"{a.batch} texts, {a.turns} turns: {total / a.turns / a.batch:.2f} tokens a turn; "
          f"{length.tolist()} of {[len(t) for t in emitted]} positions cached, "
          f"{int((cache.refs > 0).sum())} pages in use")
    if dfl2.dfl2_device_error():
        raise SystemExit("a kernel recorded an error")


if __name__ == "__main__":
    main()
