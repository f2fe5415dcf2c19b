"""dfl2_window_attn over a cache that dfl2_cache_evict holds at a budget: where the last window - 1
positions and the window layer's sinks are kept, it is the window over the text's positions, of
which the cache has lost most."""
import numpy as np
import pytest
import torch

import draft_selection_gb300 as dfl2
from _tree_ref import ancestors, attention, attention_bounds
from test_gpu_tree_attn import _lib, random_parents  # noqa: F401  (the fixture builds and loads)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks,recent", [(24, 3, 23), (24, 3, 30), (7, 0, 6), (1, 2, 0)])
def test_the_window_of_the_text(window, sinks, recent):
    B, T, Hq, H, D, page, keep = 2, 9, 4, 2, 64, 8, 50
    rng = np.random.RandomState(window)
    dev = dict(dtype=torch.int32, device="cuda")
    cols = -(-(keep + 2 * T) // page) + 1
    cache = dfl2.cache(1, B * cols, H, page, D, B, cols, torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, **dev)  # noqa: E731
    length, after, served, kept = i32(B), i32(B), i32(B), i32(B, keep)
    mask, depth, path, n_path = i32(B, T, 1), i32(B, T), i32(B, T), i32(B)
    weight = torch.zeros(B, cols * page, device="cuda")
    attn_ws = dfl2.workspace(dfl2.dfl2_tree_attn_workspace_size(B, T, Hq, H, D, torch.bfloat16))
    evict_ws = dfl2.workspace(dfl2.dfl2_cache_evict_workspace_size(B, keep))
    out = torch.zeros(B, T, Hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(B, T, Hq, device="cuda")
    text = [[np.zeros((0, H, D)) for _ in range(2)] for _ in range(B)]  # every token's K and V
    for step in range(25):
        g = torch.Generator(device="cuda").manual_seed(step)
        q = torch.randn(B, T, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
        kv = torch.randn(B, T, 2, H, D, generator=g, device="cuda").to(torch.bfloat16)
        parents = [random_parents(np.random.default_rng(step * B + b), T) for b in range(B)]
        dfl2.dfl2_cache_reserve(cache, length, T, served)
        dfl2.dfl2_tree_mask(torch.tensor(parents, **dev), mask, depth)
        dfl2.dfl2_cache_write(cache, kv[:, :, 0], kv[:, :, 1], length)
        dfl2.dfl2_window_attn(q, cache, 0, length, mask, depth, sinks, window, out, attn_ws, lse=lse)
        assert served.tolist() == [1] * B
        paths = np.full((B, T), -1, np.int32)
        for b in range(B):
            n = len(text[b][0])
            tree = ancestors(parents[b])
            deep = tree.sum(1) - 1
            place = np.concatenate([np.arange(n), n + deep])
            vis = np.concatenate([np.ones((T, n), bool), tree], 1)
            vis &= (place < sinks) | (place > (n + deep - window)[:, None])
            new = kv[b].double().cpu().numpy()
            k, v = (np.concatenate([text[b][z], new[:, z]]) for z in range(2))
            ref = attention(q[b].double().cpu().numpy(), k, v, vis, D ** -0.5)
            ob, lb = attention_bounds(ref, torch.bfloat16, D, n + T)
            assert (np.abs(out[b].double().cpu().numpy() - ref[0]) <= ob).all(), (step, b)
            assert (np.abs(lse[b].double().cpu().numpy() - ref[1]) <= lb).all(), (step, b)
            node = int(rng.randint(T))
            walk = np.flatnonzero(tree[node])
            paths[b, :len(walk)] = walk
            for z in range(2):
                text[b][z] = np.concatenate([text[b][z], new[walk, z]])
        path.copy_(torch.from_numpy(paths))
        n_path.copy_(torch.from_numpy((paths >= 0).sum(1).astype(np.int32)))
        dfl2.dfl2_cache_compact(cache, length, T, path, n_path, length)
        weight.uniform_(generator=g)
        after.copy_(length)
        dfl2.dfl2_cache_evict(cache, after, keep, sinks, recent, weight, kept, length, served, evict_ws)
        assert served.tolist() == [1] * B
    assert dfl2.dfl2_device_error() == 0
    assert min(len(t[0]) for t in text) > keep and length.tolist() == [keep] * B
