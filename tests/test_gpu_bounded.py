"""The operators of a long, sampled sequence together, turn after turn as a server makes them:
pages and rows for a tree, attention in a layer with a window and in one without, acceptance by
sampling, compaction, weighing and eviction, against a model that keeps every position's row in
a list."""
import numpy as np
import pytest
import torch

import draft_selection_gb300 as dfl2
from _sampled_ref import accept
from _tree_ref import ancestors, attention, attention_bounds
from test_gpu_tree_attn import _lib  # noqa: F401  (the fixture builds and loads the library)
from test_gpu_tree_verify import make

pytestmark = pytest.mark.gpu


def within(got, ref, dtype, D, n):
    ob, lb = attention_bounds(ref, dtype, D, n)
    assert (np.abs(got[0].double().cpu().numpy() - ref[0]) <= ob).all()
    assert (np.abs(got[1].double().cpu().numpy() - ref[1]) <= lb).all()


@pytest.mark.parametrize("dtype,D,page,captured", [(torch.bfloat16, 128, 16, False),
                                                   (torch.float16, 64, 32, False),
                                                   (torch.bfloat16, 64, 8, True)])
def test_turns(dtype, D, page, captured):
    B, T, Hq, H, V, layers = 3, 13, 4, 2, 211, 2
    keep, sinks, recent, window = 60, 3, 20, 24
    rng = np.random.RandomState(D + page)
    dev = dict(dtype=torch.int32, device="cuda")
    cols = -(-(keep + 2 * T) // page) + 1
    cache = dfl2.cache(layers, B * cols, H, page, D, B, cols, dtype)
    i32 = lambda *s: torch.zeros(*s, **dev)  # noqa: E731
    length, before, after, served, kept = i32(B), i32(B), i32(B), i32(B), i32(B, keep)
    mask, depth, parents, tokens = i32(B, T, 1), i32(B, T), i32(B, T), i32(B, T)
    path, n_path, nxt = i32(B, T), i32(B), i32(B)
    weight = torch.full((B, cols * page), float("nan"), device="cuda")
    q = torch.zeros(layers, B, T, Hq, D, dtype=dtype, device="cuda")
    kv = torch.zeros(layers, B, T, 2, H, D, dtype=dtype, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(layers, B, T, Hq, device="cuda")
    x = make(B, T, V, False, 0)
    p, cand = torch.zeros(B, T, V, device="cuda"), i32(B, T, 16)
    dq, u = torch.zeros(B, T, 16, device="cuda"), torch.zeros(B, T, device="cuda")
    attn_ws = dfl2.workspace(dfl2.dfl2_tree_attn_workspace_size(B, T, Hq, H, D, dtype))
    weigh_ws = dfl2.workspace(dfl2.dfl2_cache_weigh_workspace_size())
    evict_ws = dfl2.workspace(dfl2.dfl2_cache_evict_workspace_size(B, keep))

    def turn():
        dfl2.dfl2_cache_reserve(cache, length, T, served)
        dfl2.dfl2_tree_mask(parents, mask, depth)
        for layer in range(layers):
            dfl2.dfl2_cache_write(cache, kv[layer, :, :, 0], kv[layer, :, :, 1], length, layer=layer)
        dfl2.dfl2_window_attn(q[0], cache, 0, length, mask, depth, sinks, window, out[0], attn_ws,
                              lse=lse[0])
        dfl2.dfl2_tree_attn(q[1], cache, 1, length, mask, out[1], attn_ws, lse=lse[1])
        dfl2.dfl2_tree_verify(p, tokens, parents, cand, dq, u, path, n_path, nxt)
        before.copy_(length)
        dfl2.dfl2_cache_compact(cache, length, T, path, n_path, length)
        dfl2.dfl2_cache_weigh(q[1], lse[1], cache, 1, before, weight, weigh_ws, path=path,
                              n_path=n_path, first=True)
        after.copy_(length)
        dfl2.dfl2_cache_evict(cache, after, keep, sinks, recent, weight, kept, length, served,
                              evict_ws)

    graph = None
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            turn()
    model = [[np.zeros((0, H, D)) for _ in range(2 * layers)] for _ in range(B)]  # K, V by layer
    sums = [np.zeros(0) for _ in range(B)]
    scale = D ** -0.5
    for step in range(40):  # (some 2.4 tokens a turn: the budget is reached after two thirds)
        x = make(B, T, V, False, 100 + step)
        for t, name in ((p, "p"), (tokens, "tokens"), (parents, "parents"), (cand, "cand"), (dq, "q"),
                        (u, "u")):
            t.copy_(torch.from_numpy(np.ascontiguousarray(x[name])))
        g = torch.Generator(device="cuda").manual_seed(step)
        q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        kv.copy_(torch.randn(kv.shape, generator=g, device="cuda"))
        graph.replay() if graph else turn()
        torch.cuda.synchronize()
        assert dfl2.dfl2_device_error() == 0 and served.tolist() == [1] * B
        q64, kv64 = q.double().cpu().numpy(), kv.double().cpu().numpy()
        w = weight.double().cpu().numpy()
        for b in range(B):
            n = len(sums[b])
            assert before[b] == n
            seen = np.concatenate([np.ones((T, n), bool), ancestors(x["parents"][b].tolist())], 1)
            deep = seen[:, n:].sum(1) - 1
            place = np.concatenate([np.arange(n), n + deep])
            near = seen & ((place < sinks) | (place > (n + deep - window)[:, None]))
            for layer, vis in ((0, near), (1, seen)):
                k = np.concatenate([model[b][2 * layer], kv64[layer, b, :, 0]])
                v = np.concatenate([model[b][2 * layer + 1], kv64[layer, b, :, 1]])
                ref = attention(q64[layer, b], k, v, vis, scale)
                within((out[layer, b], lse[layer, b]), ref, dtype, D, n + T)
            want, token = accept(lambda i: x["p"][b, i], x["tokens"][b], x["parents"][b], x["cand"][b],
                                 x["q"][b], x["u"][b], False)
            assert path[b, :int(n_path[b])].tolist() == want and int(nxt[b]) == token
            for z in range(2 * layers):
                model[b][z] = np.concatenate([model[b][z], kv64[z // 2, b, want, z % 2]])
            # weights: float32 sums of terms that are 2^-13 off at most (scores of some 2^3 with
            # D rounded products, and an lse of the same size)
            got = np.zeros(n + len(want))
            for i, node in enumerate(want):
                for h in range(Hq):
                    s = model[b][2][:n + i + 1, h * H // Hq] @ q64[1, b, node, h] * scale
                    got[:n + i + 1] += np.exp(s - float(lse[1, b, node, h]))
            sums[b] = np.concatenate([sums[b], np.zeros(len(want))]) + got
            assert after[b] == len(sums[b])
            keeps = list(range(len(sums[b])))
            if len(keeps) > keep:
                keeps = kept[b].tolist()
                # by the library's own weights, which the sums here follow
                assert len(keeps) == keep == int(length[b])
                assert keeps[:sinks] == list(range(sinks))
                assert keeps[keep - recent:] == list(range(len(sums[b]) - recent, len(sums[b])))
                lost = np.setdiff1d(np.arange(len(sums[b])), keeps)
                mid = np.array(keeps[sinks:keep - recent])
                assert sums[b][lost].max() <= sums[b][mid].min() * (1 + 2.0**-12)
                assert sorted(set(keeps)) == keeps
            sums[b] = sums[b][keeps]
            model[b] = [m[keeps] for m in model[b]]
            assert np.allclose(w[b, :len(keeps)], sums[b], rtol=2.0**-12, atol=0)
            for z in range(2 * layers):
                held = (cache.v if z % 2 else cache.k)[z // 2][cache.table[b, :-(-len(keeps) // page)].long()]
                held = held.transpose(1, 2).reshape(-1, H, D)[:len(keeps)].double().cpu().numpy()
                assert np.array_equal(held, model[b][z])
        used = (cache.table >= 0).sum(1).tolist()
        assert used == [-(-len(s) // page) for s in sums]
        assert int((cache.refs > 0).sum()) == sum(used) == int(cache.refs.sum())
    assert min(len(s) for s in sums) > 13 and max(len(s) for s in sums) == keep
