"""Cases of the operators for long and sampled sequences around the verified tree.

Four kinds of pass, each as a serving loop makes it:

  window  the target's attention in a layer whose tokens see the last `window`
          positions and the first `sinks` ones, over the paged cache
  weigh   the attention weight that every cached position received from the
          tokens a turn kept, added to what it had
  evict   a step of a sequence held at a budget of positions: pages for new
          tokens, their keys and values written, and the positions of least
          accumulated weight given up again
  verify  a tree of sampled tokens accepted or replaced by the target's
          probabilities, so that the target's distribution is kept

With ``own`` false a pass is elementary torch operations (float32; the
acceptance, whose borders matter, float64); with ``own`` true it is the calls a
user makes of the library.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one chat user, one token a step, a long conversation: the latency of a call
        dict(name="window_b1", op="window", B=1, T=1, Hq=32, Hkv=8, D=128, page=16, lo=9001, hi=9001,
             window=1024, sinks=4, dtype="bf16", mask="chain"),
        # a full batch of ordinary decoding, requests shorter and longer than the window
        dict(name="window_b64", op="window", B=64, T=1, Hq=32, Hkv=8, D=128, page=16, lo=200,
             hi=16000, window=4096, sinks=4, dtype="bf16", mask="chain"),
        # the batched serving setting with a tree of 33 nodes
        dict(name="window_tree", op="window", B=64, T=33, Hq=32, Hkv=8, D=128, page=64, lo=900,
             hi=9000, window=2048, sinks=64, dtype="bf16", mask="tree"),
        # narrow heads, float16, seven query heads to a key head, a window that ends inside
        # pages and is shorter than the tree
        dict(name="window_f16", op="window", B=9, T=61, Hq=14, Hkv=2, D=64, page=32, lo=7, hi=20011,
             window=57, sinks=131, dtype="f16", mask="tree"),
        # one decoding step of one user
        dict(name="weigh_b1", op="weigh", B=1, T=1, Hq=32, Hkv=8, D=128, page=16, lo=1500, hi=1500,
             dtype="bf16", path="all"),
        # a batched turn, the nodes that were accepted
        dict(name="weigh_b64", op="weigh", B=64, T=33, Hq=32, Hkv=8, D=128, page=64, lo=900,
             hi=4100, dtype="bf16", path="some"),
        # chunks of long prompts, seven query heads to a key head
        dict(name="weigh_prompt", op="weigh", B=4, T=256, Hq=28, Hkv=4, D=128, page=32, lo=3000,
             hi=12345, dtype="f16", path="all"),
        # one user at a budget, a turn's tokens more
        dict(name="evict_b1", op="evict", B=1, Hkv=8, D=128, page=16, layers=32, lo=1041, hi=1041,
             keep=1024, sinks=4, recent=128, dtype="bf16"),
        # a batch after a chunk of prompt
        dict(name="evict_b16", op="evict", B=16, Hkv=8, D=128, page=32, layers=16, lo=1500, hi=4000,
             keep=2000, sinks=16, recent=333, dtype="f16"),
        # one block of 16 behind the verified token, siblings at the first positions
        dict(name="verify_b1", op="verify", B=1, T=33, V=151936, replace=False),
        # the batched serving setting
        dict(name="verify_b64", op="verify", B=64, T=33, V=151936, replace=False),
        # a vocabulary of odd size, siblings drawn independently
        dict(name="verify_odd", op="verify", B=7, T=61, V=32003, replace=True),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "weigh", "weigh", "evict", "verify"])
    if op == "verify":
        while True:
            c = dict(op=op, B=_spread(rng, 1, 96), T=_spread(rng, 1, 128), V=_spread(rng, 1000, 262144),
                     replace=rng.random() < 0.5)
            if c["B"] * c["T"] * c["V"] <= 3 << 27 and c["B"] * c["V"] <= 9_000_000:
                return c
    dtype = rng.choice(["bf16", "f16"])
    page = rng.choice([16, 32, 64, 128])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "evict":
        while True:
            c = dict(op=op, B=_spread(rng, 1, 32), Hkv=Hkv, D=D, page=page, layers=_spread(rng, 1, 40),
                     dtype=dtype, keep=_spread(rng, 20, 6000))
            c["lo"] = c["keep"] + rng.randint(-10, 40)
            c["hi"] = c["keep"] + _spread(rng, 40, 4000)
            c["sinks"] = rng.randint(0, c["keep"] // 4)
            c["recent"] = rng.randint(0, c["keep"] // 2)
            if c["B"] * (c["hi"] + page) * Hkv * D * c["layers"] <= 1 << 29:
                return c
    while True:
        c = dict(op=op, B=_spread(rng, 1, 96), T=_spread(rng, 1, 96),
                 Hq=Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8]), Hkv=Hkv, D=D, page=page,
                 lo=_spread(rng, 1, 8000), dtype=dtype)
        c["hi"] = c["lo"] + _spread(rng, 1, 16000)
        if op == "window":
            c.update(window=_spread(rng, 8, 6000), sinks=rng.choice([0, 1, 4, _spread(rng, 1, 300)]),
                     mask=rng.choice(["chain", "tree"]))
        else:
            c["path"] = rng.choice(["all", "some"])
        scores = c["B"] * c["Hq"] * c["T"] * _most_keys(c)
        w, cache = work(c), c["B"] * c["hi"] * Hkv * D
        if w["flops"] <= 6e10 and w["bytes"] <= 9e8 and scores <= 1 << 28 and cache <= 1 << 28:
            return c


# ----------------------------------------------------------------------------- host-side facts
def _lengths(c, n):
    """The sequences' lengths: the same for every seed, so that work() knows them."""
    rng = np.random.RandomState((c["lo"] * 37 + c["hi"] * 19 + n) % (1 << 31))
    v = rng.randint(c["lo"], c["hi"] + 1, n).astype(np.int64)
    v[0] = c["hi"]
    return np.maximum(v, 0)


def _kept_counts(c):
    """How many of a turn's nodes each sequence kept."""
    if c["path"] == "all":
        return np.full(c["B"], c["T"], np.int64)
    rng = np.random.RandomState(c["B"] * 131 + c["T"])
    return np.minimum(c["T"], rng.geometric(0.25, c["B"]))


def _most_keys(c):
    far = c["hi"]
    if c["op"] == "window":
        far = min(far, c["sinks"] + c["window"])
    return far + c["T"]


def work(c):
    if c["op"] == "verify":  # the row of the last draw; what the tests look up is next to nothing
        return {"bytes": float(c["B"] * (c["V"] * 4 + 16 * 12 + c["T"] * 16)), "flops": 0.0}
    row = 2 * c["D"] * c["Hkv"] * 2  # one token's keys and values in one layer
    if c["op"] == "evict":
        full = _lengths(c, c["B"])
        more = np.maximum(0, full - c["keep"])
        move = np.where(more > 0, c["keep"] - c["sinks"], 0)
        return {"bytes": float((more + move).sum() * row * c["layers"] * 2 + full.sum() * 4),
                "flops": 0.0}
    B, T, Hq, D = c["B"], c["T"], c["Hq"], c["D"]
    n = _lengths(c, B)
    if c["op"] == "window":
        n = np.minimum(n, c["sinks"] + c["window"] - 1) + T
        q = B * T * Hq * D * 2
        return {"bytes": float(n.sum() * row + 2 * q + q // D * 2),
                "flops": 4.0 * Hq * D * T * float(n.sum())}
    t = _kept_counts(c)
    q = int(t.sum()) * Hq
    return {"bytes": float((n + t).sum() * (row // 2 + 8) + q * (D * 2 + 4)),
            "flops": 2.0 * Hq * D * float((t * (n + t)).sum())}


# ----------------------------------------------------------------------------- inputs
def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(_dev())


def _parents(rng, B, T):
    """Trees as drafting leaves them: mostly a spine, with siblings near the root."""
    p = np.zeros((B, T), np.int32)
    p[:, 0] = -1
    for i in range(1, T):
        p[:, i] = np.maximum(0, i - rng.geometric(0.45, B))
    return p


def _ancestors(p):
    B, T = p.shape
    a = np.zeros((B, T, T), bool)
    for i in range(T):
        a[:, i, i] = True
        if i:
            a[:, i] |= a[np.arange(B), p[:, i]]
    return a


def _words(flags):
    """Truth values [.., n] as bits of int32 words [.., ceil(n / 32)]."""
    n = flags.shape[-1]
    full = np.zeros(flags.shape[:-1] + ((n + 31) // 32 * 32,), np.uint64)
    full[..., :n] = flags
    w = (full.reshape(flags.shape[:-1] + (-1, 32)) << np.arange(32, dtype=np.uint64)).sum(-1)
    return w.astype(np.uint32).view(np.int32)


def _pool(rng, held, cols, pages):
    """A table whose row b holds held[b] pages, which lie in no order, as after hours of serving."""
    order = rng.permutation(pages)
    table = np.full((len(held), cols), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        refs[order[at:at + n]] = 1
        at += n
    return table, refs


def _prepare_verify(c, rng, g):
    B, T, V = c["B"], c["T"], c["V"]
    z = torch.empty(B, T, V, device=_dev()).normal_(generator=g)
    z[:, :, ::max(1, V // 50)] += 6.0  # the tokens that come into question
    shift = torch.randint(0, V, (1,), generator=g, device=_dev())
    z = torch.roll(z, int(shift), 2)
    cand = torch.topk(z, 16, dim=2).indices
    near = torch.gather(z, 2, cand)
    draft = near + 0.5 * torch.empty_like(near).normal_(generator=g)
    draft, order = torch.sort(draft, dim=2, descending=True)
    cand = torch.gather(cand, 2, order)
    z.sub_(z.amax(2, keepdim=True)).exp_()
    z.div_(z.sum(2, keepdim=True))
    draft = torch.exp(draft - draft.amax(2, keepdim=True))
    q = draft / draft.sum(2, keepdim=True)
    # siblings drawn one after the other from q, without or with replacement
    par = _parents(rng, B, T)
    qn, cn = q.cpu().numpy().astype(np.float64), cand.cpu().numpy()
    if c["replace"]:
        pick = (rng.random_sample((B, T, T, 1)) > qn.cumsum(-1)[:, :, None]).sum(-1).clip(0, 15)
    else:
        pick = np.argsort(-(np.log(qn + 1e-30) + rng.gumbel(size=qn.shape)), axis=-1)
    tokens = rng.randint(0, V, (B, T)).astype(np.int32)
    rank = np.zeros((B, T), np.int64)
    every = np.arange(B)
    for i in range(1, T):
        up = par[:, i]
        r = np.minimum(rank[every, up], pick.shape[-1] - 1)
        tokens[:, i] = cn[every, up, pick[every, up, r]]
        rank[every, up] += 1
    i32 = dict(dtype=torch.int32, device=_dev())
    return {"c": c, "fan": int(rank.max()), "p": z, "q": q.float().contiguous(), "cand": cand.to(torch.int32).contiguous(),
            "tokens": _t(tokens), "parents": _t(par),
            "u": torch.rand(B, T, generator=g, device=_dev()),
            "path": torch.empty(B, T, **i32), "n_path": torch.empty(B, **i32),
            "next": torch.empty(B, **i32)}


def prepare(case, seed):
    c = dict(case)
    rng = np.random.RandomState(int(seed) % (1 << 31))
    g = torch.Generator(device=_dev())
    g.manual_seed(int(seed) * 6007 + 29)
    if c["op"] == "verify":
        return _prepare_verify(c, rng, g)
    dt, ps, H, D, B = DTYPES[c["dtype"]], c["page"], c["Hkv"], c["D"], c["B"]
    f32, i32 = dict(dtype=torch.float32, device=_dev()), dict(dtype=torch.int32, device=_dev())
    n, L = _lengths(c, B), c.get("layers", 1)
    s = {"c": c}
    if c["op"] == "evict":
        base = np.minimum(n, c["keep"])
        more = n - base
        held, most = -(-base // ps), -(-n // ps)
        s.update(full=_t(n.astype(np.int32)), base=_t(base.astype(np.int32)),
                 more=_t(more.astype(np.int32)), kept=torch.empty(B, c["keep"], **i32),
                 new_length=torch.empty(B, **i32), got=torch.empty(B, **i32),
                 served=torch.empty(B, **i32))
        s["new"] = torch.empty(L, B, max(1, int(more.max())), 2, H, D, dtype=dt,
                               device=_dev()).normal_(generator=g)
    else:
        T, Hq = c["T"], c["Hq"]
        held = most = -(-(n + T) // ps)
        s["length"] = _t(n.astype(np.int32))
        # the queries as they leave a joint projection: a strided part of it
        s["q"] = torch.empty(B, T, Hq + 2 * H, D, dtype=dt, device=_dev()).normal_(generator=g)[:, :, :Hq]
    cols, pages = int(most.max()), int(most.sum()) + 3
    table, refs = _pool(rng, held, cols, pages)
    s.update(table=_t(table), refs=_t(refs), bits=_t(_words(refs == 0)))
    s["k"] = torch.empty(L, pages, H, ps, D, dtype=dt, device=_dev()).normal_(generator=g)
    s["v"] = torch.empty_like(s["k"]).normal_(generator=g)
    if c["op"] == "window":
        s["out"] = torch.empty(B, T, Hq, D, dtype=dt, device=_dev())
        s["lse"] = torch.empty(B, T, Hq, **f32)
        s["mask"] = s["depth"] = None
        if c["mask"] == "tree":
            a = _ancestors(_parents(rng, B, T))
            s["mask"], s["depth"] = _t(_words(a)), _t((a.sum(-1) - 1).astype(np.int32))
    else:
        # weights as some turns leave them: a few positions hold most
        s["weight"] = torch.empty(B, cols * ps, **f32).normal_(generator=g).mul_(2.0).exp_()
        s["weight"].mul_(H / c["hi"])
    if c["op"] == "weigh":
        s["path"] = s["n_path"] = None
        t = _kept_counts(c)
        if c["path"] == "some":
            path = np.full((B, T), -1, np.int32)
            for b in range(B):
                path[b, :t[b]] = np.sort(rng.permutation(T)[:t[b]])
            s["path"], s["n_path"] = _t(path), _t(t.astype(np.int32))
        s["first"] = bool(rng.randint(2))
        # what the attention call left: the logarithm of each query's sum
        node, _, x = _weigh_scores(s)
        sums = torch.logsumexp(x, 4).permute(0, 3, 1, 2).reshape(B, T, Hq)
        s["lse"] = torch.empty(B, T, Hq, **f32).normal_(generator=g)
        b, i = torch.nonzero(node >= 0, as_tuple=True)
        s["lse"][b, node[b, i]] = sums[b, i]
    if own:
        import draft_selection_gb300 as dfl2
        s["cache"] = dfl2.Cache(s["k"], s["v"], s["table"], s["refs"], s["bits"])
        if c["op"] == "window":
            s["ws"] = dfl2.workspace(dfl2.dfl2_tree_attn_workspace_size(B, T, Hq, H, D, dt))
        if c["op"] == "evict":
            s["ws"] = dfl2.workspace(dfl2.dfl2_cache_evict_workspace_size(B, c["keep"]))
    return s


# ----------------------------------------------------------------------------- plain forms
def _rows_of(s, pos, there, what):
    """Rows of K or V at positions pos [B, S] of layer 0 as float32 [B, H, S, D], 0 where there is none."""
    ps = s["c"]["page"]
    at = torch.where(there, pos, torch.zeros_like(pos))
    page = torch.gather(s["table"], 1, at // ps).clamp(min=0).long()
    x = s[what][0].permute(0, 2, 1, 3)[page, at % ps].float()
    return (x * there[:, :, None, None]).permute(0, 2, 1, 3)


def _plain_window(s):
    c = s["c"]
    B, T, Hq, H, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
    G, W, sinks, dev = Hq // H, c["window"], c["sinks"], _dev()
    length = s["length"].long()
    near = (length[:, None] - W + 1) + torch.arange(W - 1 + T, device=dev)  # no node sees less
    first = torch.arange(sinks, device=dev).expand(B, sinks)
    pos = torch.cat([first, near], 1)
    there = torch.cat([first < length[:, None] + T, (near >= sinks) & (near >= 0)], 1)
    S = pos.shape[1]
    node = pos - length[:, None]
    i = torch.arange(T, device=dev)
    depth = i.expand(B, T) if s["depth"] is None else s["depth"].long()
    if s["mask"] is None:
        tree = (i[:, None] >= i).expand(B, T, T)
    else:
        tree = (s["mask"][:, :, i // 32] >> (i % 32)) & 1 == 1
    at = node.clamp(0, T - 1)
    is_node = (node >= 0)[:, None]
    seen = torch.gather(tree, 2, at[:, None].expand(B, T, S)) | ~is_node
    place = torch.where(node < 0, pos, length[:, None] + torch.gather(depth, 1, at))
    seen = seen & ((place < sinks)[:, None] | (place[:, None] > (length[:, None] + depth - W)[:, :, None]))
    seen = seen & there[:, None]
    k, v = _rows_of(s, pos, there, "k"), _rows_of(s, pos, there, "v")
    q = s["q"].float().view(B, T, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * T, D)
    x = torch.matmul(q, k.transpose(2, 3)).view(B, H, G, T, S) / math.sqrt(D)
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, H, G * T, S), v).view(B, H, G, T, D)
    o = torch.where(z > 0, o / z, torch.zeros_like(o))
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(s["q"].dtype),
            "lse": (m + torch.log(z))[..., 0].permute(0, 3, 1, 2).reshape(B, T, Hq)}


def _weigh_scores(s):
    """The kept queries' node numbers [B, T] (-1 past their count), their places among the
    positions, and their scores [B, H, G, T, S], -inf where a query does not see a position."""
    c = s["c"]
    B, T, Hq, H, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
    G, dev, length = Hq // H, _dev(), s["length"].long()
    S = s["table"].shape[1] * c["page"]
    i = torch.arange(T, device=dev).expand(B, T)
    node = i if s["path"] is None else s["path"].long()
    n = torch.full_like(length, T) if s["n_path"] is None else s["n_path"].long()
    node = torch.where(i < n[:, None], node, torch.full_like(node, -1))
    q = torch.gather(s["q"].float(), 1, node.clamp(min=0)[:, :, None, None].expand(B, T, Hq, D))
    q = q.view(B, T, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * T, D)
    pos = torch.arange(S, device=dev).expand(B, S)
    k = _rows_of(s, pos, pos < (length + n)[:, None], "k")
    x = torch.matmul(q, k.transpose(2, 3)).view(B, H, G, T, S) / math.sqrt(D)
    seen = (pos[:, None] <= length[:, None, None] + i[:, :, None]) & (node >= 0)[:, :, None]
    return node, pos, x.masked_fill(~seen[:, None, None], -math.inf)


def _plain_weigh(s):
    c = s["c"]
    B, T, H = c["B"], c["T"], c["Hkv"]
    node, pos, x = _weigh_scores(s)
    lse = torch.gather(s["lse"], 1, node.clamp(min=0)[:, :, None].expand(-1, -1, c["Hq"]))
    lse = lse.view(B, T, H, -1).permute(0, 2, 3, 1)[..., None]
    got = torch.exp(x - lse).sum((1, 2, 3))
    new = (pos >= s["length"][:, None]) & (pos < s["length"][:, None] + (node >= 0).sum(1)[:, None])
    old = torch.where(new & s["first"], torch.zeros_like(got), s["weight"])
    s["weight"].copy_(old + got)


def _plain_evict(s):
    c = s["c"]
    ps, B, keep, dev = c["page"], c["B"], c["keep"], _dev()
    table, refs, full, base, more = s["table"], s["refs"], s["full"].long(), s["base"].long(), s["more"]
    col = torch.arange(table.shape[1], device=dev)
    # pages for the new tokens, the lowest free ones first
    need = (col < ((full + ps - 1) // ps)[:, None]) & (table < 0) & (more > 0)[:, None]
    order = torch.argsort((refs != 0).to(torch.int8), stable=True)
    ok = need.sum(1).cumsum(0) <= (refs == 0).sum()
    rank = (need.view(-1).cumsum(0).view(need.shape) - 1).clamp(0, refs.numel() - 1)
    page = torch.where(need, order[rank].to(torch.int32), table)
    refs.index_add_(0, page.clamp(min=0).view(-1).long(), need.view(-1).to(torch.int32))
    table.copy_(page)
    s["got"].copy_(ok)
    # their keys and values
    b, t = torch.nonzero(torch.arange(s["new"].shape[2], device=dev) < more[:, None], as_tuple=True)
    pos = base[b] + t
    k, v = s["k"].permute(1, 3, 0, 2, 4), s["v"].permute(1, 3, 0, 2, 4)
    at = table[b, pos // ps].long()
    k[at, pos % ps] = s["new"][:, b, t, 0].transpose(0, 1)
    v[at, pos % ps] = s["new"][:, b, t, 1].transpose(0, 1)
    # the positions that stay
    S = table.shape[1] * ps
    pos = torch.arange(S, device=dev).expand(B, S)
    w = torch.where(torch.isnan(s["weight"]), torch.full_like(s["weight"], -math.inf), s["weight"])
    by_weight = torch.argsort(w, dim=1, descending=True, stable=True)
    group = torch.where(pos >= full[:, None], 2, 1)
    group = torch.where((pos < c["sinks"]) | (pos >= full[:, None] - c["recent"]) & (group < 2), 0, group)
    group = torch.gather(group, 1, by_weight)
    first = torch.gather(by_weight, 1, torch.argsort(group, dim=1, stable=True))[:, :keep]
    first = torch.where((full > keep)[:, None], torch.sort(first, dim=1).values, pos[:, :keep])
    s["kept"].copy_(torch.where(first < full[:, None], first, torch.full_like(first, -1)))
    b, i = torch.nonzero((s["kept"] >= 0) & (full > keep)[:, None], as_tuple=True)
    a = first[b, i]
    pa, pz = table[b, a // ps].long(), table[b, i // ps].long()
    k[pz, i % ps] = k[pa, a % ps]
    v[pz, i % ps] = v[pa, a % ps]
    s["weight"][b, i] = s["weight"][b, a]
    s["new_length"].copy_(torch.minimum(full, torch.full_like(full, keep)))
    s["served"].fill_(1)
    gone = (col >= ((s["new_length"] + ps - 1) // ps)[:, None]) & (table >= 0) & (full > keep)[:, None]
    refs.index_add_(0, table.clamp(min=0).view(-1).long(), -gone.view(-1).to(torch.int32))
    table.copy_(torch.where(gone, torch.full_like(table, -1), table))
    n = refs.numel()
    free = torch.zeros((n + 31) // 32 * 32, dtype=torch.int64, device=dev)
    free[:n] = refs == 0
    word = (free.view(-1, 32) << torch.arange(32, device=dev)).sum(1)
    s["bits"].copy_(torch.where(word >= 1 << 31, word - (1 << 32), word))


def _plain_verify(s):
    c = s["c"]
    B, T, V = c["B"], c["T"], c["V"]
    dev = _dev()
    cand, par = s["cand"].long(), s["parents"].long()
    p, q, u = torch.gather(s["p"], 2, cand).double(), s["q"].double(), s["u"].double()
    node = torch.arange(T, device=dev)
    # the slot of every node's token among its parent's candidates
    up = par.clamp(min=0)
    hit = torch.gather(cand, 1, up[:, :, None].expand(B, T, 16)) == s["tokens"][:, :, None]
    rank = ((par[:, :, None] == par[:, None, :]) & (node < node[:, None])).sum(2)
    # every node's children in turn, all nodes side by side: what is left of the target's mass
    # (r at the candidates, rest elsewhere) and of the drafter's (d)
    r, d, g = p, q, torch.ones(B, T, dtype=torch.float64, device=dev)
    whole = (1.0 - p.sum(2)).clamp(min=0.0)
    rest = whole
    took = torch.full((B, T), -1, dtype=torch.long, device=dev)
    over = torch.zeros(B, T, dtype=torch.bool, device=dev)
    for turn in range(s["fan"]):
        mine = (rank == turn) & (par >= 0)
        child = torch.zeros(B, T + 1, dtype=torch.long, device=dev)
        child.scatter_(1, torch.where(mine, par, torch.full_like(par, T)), node.expand(B, T))
        child = child[:, :T]  # 0: none
        at = torch.gather(hit, 1, child[:, :, None].expand(B, T, 16)) & (child > 0)[:, :, None]
        R, D = rest + r.sum(2), d.sum(2)
        rk, dk = (r * at).sum(2), (d * at).sum(2)
        test = (dk > 0) & (took < 0) & ~over
        yes = test & (torch.gather(u, 1, child) * dk * R < rk * D)
        no = test & ~yes
        took = torch.where(yes, child, took)
        r2 = (r / R[:, :, None] - d / D[:, :, None]).clamp(min=0.0)
        none = no & (rest / R + r2.sum(2) == 0.0)
        over = over | none
        r = torch.where(none[:, :, None], p, torch.where(no[:, :, None], r2, r))
        rest, g = (torch.where(none, x, torch.where(no, y / R, y)) for x, y in ((whole, rest), (torch.ones_like(g), g)))
        if not c["replace"]:
            d = torch.where(no[:, :, None] & at, torch.zeros_like(d), d)
    # the path: nodes that their parents took, and whose ancestors were all taken
    kept = (torch.gather(took, 1, up) == node) | (node == 0)
    for _ in range(T.bit_length()):
        kept = kept & torch.gather(kept, 1, up)
        up = torch.gather(up, 1, up)
    n = kept.sum(1)
    order = torch.argsort((~kept).to(torch.int8), dim=1, stable=True)
    s["path"].copy_(torch.where(node < n[:, None], order, torch.full_like(order, -1)))
    s["n_path"].copy_(n)
    every = torch.arange(B, device=dev)
    last = order[every, n - 1]
    row = s["p"][every, last].double()
    left = row.scatter(1, cand[every, last], r[every, last] / g[every, last][:, None])
    left = torch.where(left.sum(1, keepdim=True) > 0, left, row)
    run_sum = left.cumsum(1)
    more = run_sum > (u[:, 0] * run_sum[:, -1])[:, None]
    end = torch.where(left > 0, torch.arange(V, device=dev), -1).amax(1)
    s["next"].copy_(torch.where(more.any(1), more.to(torch.int8).argmax(1), end))


# ----------------------------------------------------------------------------- one pass
OUT = {"window": ("out", "lse"), "weigh": ("weight",), "verify": ("path", "n_path", "next"),
       "evict": ("k", "v", "weight", "table", "refs", "bits", "kept", "new_length", "got", "served")}


def run(s):
    c = s["c"]
    op = c["op"]
    if not own:
        if op == "window":
            return _plain_window(s)
        {"weigh": _plain_weigh, "evict": _plain_evict, "verify": _plain_verify}[op](s)
        return {n: s[n] for n in OUT[op]}
    import draft_selection_gb300 as dfl2
    if op == "window":
        dfl2.dfl2_window_attn(s["q"], s["cache"], 0, s["length"], s["mask"], s["depth"], c["sinks"],
                              c["window"], s["out"], s["ws"], lse=s["lse"])
    elif op == "weigh":
        dfl2.dfl2_cache_weigh(s["q"], s["lse"], s["cache"], 0, s["length"], s["weight"],
                              path=s["path"], n_path=s["n_path"], first=s["first"])
    elif op == "evict":
        new = s["new"]
        dfl2.dfl2_cache_reserve(s["cache"], s["base"], s["more"], s["got"])
        dfl2.dfl2_cache_write(s["cache"], new[:, :, :, 0], new[:, :, :, 1], s["base"],
                              count=s["more"])
        dfl2.dfl2_cache_evict(s["cache"], s["full"], c["keep"], c["sinks"], c["recent"],
                              s["weight"], s["kept"], s["new_length"], s["served"], s["ws"])
    else:
        dfl2.dfl2_tree_verify(s["p"], s["tokens"], s["parents"], s["cand"], s["q"], s["u"],
                              s["path"], s["n_path"], s["next"], replace=c["replace"])
    return {n: s[n] for n in OUT[op]}


# ----------------------------------------------------------------------------- in 64 bits
def _line(s, what, b, n):
    """A sequence's first n rows of K or V in layer 0, [H, n, D] in 64 bits."""
    pages = s["table"][b, :-(-n // s["c"]["page"])].long()
    x = s[what][0][pages].double()
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :n]


def _exact_window(s):
    c = s["c"]
    B, T, Hq, H, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device=_dev())
    lse = torch.zeros(B, T, Hq, dtype=torch.float64, device=_dev())
    for b in range(B):
        n = int(s["length"][b])
        sees = np.tril(np.ones((T, T), bool))
        deep = np.arange(T)
        if s["mask"] is not None:
            w = s["mask"][b].cpu().numpy().view(np.uint32)
            sees = (w[:, np.arange(T) // 32] >> (np.arange(T) % 32) & 1).astype(bool)
            deep = s["depth"][b].cpu().numpy()
        place = np.concatenate([np.arange(n), n + deep])
        vis = np.concatenate([np.ones((T, n), bool), sees], 1)
        vis &= (place < c["sinks"]) | (place > (n + deep - c["window"])[:, None])
        cols = np.flatnonzero(vis.any(0))
        vis, cols = _t(vis[:, cols]), _t(cols)
        k, v = _line(s, "k", b, n + T)[:, cols], _line(s, "v", b, n + T)[:, cols]
        for h in range(Hq):
            x = s["q"][b, :, h].double() @ k[h * H // Hq].T * D ** -0.5
            x[~vis] = -math.inf
            lse[b, :, h] = torch.logsumexp(x, 1)
            out[b, :, h] = torch.softmax(x, 1) @ v[h * H // Hq]
    return {"out": out, "lse": lse}


def _exact_weigh(s):
    c = s["c"]
    B, T, Hq, H, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
    w = s["weight"].double()
    for b in range(B):
        n = int(s["length"][b])
        nodes = list(range(T)) if s["path"] is None else s["path"][b, :int(s["n_path"][b])].tolist()
        t = len(nodes)
        if s["first"]:
            w[b, n:n + t] = 0
        k = _line(s, "k", b, n + t)
        sees = torch.arange(n + t, device=_dev()) <= n + torch.arange(t, device=_dev())[:, None]
        for h in range(Hq):
            x = s["q"][b, nodes, h].double() @ k[h * H // Hq].T * D ** -0.5
            e = torch.exp(x - s["lse"][b, nodes, h].double()[:, None])
            w[b, :n + t] += (e * sees).sum(0)
    return {"weight": w}


def _exact_evict(s):
    c = s["c"]
    ps, keep = c["page"], c["keep"]
    table, refs = s["table"].cpu().tolist(), s["refs"].cpu().tolist()
    weight = s["weight"].cpu().tolist()
    k, v = s["k"].clone(), s["v"].clone()
    free = [p for p, r in enumerate(refs) if r == 0][::-1]
    lens = s["full"].tolist()
    kept = [[-1] * keep for _ in lens]
    for b, n in enumerate(lens):
        for x in range(-(-n // ps)):
            if table[b][x] < 0:
                table[b][x] = free.pop()
                refs[table[b][x]] = 1
    for b, n in enumerate(lens):
        at = lambda p: (table[b][p // ps], p % ps)  # noqa: E731, B023
        for t, p in enumerate(range(min(n, keep), n)):
            z, i = at(p)
            k[:, z, :, i], v[:, z, :, i] = s["new"][:, b, t, 0], s["new"][:, b, t, 1]
        stay = list(range(n))
        if n > keep:
            mid = range(c["sinks"], n - c["recent"])
            best = sorted(mid, key=lambda j: (-weight[b][j], j))[:keep - c["sinks"] - c["recent"]]  # noqa: B023
            stay = sorted([*range(c["sinks"]), *best, *range(n - c["recent"], n)])
            pairs = [(at(j), at(i)) for i, j in enumerate(stay) if i != j]
            idx = _t(np.array([[*a, *z] for a, z in pairs], np.int64).reshape(-1, 4))
            for y in (k, v):
                y = y.permute(1, 3, 0, 2, 4)
                y[idx[:, 2], idx[:, 3]] = y[idx[:, 0], idx[:, 1]]
            weight[b][:keep] = [weight[b][j] for j in stay]
            for x in range(-(-keep // ps), len(table[b])):
                if table[b][x] >= 0:
                    refs[table[b][x]] -= 1
                    table[b][x] = -1
        kept[b][:len(stay)] = stay
    i = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    one = [1] * len(lens)
    return {"k": k.double(), "v": v.double(), "weight": torch.tensor(weight, dtype=torch.float64),
            "table": i(table), "refs": i(refs), "bits": _t(_words(np.array(refs) == 0)),
            "kept": i(kept), "new_length": i([min(n, keep) for n in lens]), "got": i(one),
            "served": i(one)}


def _exact_verify(s):
    c = s["c"]
    B, T = c["B"], c["T"]
    tokens, par, cand = s["tokens"].tolist(), s["parents"].tolist(), s["cand"].tolist()
    q, u = s["q"].double().tolist(), s["u"].double().tolist()
    paths, counts, nexts = [], [], []
    for b in range(B):
        walk = [0]
        while True:
            cur = walk[-1]
            row = s["p"][b, cur].cpu().numpy().astype(np.float64)
            at, d = cand[b][cur], list(q[b][cur])
            r, off = [float(row[x]) for x in at], 1.0
            rest = max(0.0, 1.0 - math.fsum(r))
            took = None
            for i in range(1, T):
                if par[b][i] != cur or tokens[b][i] not in at:
                    continue
                j = at.index(tokens[b][i])
                if d[j] <= 0:
                    continue
                R, D = rest + math.fsum(r), math.fsum(d)
                if u[b][i] * (d[j] / D) < r[j] / R:
                    took = i
                    break
                r = [max(0.0, x / R - y / D) for x, y in zip(r, d)]
                rest, off = rest / R, off / R
                if rest + math.fsum(r) == 0.0:
                    r, rest, off = [float(row[x]) for x in at], 1.0, 1.0
                    break
                if not c["replace"]:
                    d[j] = 0.0
            if took is None:
                break
            walk.append(took)
        left = row * off
        left[at] = r
        if left.sum() <= 0:
            left = row
        total = np.cumsum(left)
        over = np.flatnonzero(total > u[b][0] * total[-1])
        nexts.append(int(over[0]) if len(over) else int(np.flatnonzero(left > 0)[-1]))
        paths.append(walk + [-1] * (T - len(walk)))
        counts.append(len(walk))
    i = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return {"path": i(paths), "n_path": i(counts), "next": i(nexts)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("window", "weigh") and work(case)["flops"] > 8e12:
        return None  # about a second for each 1e12 operations in 64 bits
    return {"window": _exact_window, "weigh": _exact_weigh, "evict": _exact_evict,
            "verify": _exact_verify}[case["op"]](s)
