"""The operators of tree verification: what they are measured on.

  masks    a batch of draft trees, given by parents, becomes the visibility words of the decode
  attend   the verify decode of a tree of drafted tokens over the paged cache
  verify   drafted tokens against the target's distribution: the accepted path and the next token
  commit   the accepted path's cache rows, of all layers, become the last rows of the request

Each case is one of these calls. Where ``own`` is false ``run`` computes them from torch's
elementary operations; where it is true it calls the library. ``exact`` states them a second
time, request by request, in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

D, DV, PAGE = 576, 512, 64
SM_SCALE = 1.0 / math.sqrt(192.0)
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one request's draft of a dozen tokens; a serving batch with wide drafts
        dict(name="masks_one", op="masks", batch=1, lo=12, hi=12, width=3, depth=8),
        dict(name="masks_batch", op="masks", batch=512, lo=20, hi=64, width=4, depth=8),
        # eight drafted tokens of one request over a short context: latency
        dict(name="attend_short", op="attend", batch=1, heads=12, q_lo=8, q_hi=8, lo=4096, hi=4096, width=3,
             depth=8, cache="bf16", block=0),
        # a serving batch with a block-scaled cache, small trees of odd sizes
        dict(name="attend_batch", op="attend", batch=32, heads=48, q_lo=5, q_hi=16, lo=8192, hi=16384, width=3,
             depth=8, cache="scaled", block=64),
        # wide trees of a few requests: many rows for each key
        dict(name="attend_wide", op="attend", batch=4, heads=16, q_lo=64, q_hi=64, lo=32768, hi=32768, width=4,
             depth=8, cache="bf16", block=0),
        # one long context and a tree whose size is a prime
        dict(name="attend_long", op="attend", batch=1, heads=12, q_lo=29, q_hi=29, lo=1 << 18, hi=1 << 18, width=4,
             depth=8, cache="e4m3", block=0),
        # one request, a chain drawn from a draft model's distribution: latency
        dict(name="verify_one", op="verify", batch=1, lo=5, hi=5, width=1, depth=8, vocab=131072,
             kind="bf16", draft=True, greedy=False),
        # greedy decoding with trees of the draft's best tokens, an odd vocabulary
        dict(name="verify_greedy", op="verify", batch=8, lo=30, hi=64, width=4, depth=8, vocab=50001,
             kind="fp32", draft=False, greedy=True),
        # a serving batch, trees of the draft's best tokens, a temperature for each request
        dict(name="verify_trees", op="verify", batch=32, lo=12, hi=32, width=3, depth=8, vocab=131072,
             kind="bf16", draft=False, greedy=False),
        # many requests, chains drawn from the draft's distribution
        dict(name="verify_chains", op="verify", batch=256, lo=4, hi=6, width=1, depth=8, vocab=131072,
             kind="bf16", draft=True, greedy=False),
        # a few requests, one layer of a block-scaled cache
        dict(name="commit_few", op="commit", batch=4, nodes=8, layers=1, lo=100, hi=200, cache="scaled", block=16),
        # a serving batch, the whole model's layers
        dict(name="commit_layers", op="commit", batch=128, nodes=32, layers=48, lo=64, hi=250, cache="bf16", block=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["masks", "attend", "verify", "commit"])
    if op == "masks":
        hi = _log(rng, 12, 128)
        return dict(op=op, batch=_log(rng, 1, 32768 // max(hi, 64)), lo=max(12, hi // rng.randint(1, 8)), hi=hi,
                    width=rng.randint(2, 8), depth=rng.randint(3, 12))
    if op == "attend":
        heads, q_hi = rng.choice([1, 6, 12, 16, 24, 33, 48, 96, 128]), _log(rng, 1, 96)
        batch = _log(rng, 1, 32)
        most = min(1 << 20, int(1e8 / (heads * q_hi)))  # keys in all, times the rows that see them
        hi = _log(rng, q_hi, max(q_hi, most // batch))
        kind = rng.choice(["bf16", "bf16", "e4m3", "scaled"])
        return dict(op=op, batch=batch, heads=heads, q_lo=rng.randint(1, q_hi), q_hi=q_hi,
                    lo=max(q_hi, int(hi * rng.uniform(0.4, 1.0))), hi=hi, width=rng.randint(1, 6),
                    depth=rng.randint(3, 12), cache=kind,
                    block=rng.choice([1, 4, 16, 32, 64]) if kind == "scaled" else 0)
    if op == "verify":
        vocab, draft = _log(rng, 1000, 262144), rng.random() < 0.5
        most = max(1, int(1.3e8 / vocab))  # rows of logits
        hi = _log(rng, 1, min(64, most))
        return dict(op=op, batch=_log(rng, 1, max(1, min(256, most // hi))), lo=max(1, hi // rng.randint(1, 4)), hi=hi,
                    width=rng.randint(1, 4), depth=rng.randint(3, 12), vocab=vocab,
                    kind=rng.choice(["bf16", "fp32"]), draft=draft, greedy=not draft and rng.random() < 0.25)
    kind = rng.choice(["bf16", "e4m3", "scaled", "scaled"])
    nodes, layers = _log(rng, 1, 64), _log(rng, 1, 64)
    lo = nodes + rng.randint(0, 150)
    return dict(op=op, batch=_log(rng, 1, min(256, 6144 // layers)), nodes=nodes, layers=layers, lo=lo,
                hi=lo + rng.randint(0, 100), cache=kind,
                block=rng.choice([1, 4, 16, 32, 64]) if kind == "scaled" else 0)


def _sizes(case):
    """Tree sizes and lengths (or accepted tokens): they go by the case alone, so work() knows them."""
    g = np.random.default_rng([case["batch"], case.get("lo", 0), case["hi"], case.get("nodes", 0)])
    if case["op"] in ("masks", "verify"):
        return g.integers(case["lo"], case["hi"] + 1, size=case["batch"]), None
    n = g.integers(case["lo"], case["hi"] + 1, size=case["batch"])
    if case["op"] == "attend":
        return np.minimum(g.integers(case["q_lo"], case["q_hi"] + 1, size=case["batch"]), n), n
    return n, np.minimum(g.integers(1, 9, size=case["batch"]), case["nodes"])


VISITED = 3.2  # rows of logits that a walk down a tree looks at, measured on these inputs


def work(case):
    op = case["op"]
    a, n = _sizes(case)
    if op == "masks":
        words = -(-int(a.max()) // 32)
        return {"bytes": float(a.sum()) * (8 + 4 * words), "flops": float(a.sum())}
    if op == "attend":
        row = {"bf16": 2.0 * D, "e4m3": float(D), "scaled": D + 4.0 / max(1, case["block"])}[case["cache"]]
        rows = float(a.sum()) * case["heads"]
        seen = case["heads"] * float((a * (n - a + 1)).sum())
        return {"bytes": float(n.sum()) * row + rows * (2 * D + 2 * DV + 4), "flops": 2.0 * (D + DV) * seen}
    if op == "verify":
        visited = float(np.minimum(a, VISITED).sum()) * case["vocab"]
        cell = (2 if case["kind"] == "bf16" else 4) * (2 if case["draft"] else 1)
        noise = 0 if case["greedy"] else 4.0 * case["vocab"] * case["batch"]
        return {"bytes": visited * cell + noise, "flops": 4.0 * visited}
    row = 2 * D if case["cache"] == "bf16" else D
    moved = float((n - 1).sum()) * case["layers"]
    return {"bytes": 2.0 * row * moved + 8.0 * float(n.sum()), "flops": moved}


# ------------------------------------------------------------------------------- inputs
def _trees(seed, sizes, width, depth):
    """Parents of every request's nodes (indices within the request, -1 for the root), at most
    ``width`` children each and ``depth`` levels below the root, or as many as the nodes need;
    later nodes hang on recent ones more often than on old ones."""
    r = random.Random(int(seed))
    out = []
    for q in sizes:
        parents, level, left, most = [-1], [0], [width], depth
        open_ = [0]
        for i in range(1, int(q)):
            if not open_:
                most += 1
                open_ = [k for k in range(i) if left[k] and level[k] < most]
            k = len(open_) - 1 - int(len(open_) * r.random() ** 2)
            p = open_[k]
            parents.append(p)
            level.append(level[p] + 1)
            left[p] -= 1
            if left[p] == 0:
                open_.pop(k)
            left.append(width)
            if level[i] < most:
                open_.append(i)
        out.append(parents)
    return out


def _levels(case):
    """Nodes of the longest way down that a case's trees may have."""
    most = case["depth"]
    while sum(case["width"] ** k for k in range(most + 1)) < case["hi"]:
        most += 1
    return min(case["hi"], most + 1)


def _cu(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)


def _flat(trees):
    return np.concatenate([np.asarray(p, np.int32) for p in trees])


def _words(trees, words):
    """Visibility words by the rule that a node sees its parent's tokens and itself: [total, words]."""
    rows = []
    for parents in trees:
        seen = []
        for i, p in enumerate(parents):
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        rows += [[(s >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for s in seen]
    return np.asarray(rows, np.uint32).view(np.int32)


def _pages(g, lens):
    """A page table over one shuffled pool: [B, pages of the longest], and the pool's size."""
    per = (np.asarray(lens) + PAGE - 1) // PAGE
    perm = g.permutation(int(per.sum()))
    table = np.zeros((len(per), max(1, int(per.max()))), np.int32)
    at = 0
    for b, k in enumerate(per):
        table[b, :k] = perm[at:at + k]
        at += int(k)
    return torch.from_numpy(table).cuda(), int(per.sum())


def _quantised(x, block, two):
    """e4m3 codes of rows [pages * 64, 576] and a scale for each block: powers of two, or amax / 448."""
    pages = x.shape[0] // PAGE
    blocks = x.view(pages, PAGE // block, block * D)
    s = blocks.abs().amax(2) / 448.0
    if two:
        s = torch.exp2(torch.ceil(torch.log2(s)))
    codes = (blocks / s[:, :, None]).clamp_(-448.0, 448.0).to(F8).view(torch.uint8).view(pages, PAGE, D)
    return codes, s.contiguous()


def _latent(gen, rows):
    """Latent rows N(0, 1), each token with a magnitude of its own."""
    x = torch.randn((rows, D), generator=gen, device="cuda")
    return x.mul_(torch.exp(0.5 * torch.randn((rows, 1), generator=gen, device="cuda")))


def _prepare_verify(case, st, gen, trees, sizes):
    batch, total, vocab = len(sizes), int(sizes.sum()), case["vocab"]
    kind = torch.bfloat16 if case["kind"] == "bf16" else torch.float32
    # a language model's logits: a wide bell, and a few tokens far above it
    x = torch.randn((total, vocab), generator=gen, device="cuda").mul_(2.0)
    few = torch.randint(0, vocab, (total, 12), generator=gen, device="cuda")
    x.scatter_add_(1, few, torch.empty((total, 12), device="cuda").exponential_(0.4, generator=gen) + 7.0)
    st["logits"] = x.to(kind)
    temp = 0.5 + 0.6 * torch.rand(batch, generator=gen, device="cuda")
    temp[torch.rand(batch, generator=gen, device="cuda") < 0.1] = 0.0  # greedy requests among the others
    st["temperature"] = None if case["greedy"] else temp
    of = torch.from_numpy(np.repeat(np.arange(batch), sizes)).cuda()
    x.add_(torch.randn((total, vocab), generator=gen, device="cuda").mul_(0.6))  # the draft model differs a little
    st["draft"] = x.to(kind) if case["draft"] else None
    flat = torch.from_numpy(_flat(trees)).cuda().long()
    up = (torch.from_numpy(_cu(sizes)).cuda().long()[of] + flat).clamp(min=0)  # a node's parent's row
    rank = np.concatenate([[p[:i].count(v) for i, v in enumerate(p)] for p in trees]).astype(np.int64)
    if case["draft"]:
        tokens = torch.empty(total, dtype=torch.long, device="cuda")
        for a in range(0, total, 256):  # each node's token drawn from its parent's distribution
            rows = up[a:a + 256]
            t = torch.where(temp[of[rows]] > 0, temp[of[rows]], torch.full_like(temp[of[rows]], 0.05))
            y = st["draft"][rows].float().div_(t[:, None])
            y.sub_(torch.empty_like(y).exponential_(generator=gen).log_())
            tokens[a:a + 256] = y.argmax(1)
    else:
        best = x.topk(case["width"], dim=1).indices
        tokens = best[up, torch.from_numpy(rank).cuda()]
    st["tokens"] = tokens.int()
    st["uniforms"] = st["noise"] = None
    if not case["greedy"]:
        st["uniforms"] = torch.rand(total, generator=gen, device="cuda")
        st["noise"] = torch.empty((batch, vocab), device="cuda").exponential_(generator=gen).clamp_(min=1e-30)
    st["levels"] = _levels(case)
    for k in ("path", "out"):
        st[k] = torch.full((batch, st["levels"]), -1, dtype=torch.int32, device="cuda")
    st["accepted"] = torch.zeros(batch, dtype=torch.int32, device="cuda")
    return st


def _prepare_commit(case, st, gen, g, n, accepted):
    nodes, layers = case["nodes"], case["layers"]
    st["table"], pool = _pages(g, n)
    st["lens"] = torch.from_numpy(n.astype(np.int32)).cuda()
    st["cu"] = torch.from_numpy((np.arange(len(n) + 1) * nodes).astype(np.int32)).cuda()
    path = np.full((len(n), nodes), -1, np.int32)
    for b, k in enumerate(accepted):
        path[b, 0] = 0
        path[b, 1:k] = 1 + np.sort(g.permutation(nodes - 1)[:k - 1])
    st["path"] = torch.from_numpy(path).cuda()
    st["accepted"] = torch.from_numpy(accepted.astype(np.int32)).cuda()
    st["new_lens"] = torch.zeros(len(n), dtype=torch.int32, device="cuda")
    st["scales"], st["block"] = None, case["block"]
    rows = pool * PAGE
    kv = [_latent(gen, rows) for _ in range(layers)] if layers <= 2 else None
    if case["cache"] == "bf16":
        st["kv"] = torch.empty((layers, pool, PAGE, D), dtype=torch.bfloat16, device="cuda")
        for i in range(layers):
            st["kv"][i] = (kv[i] if kv else _latent(gen, rows)).view(pool, PAGE, D)
        return st
    st["kv"] = torch.empty((layers, pool, PAGE, D), dtype=torch.uint8, device="cuda")
    st["scales"] = torch.empty((layers, pool, PAGE // (case["block"] or PAGE)), device="cuda")
    for i in range(layers):
        x = kv[i] if kv else _latent(gen, rows)
        st["kv"][i], st["scales"][i] = _quantised(x, case["block"] or PAGE, True)
    if case["cache"] == "e4m3":  # one scale for the whole cache: its codes are all there is to move
        st["scales"] = None
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    a, n = _sizes(case)
    g = np.random.default_rng([int(seed), case["batch"], case["hi"]])
    st = {"case": case, "op": case["op"]}
    if case["op"] == "commit":
        return _prepare_commit(case, st, gen, g, a, n)
    trees = _trees(seed, a, case["width"], case["depth"])
    st["sizes"] = a
    st["cu"] = torch.from_numpy(_cu(a)).cuda()
    st["parents"] = torch.from_numpy(_flat(trees)).cuda()
    st["most"] = int(a.max())
    words = -(-st["most"] // 32)
    if case["op"] == "masks":
        st["masks"] = torch.zeros((int(a.sum()), words), dtype=torch.int32, device="cuda")
        st["depths"] = torch.zeros(int(a.sum()), dtype=torch.int32, device="cuda")
        return st
    if case["op"] == "verify":
        return _prepare_verify(case, st, gen, trees, a)
    st["n"], st["q_lens"] = n.astype(np.int32), a.astype(np.int32)
    st["masks"] = torch.from_numpy(_words(trees, words)).cuda()
    st["trees"] = trees
    st["lens"], st["q_dev"] = torch.from_numpy(st["n"]).cuda(), torch.from_numpy(st["q_lens"]).cuda()
    st["table"], pool = _pages(g, n)
    x = _latent(gen, pool * PAGE)
    st["kv_scale"], st["scales"], st["block"] = 1.0, None, case["block"]
    if case["cache"] == "bf16":
        st["kv"] = x.to(torch.bfloat16).view(pool, PAGE, D)
    elif case["cache"] == "e4m3":
        st["kv_scale"] = float(x.abs().max()) / 448.0
        st["kv"] = (x / st["kv_scale"]).clamp_(-448.0, 448.0).to(F8).view(torch.uint8).view(pool, PAGE, D)
    else:
        st["kv"], st["scales"] = _quantised(x, case["block"], False)
    del x
    total = int(a.sum())
    st["of"] = torch.from_numpy(np.repeat(np.arange(len(a)), a)).cuda()
    st["nth"] = torch.from_numpy(np.concatenate([np.arange(k) for k in a])).cuda()
    st["q"] = torch.randn((total, case["heads"], D), generator=gen, device="cuda").to(torch.bfloat16)
    st["out"] = torch.empty((total, case["heads"], DV), dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.empty((total, case["heads"]), device="cuda")
    if own:
        from mla_speculative_verify_gb300.decoder import VerifyDecoder

        kind = "bf16" if case["cache"] == "bf16" else "fp8"
        st["decoder"] = VerifyDecoder(st["n"], st["q_lens"], case["heads"], kind, tree=True)
    return st


# ------------------------------------------------------------------------------- the plain forms
def _by_request(st, x, fill):
    """[total] values as [B, most], ``fill`` behind a request's last."""
    cu = st["cu"].long()
    j = torch.arange(st["most"], device="cuda")
    at = (cu[:-1, None] + j).clamp(max=x.shape[0] - 1)
    return torch.where(j < (cu[1:] - cu[:-1])[:, None], x[at], torch.full_like(x[at], fill))


def _masks(st):
    """A tree's reach by squaring: ancestors within 1, 2, 4, .. steps."""
    parents = _by_request(st, st["parents"], -1).long()
    n = st["most"]
    eye = torch.eye(n, device="cuda")
    reach = eye + torch.where(parents[:, :, None] == torch.arange(n, device="cuda"), 1.0, 0.0)
    for _ in range(max(1, (n - 1).bit_length())):
        reach = ((reach @ reach) > 0).float()
    cu, words = st["cu"].long(), st["masks"].shape[1]
    of = torch.searchsorted(cu, torch.arange(st["parents"].shape[0], device="cuda"), right=True) - 1
    seen = reach[of, torch.arange(st["parents"].shape[0], device="cuda") - cu[of]] > 0  # [total, n]
    bits = torch.nn.functional.pad(seen, (0, 32 * words - n)).view(-1, words, 32).long()
    w = (bits << torch.arange(32, device="cuda")).sum(2)
    st["masks"].copy_(torch.where(w >= 1 << 31, w - (1 << 32), w))
    st["depths"].copy_(seen.sum(1) - 1)
    return {"masks": st["masks"], "depths": st["depths"]}


def _attend(st):
    heads, batch, most = st["q"].shape[1], len(st["n"]), st["most"]
    lens, q_dev, cu = st["lens"].long(), st["q_dev"].long(), st["cu"].long()
    j = torch.arange(int(st["n"].max()), device="cuda")
    slot = st["table"].long()[:, j // PAGE] * PAGE + j % PAGE
    kv = st["kv"].view(-1, D)[slot]
    k = kv.float() if kv.dtype == torch.bfloat16 else kv.view(F8).float()
    if st["scales"] is not None:
        k = k * st["scales"].view(-1)[slot // st["block"]][:, :, None]
    elif kv.dtype == torch.uint8:
        k = k * st["kv_scale"]
    i = torch.arange(most, device="cuda")
    tok = (cu[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    s = (st["q"][tok].float().view(batch, most * heads, D) @ k.transpose(1, 2)).mul_(SM_SCALE)
    # draft token a of the request is key lens - q + a: its bit says whether token i sees it
    bits = (st["masks"][tok][:, :, i // 32] >> (i % 32)) & 1  # [B, most, most]
    rel = j - (lens - q_dev)[:, None]
    sees = bits.gather(2, rel.clamp(0, most - 1)[:, None, :].expand(-1, most, -1)) > 0
    sees = (rel < 0)[:, None, :] | (sees & (rel < q_dev[:, None])[:, None, :])
    s.masked_fill_(~sees.repeat_interleave(heads, 1), -math.inf)
    m = s.amax(2, keepdim=True)
    p = torch.exp(s.sub_(m))
    l = p.sum(2, keepdim=True)
    o = (p @ k[:, :, :DV]) / l
    of, nth = st["of"], st["nth"]
    return {"out": o.view(batch, most, heads, DV)[of, nth].to(torch.bfloat16),
            "lse": (m + torch.log(l)).view(batch, most, heads)[of, nth]}


def _verify(st):
    """The walk, all requests together: a level of the tree a step, a child a turn."""
    c = st["case"]
    batch, vocab = st["cu"].shape[0] - 1, c["vocab"]
    cu = st["cu"].long()
    parents, tokens = _by_request(st, st["parents"], -2).long(), _by_request(st, st["tokens"], 0).long()
    u = torch.zeros(batch, dtype=torch.long, device="cuda")
    alive = torch.ones(batch, dtype=torch.bool, device="cuda")
    path, out = torch.full_like(st["path"], -1), torch.full_like(st["out"], -1)
    count = torch.zeros_like(st["accepted"])
    greedy = torch.ones(batch, dtype=torch.bool, device="cuda") if st["temperature"] is None else st["temperature"] == 0
    temp = None if st["temperature"] is None else torch.where(greedy, 1.0, st["temperature"].double())[:, None]
    for step in range(st["levels"]):
        row = (cu[:-1] + u).clamp(max=st["logits"].shape[0] - 1)
        x = st["logits"][row]
        best = x.float().amax(1, keepdim=True)
        top = torch.where(x.float() == best, torch.arange(vocab, device="cuda"), vocab).amin(1)
        if temp is not None:
            r = torch.exp((x.double() - best) / temp)
            r = r / r.sum(1, keepdim=True)
            left = torch.ones(batch, dtype=torch.float64, device="cuda")
            taken = torch.zeros_like(left)
            p0 = r
            if st["draft"] is not None:
                q = st["draft"][row].double()
                q = torch.exp((q - q.amax(1, keepdim=True)) / temp)
                q = q / q.sum(1, keepdim=True)
        hit = torch.full_like(u, -1)
        kids = parents == u[:, None]
        nth = kids.cumsum(1) * kids
        for k in range(c["width"] if step + 1 < st["levels"] else 0):
            is_k = nth == k + 1
            child = is_k.int().argmax(1)
            has = is_k.any(1) & (hit < 0) & alive
            t = tokens.gather(1, child[:, None])
            ok = t[:, 0] == top
            if temp is not None:
                px = r.gather(1, t)[:, 0]
                coin = _by_request(st, st["uniforms"], 1.0).gather(1, child[:, None])[:, 0].double() * left
                if st["draft"] is not None:
                    coin = coin * q.gather(1, t)[:, 0]
                ok = torch.where(greedy, ok, coin < px)
                no = has & ~ok
                if st["draft"] is not None:
                    taken = taken + torch.where(no, left, 0.0)
                    r = torch.where(no[:, None], (p0 - taken[:, None] * q).clamp_(min=0.0), r)
                else:
                    r = r.scatter(1, t, torch.where(no, 0.0, px)[:, None])
                left = torch.where(no, r.sum(1), left)
            hit = torch.where(has & ok, child, hit)
        last = top
        if temp is not None:
            r = torch.where((r.amax(1, keepdim=True) > 0), r, p0)
            last = torch.where(greedy, top, (r / st["noise"]).argmax(1))
        goes = alive & (hit >= 0)
        path[:, step] = torch.where(alive, u, -1).int()
        word = torch.where(goes, tokens.gather(1, hit.clamp(min=0)[:, None])[:, 0], last)
        out[:, step] = torch.where(alive, word, -1).int()
        count += alive.int()
        u, alive = torch.where(goes, hit, u), goes
    for k, v in (("path", path), ("out", out), ("accepted", count)):
        st[k].copy_(v)
    return {"path": st["path"], "tokens": st["out"], "accepted": st["accepted"]}


def _values(st):
    return st["kv"] if st["kv"].dtype == torch.bfloat16 else st["kv"].view(F8)


def _commit(st):
    c = st["case"]
    layers, nodes, batch = c["layers"], c["nodes"], st["lens"].shape[0]
    first = st["lens"].long() - nodes                    # position of node 0
    k = torch.arange(nodes, device="cuda")
    path = st["path"].long()
    goes = (k < st["accepted"][:, None]) & (path > k)    # rows that change place
    table = st["table"].long()

    def slot(pos):
        return table.gather(1, (pos // PAGE).clamp(0, table.shape[1] - 1)) * PAGE + pos % PAGE

    src, dst = slot(first[:, None] + path.clamp(min=0))[goes], slot(first[:, None] + k)[goes]
    st["new_lens"].copy_(first + st["accepted"])
    kv = st["kv"].view(layers, -1, D)
    if st["scales"] is None:
        kv[:, dst] = kv[:, src]
        return {"kv": _values(st), "lens": st["new_lens"]}
    block = st["block"]
    scales = st["scales"].view(layers, -1)
    old = scales[:, src // block]
    need = torch.zeros_like(scales).scatter_reduce_(1, (dst // block).expand(layers, -1), old, "amax")
    hit = torch.zeros_like(scales[0], dtype=torch.bool).index_fill_(0, dst // block, True)
    # the block of a request's first moved row may begin with rows that stay
    stay = first + torch.where(goes.any(1), goes.int().argmax(1), 0)
    j = stay[:, None] // block * block + torch.arange(block, device="cuda")
    is_old = (j < stay[:, None]) & goes.any(1)[:, None]
    old_slot = slot(j)[is_old]
    had = torch.zeros_like(hit).index_fill_(0, old_slot // block, True)
    new = torch.where(hit, torch.where(had, torch.maximum(scales, need), need), scales)
    rows = torch.cat([old_slot, dst])
    ratio = torch.cat([scales[:, old_slot // block], old], 1) / new[:, rows // block]
    vals = kv[:, torch.cat([old_slot, src])].view(F8).float()
    kv[:, rows] = (vals * ratio[:, :, None]).to(F8).view(torch.uint8)
    scales.copy_(new)
    return {"kv": _values(st), "scales": st["scales"], "lens": st["new_lens"]}


def _own(st):
    from mla_speculative_verify_gb300 import cache, tree

    if st["op"] == "masks":
        tree.masks(st["parents"], st["cu"], st["masks"], st["depths"], st["most"])
        return {"masks": st["masks"], "depths": st["depths"]}
    if st["op"] == "attend":
        st["decoder"].run(st["q"], st["kv"], st["table"], st["out"], st["lse"], SM_SCALE, st["kv_scale"],
                          kv_scales=st["scales"], tree_masks=st["masks"])
        return {"out": st["out"], "lse": st["lse"]}
    if st["op"] == "verify":
        tree.verify(st["logits"], st["tokens"], st["parents"], st["cu"], st["path"], st["out"], st["accepted"],
                    temperature=st["temperature"], uniforms=st["uniforms"], noise=st["noise"],
                    draft_logits=st["draft"], max_nodes=st["most"])
        return {"path": st["path"], "tokens": st["out"], "accepted": st["accepted"]}
    cache.commit(st["kv"], st["table"], st["lens"], st["cu"], st["path"], st["accepted"], st["new_lens"], st["scales"])
    if st["scales"] is None:
        return {"kv": _values(st), "lens": st["new_lens"]}
    return {"kv": _values(st), "scales": st["scales"], "lens": st["new_lens"]}


def run(state):
    if own:
        return _own(state)
    return {"masks": _masks, "attend": _attend, "verify": _verify, "commit": _commit}[state["op"]](state)


# ------------------------------------------------------------------------------- in 64 bits
def _exact_masks(st):
    parents, cu = st["parents"].tolist(), st["cu"].tolist()
    trees = [parents[a:b] for a, b in zip(cu, cu[1:])]
    depths = []
    for t in trees:
        d = []
        for p in t:
            d.append(d[p] + 1 if p >= 0 else 0)
        depths += d
    return {"masks": torch.from_numpy(_words(trees, st["masks"].shape[1])), "depths": torch.tensor(depths)}


def _exact_attend(st):
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    t = 0
    for b, parents in enumerate(st["trees"]):
        n, q = int(st["n"][b]), len(parents)
        j = torch.arange(n, device="cuda")
        slot = st["table"][b].long()[j // PAGE] * PAGE + j % PAGE
        k = st["kv"].view(-1, D)[slot]
        k = k.double() if k.dtype == torch.bfloat16 else k.view(F8).double() * st["kv_scale"]
        if st["scales"] is not None:
            k = k * st["scales"].double().view(-1)[slot // st["block"]][:, None]
        for i in range(q):
            line, a = [], i
            while a >= 0:  # the way up to the root
                line.append(n - q + a)
                a = parents[a]
            s = st["q"][t].double() @ torch.cat([k[:n - q], k[line]]).T * SM_SCALE
            lse[t] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[t][:, None])
            out[t] = p[:, :n - q] @ k[:n - q, :DV] + p[:, n - q:] @ k[line, :DV]
            t += 1
    return {"out": out, "lse": lse}


def _exact_verify(st):
    """One request after the other, with cumulative residuals instead of the walk's closed form."""
    cu, parents, tokens = st["cu"].tolist(), st["parents"].tolist(), st["tokens"].tolist()
    path, out, count = torch.full_like(st["path"], -1).cpu(), torch.full_like(st["out"], -1).cpu(), []
    for b in range(len(cu) - 1):
        a, q = cu[b], cu[b + 1] - cu[b]
        temp = 0.0 if st["temperature"] is None else float(st["temperature"][b])
        u, k = 0, 0
        while True:
            x = st["logits"][a + u].double()
            kids = [i for i in range(1, q) if parents[a + i] == u] if k + 1 < st["levels"] else []
            path[b, k] = u
            if temp == 0.0:
                best = int((x == x.max()).nonzero()[0])
                go = next((i for i in kids if tokens[a + i] == best), None)
                word = best
            else:
                p = torch.softmax(x / temp, 0)
                r = p
                d = torch.softmax(st["draft"][a + u].double() / temp, 0) if st["draft"] is not None else None
                go = None
                for i in kids:
                    t = tokens[a + i]
                    share = r / r.sum()
                    if float(st["uniforms"][a + i].double()) * (1.0 if d is None else float(d[t])) < float(share[t]):
                        go = i
                        break
                    if d is None:
                        r = share.clone()
                        r[t] = 0.0
                    else:
                        r = (share - d).clamp(min=0.0)
                word = int(((r if float(r.sum()) > 0 else p) / st["noise"][b].double()).argmax())
            out[b, k] = word if go is None else tokens[a + go]
            k += 1
            if go is None:
                break
            u = go
        count.append(k)
    return {"path": path, "tokens": out, "accepted": torch.tensor(count)}


def _e4m3(x):
    """The e4m3 value next to x (|x| <= 448), ties to even, in 64 bits."""
    _, e = torch.frexp(x)
    step = torch.exp2(((e.double() - 1).clamp(min=-6) - 3))
    return torch.round(x / step) * step


def _exact_commit(st):
    c, block = st["case"], st["block"]
    kv = _values(st).double()
    scales = None if st["scales"] is None else st["scales"].double()
    lens, table = st["lens"].tolist(), st["table"].tolist()
    for b, n in enumerate(lens):
        first, k = n - c["nodes"], int(st["accepted"][b])
        path = st["path"][b, :k].tolist()
        where = [(table[b][(first + i) // PAGE], (first + i) % PAGE) for i in range(c["nodes"])]
        kept = sum(1 for i, p in enumerate(path) if i == p)
        if kept == k:
            continue
        rows = torch.stack([kv[:, where[p][0], where[p][1]] for p in path[kept:]], 1)  # [layers, moved, D]
        if scales is None:
            for i in range(kept, k):
                kv[:, where[i][0], where[i][1]] = rows[:, i - kept]
            continue
        of = torch.stack([scales[:, where[p][0], where[p][1] // block] for p in path[kept:]], 1)
        lo = (first + kept) // block * block
        for at in range(lo, first + k, block):
            page, sl = table[b][at // PAGE], at % PAGE
            new = [i for i in range(kept, k) if at <= first + i < at + block]
            olds = range(at, max(at, min(at + block, first + kept)))
            s = of[:, [i - kept for i in new]].amax(1)
            was = scales[:, page, sl // block].clone()
            if len(olds):
                s = torch.maximum(s, was)
                part = kv[:, page, sl:sl + len(olds)]
                kv[:, page, sl:sl + len(olds)] = _e4m3(part * (was / s)[:, None, None])
            for i in new:
                kv[:, page, (first + i) % PAGE] = _e4m3(rows[:, i - kept] * (of[:, i - kept] / s)[:, None])
            scales[:, page, sl // block] = s
    res = {"kv": kv, "lens": st["lens"].cpu() - c["nodes"] + st["accepted"].cpu()}
    return res if scales is None else {**res, "scales": scales}


def exact(case, seed):
    st = prepare(case, seed)
    return {"masks": _exact_masks, "attend": _exact_attend, "verify": _exact_verify,
            "commit": _exact_commit}[case["op"]](st)
