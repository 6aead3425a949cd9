"""The cache operators of the verify decode: what they are measured on.

  append   new latent rows go into a paged e4m3 cache with a scale for each block of tokens
  attend   the verify decode over such a cache
  weights  the attention weight that every cached key received, accumulated over calls
  evict    the keys with the least accumulated weight leave, the others move to new pages

Each case is one of these calls. Where ``own`` is false ``run`` computes them from torch's
elementary operations in fp32; where it is true it calls the library. ``exact`` states them in
64 bits a second time, request by request.
"""
import math

import numpy as np
import torch

own = False

D, DV, PAGE = 576, 512, 64
SM_SCALE = 1.0 / math.sqrt(192.0)
E_MIN, E_MAX = -60, 60   # exponents of a block's scale
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one verify step of a batch: four tokens of each request enter half-filled blocks
        dict(name="append_verify_step", op="append", batch=32, lo=4, hi=4, past=3000, block=16),
        # a batch of short prompts of odd lengths behind prefixes that end inside a page
        dict(name="append_prompts", op="append", batch=8, lo=301, hi=4099, past=130, block=64),
        # one long prompt into an empty cache
        dict(name="append_long_prompt", op="append", batch=1, lo=131072, hi=131072, past=0, block=64),
        # two verify tokens of one request over a short context: latency
        dict(name="attend_short", op="attend", batch=1, heads=12, q_lo=2, q_hi=2, lo=4096, hi=4096, block=16),
        # a serving batch, 1 to 4 verify tokens each
        dict(name="attend_batch", op="attend", batch=32, heads=48, q_lo=1, q_hi=4, lo=16384, hi=32768, block=64),
        # one request with a context of a million tokens, eight verify tokens
        dict(name="attend_million", op="attend", batch=1, heads=12, q_lo=8, q_hi=8, lo=1 << 20, hi=1 << 20, block=64),
        # the same three situations for the weights; the batch has all 128 heads on one GPU
        dict(name="weights_short", op="weights", batch=1, heads=12, q_lo=2, q_hi=2, lo=4096, hi=4096, cache="bf16",
             block=0),
        dict(name="weights_batch", op="weights", batch=32, heads=128, q_lo=1, q_hi=4, lo=8192, hi=16384,
             cache="scaled", block=64),
        dict(name="weights_million", op="weights", batch=1, heads=12, q_lo=8, q_hi=8, lo=1 << 20, hi=1 << 20,
             cache="bf16", block=0),
        # a few conversations shrink to a quarter
        dict(name="evict_few", op="evict", batch=4, lo=3001, hi=4095, budget=1000, first=4, last=128, cache="scaled",
             block=16),
        # a serving batch is cut back to 8192 keys each
        dict(name="evict_batch", op="evict", batch=32, lo=16384, hi=32768, budget=8192, first=16, last=1024,
             cache="scaled", block=64),
        # a context of a million tokens is cut to a quarter
        dict(name="evict_million", op="evict", batch=1, lo=1 << 20, hi=1 << 20, budget=1 << 18, first=64, last=4096,
             cache="bf16", block=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "weights", "evict"])
    block = rng.choice([1, 4, 16, 32, 64])
    batch = _log(rng, 1, 32)
    if op == "append":
        hi = _log(rng, 1, 131072 // batch)
        return dict(op=op, batch=batch, lo=max(1, hi // rng.randint(1, 12)), hi=hi, past=rng.randint(0, 5000), block=block)
    if op == "evict":
        hi = _log(rng, 600, (1 << 20) // batch)
        lo = max(300, int(hi * rng.uniform(0.5, 1.0)))
        budget = max(16, int(hi * rng.uniform(0.05, 0.25)))
        first = rng.randint(0, budget // 8)
        return dict(op=op, batch=batch, lo=lo, hi=hi, budget=budget, first=first, last=rng.randint(0, budget // 4),
                    cache=rng.choice(["bf16", "scaled", "scaled"]), block=block)
    heads = rng.choice([1, 6, 12, 16, 24, 33, 48, 96, 128])
    q_hi = rng.randint(1, 8)
    q_lo = rng.randint(1, q_hi)
    most = min(1 << 20, int(1e8 / (heads * q_hi)))  # keys in all, times the rows that see them
    hi = _log(rng, 64, max(64, most // batch))
    c = dict(op=op, batch=batch, heads=heads, q_lo=q_lo, q_hi=q_hi, lo=max(q_hi, int(hi * rng.uniform(0.4, 1.0))), hi=hi)
    if op == "weights":
        c["cache"] = rng.choice(["bf16", "e4m3", "scaled"])
    c["block"] = block
    return c


def _rng(case, seed):
    return np.random.default_rng([int(seed), case["batch"], case["hi"]])


def _lengths(case):
    """The lengths of a case go by its sizes alone, so that work() knows them."""
    g = np.random.default_rng([case["batch"], case["lo"], case["hi"]])
    n = g.integers(case["lo"], case["hi"] + 1, size=case["batch"])
    if case["op"] == "append":
        past = g.integers(0, case["past"] + 1, size=case["batch"])
        return n, past
    if case["op"] == "evict":
        return n, None
    return n, np.minimum(g.integers(case["q_lo"], case["q_hi"] + 1, size=case["batch"]), n)


def work(case):
    n, other = _lengths(case)
    op = case["op"]
    if op == "append":
        blocks = sum(-(-int(p + k) // case["block"]) - int(p) // case["block"] for k, p in zip(n, other))
        return {"bytes": float(n.sum()) * 3 * D + 4.0 * blocks, "flops": 2.0 * float(n.sum()) * D}
    scaled = case.get("cache", "scaled") == "scaled"
    row = 2 * D if case.get("cache") == "bf16" else D + (4.0 / case["block"] if scaled else 0.0)
    if op == "evict":
        kept = np.minimum(n, case["budget"])
        return {"bytes": 4.0 * float(n.sum()) + float(kept.sum()) * (2 * row + 8), "flops": float(n.sum())}
    rows = float((other * case["heads"]).sum())
    seen = sum(case["heads"] * sum(int(c - q + i + 1) for i in range(int(q))) for c, q in zip(n, other))
    if op == "weights":
        return {"bytes": float(n.sum()) * (row + 8) + rows * (2 * D + 4), "flops": 2.0 * D * seen}
    return {"bytes": float(n.sum()) * row + rows * (2 * D + 2 * DV + 4), "flops": 2.0 * (D + DV) * seen}


# ------------------------------------------------------------------------------- inputs
def _pages(g, lens, extra=0):
    """A page table over one shuffled pool: [B, pages of the longest], and the pool's size."""
    per = (np.asarray(lens) + PAGE - 1) // PAGE
    pool = int(per.sum()) + extra
    perm = g.permutation(pool)
    table = np.zeros((len(per), max(1, int(per.max()))), np.int32)
    at = 0
    for b, k in enumerate(per):
        table[b, :k] = perm[at:at + k]
        at += int(k)
    return torch.from_numpy(table).cuda(), pool


def _latent(gen, rows):
    """Latent rows N(0, 1), each token with a magnitude of its own."""
    x = torch.randn((rows, D), generator=gen, device="cuda")
    return x.mul_(torch.exp(0.5 * torch.randn((rows, 1), generator=gen, device="cuda")))


def _scale_of(amax):
    """The least power of two 2^e, e in [E_MIN, E_MAX], with amax <= 448 * 2^e."""
    f, e = torch.frexp(amax)
    e = torch.where(f <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    return ((e.int() + 127) << 23).view(torch.float32)  # 2^e from its bits


def _quantised(x, block, two):
    """Codes (uint8) of rows in pages and the blocks' scales: powers of two, or amax / 448."""
    pages = x.shape[0] // PAGE
    blocks = x.view(pages, PAGE // block, block * D)
    amax = blocks.abs().amax(2)
    s = _scale_of(amax) if two else amax / 448.0
    codes = (blocks / s[:, :, None]).clamp_(-448.0, 448.0).to(F8).view(torch.uint8).view(pages, PAGE, D)
    return codes, s.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    g = _rng(case, seed)
    n, other = _lengths(case)
    st = {"case": case, "op": case["op"], "block": case["block"]}
    if case["op"] == "append":
        end = n + other
        st["table"], pool = _pages(g, end)
        st["rows"] = _latent(gen, int(n.sum())).to(torch.bfloat16)
        st["codes"], st["scales"] = _quantised(_latent(gen, pool * PAGE).mul_(0.25), case["block"], True)
        st["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
        st["ends"] = torch.from_numpy(end.astype(np.int32)).cuda()
        st["most"] = int(n.max())
        return st
    st["n"] = n.astype(np.int32)
    st["lens"] = torch.from_numpy(st["n"]).cuda()
    st["table"], pool = _pages(g, n)
    x = _latent(gen, pool * PAGE)
    kind = case.get("cache", "scaled")
    st["kv_scale"], st["scales"] = 1.0, None
    if kind == "bf16":
        st["kv"] = x.to(torch.bfloat16).view(pool, PAGE, D)
    elif kind == "e4m3":
        st["kv_scale"] = float(x.abs().max()) / 448.0
        st["kv"] = (x / st["kv_scale"]).clamp_(-448.0, 448.0).to(F8).view(torch.uint8).view(pool, PAGE, D)
    else:
        st["kv"], st["scales"] = _quantised(x, case["block"], case["op"] == "evict")
    del x
    if case["op"] == "evict":
        # sums of attention weights: heavy-tailed, and many keys that nothing looked at
        w = torch.exp(2.0 * torch.randn((len(n), int(n.max())), generator=gen, device="cuda") - 6.0)
        st["weights"] = torch.where(torch.rand(w.shape, generator=gen, device="cuda") < 0.1, torch.zeros_like(w), w)
        kept = np.minimum(n, case["budget"])
        st["table_dst"], pool_dst = _pages(g, kept)
        st["kv_dst"] = torch.zeros((pool_dst, PAGE, D), dtype=st["kv"].dtype, device="cuda")
        st["scales_dst"] = (torch.ones((pool_dst, PAGE // case["block"]), device="cuda")
                            if st["scales"] is not None else None)
        st["kept"] = torch.full((len(n), case["budget"]), -1, dtype=torch.int32, device="cuda")
        st["weights_dst"] = torch.zeros((len(n), case["budget"]), device="cuda")
        st["lens_dst"] = torch.zeros(len(n), dtype=torch.int32, device="cuda")
        return st
    st["q_lens"] = other.astype(np.int32)
    total = int(other.sum())
    st["tok0"] = torch.from_numpy((np.cumsum(other) - other).astype(np.int64)).cuda()
    st["q_dev"] = torch.from_numpy(st["q_lens"]).cuda()
    st["q_most"] = int(other.max())
    st["of"] = torch.from_numpy(np.repeat(np.arange(len(n)), other)).cuda()
    st["nth"] = torch.from_numpy(np.concatenate([np.arange(k) for k in other])).cuda()
    st["q"] = torch.randn((total, case["heads"], D), generator=gen, device="cuda").to(torch.bfloat16)
    st["lse"] = torch.empty((total, case["heads"]), device="cuda")
    if case["op"] == "attend":
        st["out"] = torch.empty((total, case["heads"], DV), dtype=torch.bfloat16, device="cuda")
    else:
        s, _ = _scores(st)
        m = s.amax(2)
        st["lse"] = _packed(st, m + torch.log(torch.exp(s.sub_(m[:, :, None])).sum(2)))
        del s
        # what a few earlier calls left: a key's share of the rows' weight, times 0 to 4
        share = st["q_most"] * case["heads"] / float(n.max())
        st["weights"] = torch.rand((len(n), int(n.max())), generator=gen, device="cuda").mul_(4.0 * share)
    if own:
        from mla_speculative_verify_gb300.decoder import VerifyDecoder

        st["decoder"] = VerifyDecoder(st["n"], st["q_lens"], case["heads"], "bf16" if kind == "bf16" else "fp8")
    return st


# ------------------------------------------------------------------------------- the plain forms
def _slots(table, n):
    """The cache row of every key of every request: [B, n]."""
    j = torch.arange(n, device="cuda")
    return table.long()[:, (j // PAGE).clamp(max=table.shape[1] - 1)] * PAGE + j % PAGE


def _keys(st):
    """All keys in fp32, requests padded to the longest: [B, n, 576]."""
    slot = _slots(st["table"], int(st["n"].max()))
    kv = st["kv"].view(-1, D)
    if kv.dtype == torch.uint8:
        k = kv[slot].view(F8).float()
        if st["scales"] is None:
            return k.mul_(st["kv_scale"])
        return k.mul_(st["scales"].view(-1)[slot // st["block"]][:, :, None])
    return kv[slot].float()


def _scores(st):
    """Scores [B, q * H, n] in fp32 (-inf where masked), requests padded, and the keys."""
    heads, batch, most = st["q"].shape[1], len(st["n"]), st["q_most"]
    k = _keys(st)
    i = torch.arange(most, device="cuda")
    tok = (st["tok0"][:, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][tok].float().view(batch, most * heads, D)
    s = (q @ k.transpose(1, 2)).mul_(SM_SCALE)
    seen = st["lens"].long()[:, None] - st["q_dev"].long()[:, None] + i + 1
    seen = seen.minimum(st["lens"].long()[:, None])
    hidden = torch.arange(k.shape[1], device="cuda") >= seen.repeat_interleave(heads, 1)[:, :, None]
    return s.masked_fill_(hidden, -math.inf), k


def _packed(st, x):
    """Padded rows [B, q * H, ...] to the tokens' own: [total_q, H, ...]."""
    heads = st["q"].shape[1]
    return x.view(x.shape[0], -1, heads, *x.shape[2:])[st["of"], st["nth"]]


def _padded(st, x):
    """[total_q, H] to [B, q * H], +inf where a request has no such token."""
    heads = x.shape[1]
    y = torch.full((len(st["n"]), st["q_most"], heads), math.inf, device="cuda")
    y[st["of"], st["nth"]] = x
    return y.view(len(st["n"]), -1)


def _attend(st):
    s, k = _scores(st)
    m = s.amax(2, keepdim=True)
    p = torch.exp(s.sub_(m))
    l = p.sum(2, keepdim=True)
    o = (p @ k[:, :, :DV]) / l
    return {"out": _packed(st, o).to(torch.bfloat16), "lse": _packed(st, (m + torch.log(l))[:, :, 0])}


DECAY = 0.9375


def _weights(st):
    s, _ = _scores(st)
    w = torch.exp(s.sub_(_padded(st, st["lse"])[:, :, None])).sum(1)
    live = torch.arange(w.shape[1], device="cuda") < st["lens"][:, None]
    st["weights"].copy_(torch.where(live, st["weights"] * DECAY + w, st["weights"]))
    return {"weights": st["weights"]}


def _append(st):
    block, batch = st["block"], st["ends"].shape[0]
    codes, scales = st["codes"].view(-1, D), st["scales"].view(-1)
    cu, ends = st["cu"].long(), st["ends"].long()
    total = st["rows"].shape[0]
    t = torch.arange(total, device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    first = ends - (cu[1:] - cu[:-1])                      # position of a request's first new row
    pos = first[b] + t - cu[b]
    slot = st["table"].long()[b, pos // PAGE] * PAGE + pos % PAGE
    x = st["rows"].float()
    need = torch.zeros_like(scales).scatter_reduce_(0, slot // block, x.abs().amax(1), "amax")
    hit = torch.zeros_like(scales, dtype=torch.bool).index_fill_(0, slot // block, True)
    need = _scale_of(need)
    # the block that a request's past ends in: its old rows stay, in the block's new scale
    j = torch.arange(block, device="cuda")
    old_pos = first[:, None] // block * block + j
    is_old = (old_pos < first[:, None]) & (cu[1:] > cu[:-1])[:, None]
    at = (first // PAGE).clamp(max=st["table"].shape[1] - 1)
    old_slot = st["table"].long()[torch.arange(batch, device="cuda"), at][:, None] * PAGE + old_pos % PAGE
    had = torch.zeros_like(hit)
    had[(old_slot // block)[is_old]] = True
    new = torch.where(hit, torch.where(had, torch.maximum(scales, need), need), scales)
    o = old_slot[is_old]
    ratio = (scales / new)[o // block]
    codes[o] = (codes[o].view(F8).float() * ratio[:, None]).to(F8).view(torch.uint8)
    codes[slot] = (x / new[slot // block][:, None]).clamp(-448.0, 448.0).to(F8).view(torch.uint8)
    scales.copy_(new)
    return {"codes": st["codes"].view(F8), "scales": st["scales"]}


def _evict(st):
    c, w, lens = st["case"], st["weights"], st["lens"].long()
    batch, most = w.shape
    budget = c["budget"]
    j = torch.arange(most, device="cuda")
    always = (j < c["first"]) | (j >= lens[:, None] - c["last"]) | (lens <= budget)[:, None]
    live = j < lens[:, None]
    order = torch.where(live, torch.where(always, torch.full_like(w, math.inf), w), torch.full_like(w, -math.inf))
    order = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :budget]  # ties: the lowest index
    new = lens.clamp(max=budget)
    r = torch.arange(order.shape[1], device="cuda")
    order = torch.where(r < new[:, None], order, torch.full_like(order, most)).sort(dim=1).values
    ok = r < new[:, None]
    src_j = order.clamp(max=most - 1)
    src = st["table"].long().gather(1, (src_j // PAGE).clamp(max=st["table"].shape[1] - 1)) * PAGE + src_j % PAGE
    dst = _slots(st["table_dst"], order.shape[1])
    st["kept"][:, :order.shape[1]] = torch.where(ok, order, torch.full_like(order, -1)).int()
    st["lens_dst"].copy_(new)
    st["weights_dst"][:, :order.shape[1]] = torch.where(ok, w.gather(1, src_j), st["weights_dst"][:, :order.shape[1]])
    src, dst = src[ok], dst[ok]
    kv, kv_dst = st["kv"].view(-1, D), st["kv_dst"].view(-1, D)
    res = {"kept": st["kept"], "lens": st["lens_dst"], "weights": st["weights_dst"]}
    if st["scales"] is None:
        kv_dst[dst] = kv[src]
        return {**res, "kv": st["kv_dst"]}
    block = st["block"]
    old = st["scales"].view(-1)[src // block]
    new_s = torch.zeros_like(st["scales_dst"].view(-1)).scatter_reduce_(0, dst // block, old, "amax")
    s_dst = st["scales_dst"].view(-1)
    s_dst.copy_(torch.where(new_s > 0, new_s, s_dst))
    ratio = old / s_dst[dst // block]
    kv_dst[dst] = (kv[src].view(F8).float() * ratio[:, None]).to(F8).view(torch.uint8)
    return {**res, "kv": st["kv_dst"].view(F8), "scales": st["scales_dst"]}


def _own(st):
    from mla_speculative_verify_gb300 import cache

    if st["op"] == "append":
        cache.append(st["rows"], st["codes"], st["scales"], st["table"], st["ends"], st["cu"], st["most"])
        return {"codes": st["codes"].view(F8), "scales": st["scales"]}
    if st["op"] == "attend":
        st["decoder"].run(st["q"], st["kv"], st["table"], st["out"], st["lse"], SM_SCALE, kv_scales=st["scales"])
        return {"out": st["out"], "lse": st["lse"]}
    if st["op"] == "weights":
        st["decoder"].key_weights(st["q"], st["kv"], st["table"], st["lse"], st["weights"], decay=DECAY,
                                  sm_scale=SM_SCALE, kv_scale=st["kv_scale"], kv_scales=st["scales"])
        return {"weights": st["weights"]}
    c = st["case"]
    cache.evict(st["weights"], st["lens"], c["budget"], c["first"], c["last"], st["kv"], st["table"], st["kv_dst"],
                st["table_dst"], st["kept"], st["lens_dst"], st["weights_dst"], st["scales"], st["scales_dst"])
    res = {"kept": st["kept"], "lens": st["lens_dst"], "weights": st["weights_dst"]}
    if st["scales"] is None:
        return {**res, "kv": st["kv_dst"]}
    return {**res, "kv": st["kv_dst"].view(F8), "scales": st["scales_dst"]}


def run(state):
    if own:
        return _own(state)
    return {"append": _append, "attend": _attend, "weights": _weights, "evict": _evict}[state["op"]](state)


# ------------------------------------------------------------------------------- in 64 bits
def _e4m3(x):
    """The e4m3 value next to x (|x| <= 448 kept, larger ones cut), ties to even, in 64 bits."""
    x = x.clamp(-448.0, 448.0)
    _, e = torch.frexp(x)
    step = (((e.long() - 1).clamp(min=-6) - 3 + 1023) << 52).view(torch.float64)  # 2^k from its bits
    return torch.round(x / step) * step


def _exact_scale(amax):
    """Counts up from the least exponent."""
    s = torch.full_like(amax, 2.0 ** E_MIN)
    for k in range(E_MIN, E_MAX):
        s = torch.where(amax > 448.0 * 2.0 ** k, 2.0 ** (k + 1), s)
    return s


def _exact_append(st):
    block = st["block"]
    vals, scales = st["codes"].view(-1, D).view(F8).double(), st["scales"].double().view(-1)
    cu, ends, table = st["cu"].tolist(), st["ends"].tolist(), st["table"].cpu().numpy().astype(np.int64)
    for b in range(len(ends)):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        p0 = ends[b] - n
        base = p0 // block * block                 # first position of the first touched block
        pos = np.arange(base, ends[b])
        slot = torch.from_numpy(table[b, pos // PAGE] * PAGE + pos % PAGE).cuda()
        pad = -len(pos) % block
        x = torch.zeros((len(pos), D), dtype=torch.float64, device="cuda")
        x[p0 - base:] = st["rows"][cu[b]:cu[b + 1]].double()
        amax = torch.nn.functional.pad(x.abs().amax(1), (0, pad)).view(-1, block).amax(1)
        s_new = _exact_scale(amax)
        ids = slot[::block] // block
        if p0 > base:
            s_new[0] = torch.maximum(s_new[0], scales[ids[0]])
            x[:p0 - base] = vals[slot[:p0 - base]] * scales[ids[0]]
        vals[slot] = _e4m3(x / s_new.repeat_interleave(block)[:len(pos), None])
        scales[ids] = s_new
    return {"codes": vals.view(st["codes"].shape), "scales": scales.view(st["scales"].shape)}


def _exact_keys(st, b):
    n = int(st["n"][b])
    j = torch.arange(n, device="cuda")
    slot = st["table"][b].long()[j // PAGE] * PAGE + j % PAGE
    kv = st["kv"].view(-1, D)[slot]
    if kv.dtype != torch.uint8:
        return kv.double()
    k = kv.view(F8).double()
    return k * st["kv_scale"] if st["scales"] is None else k * st["scales"].double().view(-1)[slot // st["block"]][:, None]


def _exact_rows(st, b):
    """Scores of request b's rows in 64 bits, a token at a time, and its keys."""
    k = _exact_keys(st, b)
    t0, q, n = int(st["tok0"][b]), int(st["q_lens"][b]), int(st["n"][b])
    for i in range(q):
        s = st["q"][t0 + i].double() @ k[:n - q + i + 1].T
        yield t0 + i, s * SM_SCALE, k


def _exact_attend(st):
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    for b in range(len(st["n"])):
        for t, s, k in _exact_rows(st, b):
            lse[t] = torch.logsumexp(s, 1)
            out[t] = torch.exp(s - lse[t][:, None]) @ k[:s.shape[1], :DV]
    return {"out": out, "lse": lse}


def _exact_weights(st):
    w = st["weights"].double()
    for b in range(len(st["n"])):
        w[b, :int(st["n"][b])] *= DECAY
        for t, s, _ in _exact_rows(st, b):
            w[b, :s.shape[1]] += torch.exp(s - st["lse"][t].double()[:, None]).sum(0)
    return {"weights": w}


def _exact_evict(st):
    c, block = st["case"], st["block"]
    w = st["weights"].cpu().numpy()
    kept, w_dst = st["kept"].cpu().numpy().copy(), st["weights_dst"].double().cpu().numpy()
    scaled = st["scales"] is not None
    kv = st["kv"].view(-1, D)
    kv_dst = st["kv_dst"].view(-1, D).view(F8).double() if scaled else st["kv_dst"].view(-1, D).double()
    s_dst = st["scales_dst"].double().view(-1) if scaled else None
    table, table_dst = (st[k].cpu().numpy().astype(np.int64) for k in ("table", "table_dst"))
    for b, n in enumerate(st["n"].tolist()):
        mid = np.arange(c["first"], n - c["last"])
        if n <= c["budget"]:
            keep = np.arange(n)
        else:
            best = mid[np.lexsort((mid, -w[b, mid].astype(np.float64)))][:c["budget"] - c["first"] - c["last"]]
            keep = np.sort(np.concatenate([np.arange(c["first"]), best, np.arange(n - c["last"], n)]))
        kept[b, :len(keep)] = keep
        w_dst[b, :len(keep)] = w[b, keep]
        r = np.arange(len(keep))
        src = torch.from_numpy(table[b, keep // PAGE] * PAGE + keep % PAGE).cuda()
        dst = torch.from_numpy(table_dst[b, r // PAGE] * PAGE + r % PAGE).cuda()
        if not scaled:
            kv_dst[dst] = kv[src].double()
            continue
        old = st["scales"].double().view(-1)[src // block]
        new = torch.nn.functional.pad(old, (0, -len(keep) % block)).view(-1, block).amax(1)
        s_dst[dst[::block] // block] = new
        kv_dst[dst] = _e4m3(kv[src].view(F8).double() * (old / new.repeat_interleave(block)[:len(keep)])[:, None])
    res = {"kept": torch.from_numpy(kept), "lens": torch.from_numpy(np.minimum(st["n"], c["budget"])),
           "weights": torch.from_numpy(w_dst), "kv": kv_dst.view(st["kv_dst"].shape)}
    return {**res, "scales": s_dst.view(st["scales_dst"].shape)} if scaled else res


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "weights": _exact_weights,
            "evict": _exact_evict}[case["op"]](st)
