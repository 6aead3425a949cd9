"""Plain 64-bit forms of the tree operators for their tests: numpy on the CPU, a request and a node
at a time, written from the definitions in include/mla_decode.h."""
import numpy as np

from mla_speculative_verify_gb300 import inputs
from tests import cache_reference as ref

DV, PAGE = 512, 64


def random_tree(g, nodes, width=3, roots=0.0):
    """Parents of a random tree; with odds ``roots`` a node hangs on nothing."""
    kids, parents = [0] * nodes, [-1]
    for i in range(1, nodes):
        free = [p for p in range(i) if kids[p] < width]
        p = int(g.choice(free))
        if g.random() < roots:
            p = -1
        else:
            kids[p] += 1
        parents.append(p)
    return parents


def lines(parents):
    """For each node its ancestors and itself, root first."""
    out = []
    for i, p in enumerate(parents):
        out.append((out[p] if 0 <= p < i else []) + [i])
    return out


def words(trees, n):
    """Mask words [total, n] (int32) and depths of trees."""
    rows, depths = [], []
    for parents in trees:
        for line in lines(parents):
            bits = sum(1 << a for a in line)
            rows.append([(bits >> (32 * w)) & 0xFFFFFFFF for w in range(n)])
            depths.append(len(line) - 1)
    return np.asarray(rows, np.uint32).reshape(-1, n).view(np.int32), np.asarray(depths, np.int32)


def sees(batch, masks, b, i):
    """The keys that verify token i of request b sees."""
    t0, q, n = int(batch.q_lens[:b].sum()), int(batch.q_lens[b]), int(batch.seq_lens[b])
    row = masks[t0 + i].view(np.uint32)
    own = [n - q + a for a in range(q) if (int(row[a // 32]) >> (a % 32)) & 1]
    return np.concatenate([np.arange(n - q), np.asarray(own, np.int64)]).astype(np.int64)


def attend(batch, masks):
    """out, lse and the bounds of their errors: cache_reference.attend's, over the keys that a row sees."""
    total = batch.q.shape[0]
    out, bound = np.zeros((total, batch.H, DV)), np.zeros((total, batch.H, DV))
    lse, lse_bound = np.full((total, batch.H), -np.inf), np.zeros((total, batch.H))
    for b in range(len(batch.seq_lens)):
        codes, v = batch.codes(b), batch.key_scales(b)
        for i, (t, q, _) in enumerate(batch.rows(b)):
            at = sees(batch, masks, b, i)
            if not len(at):
                continue
            k = codes[at] * v[at, None]
            s = inputs.SM_SCALE * (q @ k.T)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(1, keepdims=True)
            p /= l
            lse[t] = (m + np.log(l))[:, 0]
            ds = ref.score_error(batch, q, k)
            lse_bound[t] = ds.max(1) + 1e-6 * (1 + np.abs(lse[t]))
            out[t] = p @ k[:, :DV]
            term = p * v[at]
            top = term.max(1, keepdims=True)
            small = 2.0 ** -14 * top * (term < 2.0 ** -4 * top)
            bound[t] = ((3 * 2.0 ** -8 + 2 * ds.max(1, keepdims=True)) * (p @ np.abs(k[:, :DV]))
                        + small @ np.abs(codes[at, :DV]) + 1e-30)
    return out, bound, lse, lse_bound


def softmax(x, temp):
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, 3.402823466e38))
    m = x.max()
    if m == -np.inf:
        return np.zeros_like(x)
    e = np.exp((x - m) / temp)
    return e / e.sum()


def verify(logits, draft, tokens, parents, temp, uniforms, noise, width):
    """One request: (path, tokens that come out, margin). ``temp`` 0 is greedy. The margin is how
    near, relative to the larger of the two numbers compared, the nearest decision was."""
    path, out, u, margin = [], [], 0, np.inf

    def apart(a, b):
        return abs(a - b) / max(a, b, 1e-300)

    while True:
        x = np.asarray(logits[u], np.float64)
        vocab = len(x)
        kids = [i for i in range(1, len(parents)) if parents[i] == u] if len(path) + 1 < width else []
        path.append(u)
        go = None
        if temp == 0:
            x = np.where(np.isnan(x), -np.inf, np.minimum(x, 3.402823466e38))
            word = int(np.argmax(x)) if x.max() > -np.inf else -1
            go = next((i for i in kids if tokens[i] == word and word >= 0), None)
        else:
            p = softmax(x, temp)
            r = p.copy()
            q = softmax(np.asarray(draft[u], np.float64), temp) if draft is not None and kids else None
            for i in kids:
                t = tokens[i]
                if not 0 <= t < vocab:
                    continue
                bar = float(uniforms[i]) * r.sum() * (1.0 if q is None else q[t])
                margin = min(margin, apart(bar, r[t])) if r[t] > 0 else margin
                if bar < r[t]:
                    go = i
                    break
                if q is None:
                    r[t] = 0.0
                else:
                    r = np.maximum(r - r.sum() * q, 0.0)
            if go is None:
                r = r if r.max() > 0 else p
                e = np.where(noise >= 1.175494351e-38, noise, 1.175494351e-38)
                key = r / e
                word = int(np.argmax(key)) if key.max() > 0 else -1
                if word >= 0 and vocab > 1:
                    two = np.partition(key, -2)[-2:]
                    margin = min(margin, apart(two[0], two[1]))
        if go is None:
            out.append(word)
            return path, out, margin
        out.append(int(tokens[go]))
        u = go


def commit(values, scales, table, n, q, path, block):
    """One request, one layer: values [pages, 64, 576] float64 (on the e4m3 grid where scales are
    given, [pages, 64 / block]), both changed in place."""
    n0 = n - q

    def at(pos):
        return table[pos // PAGE], pos % PAGE

    moved = [k for k, p in enumerate(path) if p != k]
    if not moved:
        return
    old = [values[at(n0 + path[k])].copy() for k in moved]
    if scales is None:
        for k, row in zip(moved, old):
            values[at(n0 + k)] = row
        return
    s_old = [scales[at(n0 + path[k])[0], at(n0 + path[k])[1] // block] for k in moved]
    first = n0 + moved[0]
    for lo in range(first // block * block, n0 + len(path), block):
        page, slot = at(lo)
        new = [j for j, k in enumerate(moved) if lo <= n0 + k < lo + block]
        stay = range(lo, max(lo, min(first, lo + block)))
        s = max(s_old[j] for j in new)
        was = scales[page, slot // block]
        if len(stay):
            s = max(s, was)
        with np.errstate(divide="ignore", invalid="ignore"):
            for pos in stay:
                if s != was:
                    values[at(pos)] = ref.to_e4m3(np.float32(values[at(pos)]) * (np.float32(was) / np.float32(s)))
            for j in new:
                ratio = np.float32(s_old[j]) / np.float32(s) if s > 0 else np.float32(1)
                values[at(n0 + moved[j])] = ref.to_e4m3(np.float32(old[j]) * ratio)
        scales[page, slot // block] = s
