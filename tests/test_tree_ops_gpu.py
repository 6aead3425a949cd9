"""The tree operators on the GPU against plain 64-bit forms: visibility masks, the decode of a tree,
verification of drafted tokens, commit of the accepted path, and all of them as a server runs them."""
import numpy as np
import pytest
import torch

from mla_speculative_verify_gb300 import binding, cache, inputs, tree
from mla_speculative_verify_gb300.decoder import VerifyDecoder
from tests import cache_reference as ref
from tests import tree_reference as tref

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
PAGE, D = 64, 576


def dev(a):
    return (torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a).cuda()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cu_of(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)


def flat(trees):
    return np.asarray([p for t in trees for p in t], np.int32)


# ------------------------------------------------------------------------------- masks
@pytest.mark.parametrize("sizes,words", [([1], 1), ([8], 1), ([32, 33], 2), ([64, 1, 0, 65], 3), ([130, 7], 5), ([1024], 32),
                                         ([3] * 700, 2)])
def test_masks(sizes, words):
    g = np.random.default_rng(len(sizes))
    trees = [tref.random_tree(g, n, roots=0.05) if n else [] for n in sizes]
    want, want_d = tref.words(trees, words)
    total = sum(sizes)
    out, depths = torch.full((total, words), 7, dtype=torch.int32, device="cuda"), torch.full((total,), 7, dtype=torch.int32, device="cuda")
    status = i32([0])
    tree.masks(dev(flat(trees)), dev(cu_of(sizes)), out, depths, max(sizes), status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert np.array_equal(out.cpu().numpy(), want) and np.array_equal(depths.cpu().numpy(), want_d)
    only = torch.empty_like(out)
    tree.masks(dev(flat(trees)), dev(cu_of(sizes)), only)
    torch.cuda.synchronize()
    assert torch.equal(only, out)


def test_masks_refuses_tensors():
    p, cu = i32([-1, 0, 1]), i32([0, 3])
    for out, depths in ((i32([0, 0, 0]), None), (torch.zeros((3, 0), dtype=torch.int32, device="cuda"), None),
                        (torch.zeros((2, 1), dtype=torch.int32, device="cuda"), None),
                        (torch.zeros((3, 1), dtype=torch.int64, device="cuda"), None),
                        (torch.zeros((3, 1), dtype=torch.int32, device="cuda"), i32([0, 0]))):
        with pytest.raises(ValueError):
            tree.masks(p, cu, out, depths)


def test_masks_of_bad_trees():
    """A parent behind its node counts as none; a request that does not fit stays as it is."""
    out, depths, status = torch.full((9, 1), 7, dtype=torch.int32, device="cuda"), i32([7] * 9), i32([0])
    tree.masks(i32([-1, 0, 2, 1, -1, 0, 9, -1, -1]), i32([0, 4, 7, 9]), out, depths, 4, status)
    torch.cuda.synchronize()
    assert int(status.item()) == binding.MLA_DEVICE_BAD_TREE
    assert out[:, 0].tolist() == [1, 3, 4, 11, 1, 3, 4, 1, 2] and depths.tolist() == [0, 1, 0, 2, 0, 1, 0, 0, 0]
    for cu in ([0, 4, 3, 9], [0, 4, 10, 9], [-1, 3, 3, 3], [0, 4, 4, 9]):
        out.fill_(7)
        status.zero_()
        tree.masks(i32([-1, 0, 0, 1, -1, 0, 0, 1, 0]), i32(cu), out, None, 4, status)
        torch.cuda.synchronize()
        assert int(status.item()) == binding.MLA_DEVICE_PLAN_MISMATCH
        fits = [(a, b) for a, b in zip(cu, cu[1:]) if 0 <= a <= b <= 9 and b - a <= 4]
        touched = {i for a, b in fits for i in range(a, b)}
        assert all((int(out[i, 0]) == 7) == (i not in touched) for i in range(9)), cu


# ------------------------------------------------------------------------------- decode
def decode(batch, masks, options=None, use_tree_plan=True, stream=None):
    d = VerifyDecoder(batch.seq_lens, batch.q_lens, batch.H, "bf16" if batch.kind == "bf16" else "fp8", options=options,
                      tree=use_tree_plan)
    out = torch.full((batch.q.shape[0], batch.H, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((batch.q.shape[0], batch.H), float("nan"), device="cuda")
    status, q, kv, table = i32([0]), batch.q.cuda(), batch.kv.cuda(), dev(batch.table)
    scales, words = None if batch.scales is None else batch.scales.cuda(), None if masks is None else dev(masks)
    torch.cuda.synchronize()
    d.run(q, kv, table, out, lse, kv_scale=batch.kv_scale, status=status, stream=stream, kv_scales=scales, tree_masks=words)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out, lse


def check(batch, masks, out, lse):
    want, bound, want_lse, lse_bound = tref.attend(batch, masks)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    err = np.abs(got - want)
    assert (err <= bound).all(), float((err / np.maximum(bound, 1e-30)).max())
    none = np.isneginf(want_lse)
    assert np.array_equal(none, np.isneginf(got_lse))
    assert (got[none] == 0).all()
    assert (np.abs(got_lse - want_lse)[~none] <= lse_bound[~none]).all()


KINDS = [("bf16", 0), ("e4m3", 0), ("e4m3", 1), ("e4m3", 16), ("e4m3", 64)]
SHAPES = [(12, [1], [1]), (12, [8], [8]), (12, [70], [8]), (1, [65], [65]), (12, [700], [29]), (33, [129, 64, 300], [1, 33, 20]),
          (128, [200, 7], [13, 5]), (16, [513, 96], [64, 96]), (96, [260], [3]), (3, [330], [260])]


@pytest.mark.parametrize("kind,block", KINDS)
@pytest.mark.parametrize("heads,seq,q", SHAPES)
def test_decode_of_trees(heads, seq, q, kind, block):
    g = np.random.default_rng(heads + sum(seq))
    batch = ref.Batch(heads, seq, q, kind, block, seed=heads + block)
    masks, _ = tref.words([tref.random_tree(g, n) for n in q], (max(q) + 31) // 32 + heads % 2)
    check(batch, masks, *decode(batch, masks))


@pytest.mark.parametrize("kind,block", KINDS[:3])
@pytest.mark.parametrize("options", [dict(force_splits=3), dict(unit_pages=1), dict(max_rows_per_cta=16), dict(force_splits=40)])
def test_decode_of_trees_split(kind, block, options):
    """Pieces of the key range in which some rows see nothing, and merges of all kinds."""
    g = np.random.default_rng(7)
    batch = ref.Batch(12, [2700, 90], [40, 70], kind, block, seed=9)
    masks, _ = tref.words([tref.random_tree(g, n) for n in (40, 70)], 3)
    check(batch, masks, *decode(batch, masks, binding.PlanOptions(**options)))


@pytest.mark.parametrize("kind,block", KINDS[:4])
@pytest.mark.parametrize("splits", [0, 2, 18])
def test_rows_that_see_nothing(kind, block, splits):
    """Any bits, no ancestors' rule: rows without keys give zeros and an lse of -inf. The second
    request has keys before its verify tokens, so its rows see those."""
    g = np.random.default_rng(3)
    batch = ref.Batch(12, [1200, 90], [1200, 20], kind, block, seed=4)
    masks = g.integers(-2 ** 31, 2 ** 31, size=(1220, 38), dtype=np.int64).astype(np.int32)
    masks[[0, 1, 63, 64, 700, 1199]] = 0
    masks[5], masks[5, 37] = 0, 1 << 15  # its one key is among the last
    masks[1200:1205] = 0
    options = binding.PlanOptions(force_splits=splits) if splits else None
    out, lse = decode(batch, masks, options)
    pick = np.array([0, 1, 2, 5, 63, 64, 65, 640, 700, 1198, 1199] + list(range(1200, 1220)))
    want = tref_rows(batch, masks, pick)
    for t, (o, l, bound, l_bound) in zip(pick, want):
        got, got_l = out[t].double().cpu().numpy(), lse[t].double().cpu().numpy()
        assert (np.abs(got - o) <= bound).all(), t
        if np.isneginf(l).all():
            assert np.isneginf(got_l).all() and (got == 0).all(), t
        else:
            assert (np.abs(got_l - l) <= l_bound).all(), t


def tref_rows(batch, masks, pick):
    """tref.attend for some verify tokens only."""
    out = []
    cu = cu_of(batch.q_lens)
    for t in pick:
        b = int(np.searchsorted(cu, t, side="right") - 1)
        one = ref.Batch.__new__(ref.Batch)
        one.__dict__ = dict(batch.__dict__)
        at = tref.sees(batch, masks, b, int(t - cu[b]))
        k = batch.codes(b)[at] * batch.key_scales(b)[at, None]
        q = batch.q[t].double().numpy()
        if not len(at):
            out.append((np.zeros((batch.H, 512)), np.full(batch.H, -np.inf), np.zeros((batch.H, 512)), 0.0))
            continue
        s = inputs.SM_SCALE * (q @ k.T)
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        l = p.sum(1, keepdims=True)
        p /= l
        ds = ref.score_error(batch, q, k)
        v = batch.key_scales(b)[at]
        term = p * v
        top = term.max(1, keepdims=True)
        small = 2.0 ** -14 * top * (term < 2.0 ** -4 * top)
        lse = (m + np.log(l))[:, 0]
        bound = ((3 * 2.0 ** -8 + 2 * ds.max(1, keepdims=True)) * (p @ np.abs(k[:, :512]))
                 + small @ np.abs(batch.codes(b)[at, :512]) + 1e-30)
        out.append((p @ k[:, :512], lse, bound, ds.max(1) + 1e-6 * (1 + np.abs(lse))))
    return out


@pytest.mark.parametrize("kind,block", KINDS[:4])
@pytest.mark.parametrize("tree_plan", [False, True])
def test_a_chain_is_the_causal_decode(kind, block, tree_plan):
    batch = ref.Batch(12, [700, 64, 3000], [8, 5, 33], kind, block, seed=21)
    masks, _ = tref.words([list(range(-1, n - 1)) for n in (8, 5, 33)], 2)
    a, b = decode(batch, masks, use_tree_plan=tree_plan), decode(batch, None, use_tree_plan=tree_plan)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bits_behind_the_last_token_are_not_looked_at():
    batch = ref.Batch(12, [700, 300], [8, 5], "bf16", seed=22)
    masks, _ = tref.words([list(range(-1, n - 1)) for n in (8, 5)], 2)
    wild = masks.copy()
    wild[:, 1] = -1
    wild[:8, 0] |= np.int32(-256)
    wild[8:, 0] |= np.int32(-32)
    a, b = decode(batch, masks), decode(batch, wild)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tree_decode_refuses_tensors():
    batch = ref.Batch(12, [300], [5], "bf16", seed=1)
    d = VerifyDecoder([300], [5], 12, "bf16", tree=True)
    out, m = torch.empty((5, 12, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((5, 1), dtype=torch.int32, device="cuda")
    go = lambda masks, **kw: d.run(batch.q.cuda(), batch.kv.cuda(), dev(batch.table), out, tree_masks=masks, **kw)  # noqa: E731
    for bad in (m[:4], m.long(), m.cpu(), m.view(-1), torch.zeros((5, 2), dtype=torch.int32, device="cuda")[:, :1]):
        with pytest.raises(ValueError):
            go(bad)
    with pytest.raises(ValueError):
        go(m, kv_scales=torch.ones((5, 4), device="cuda"))
    with pytest.raises(binding.MlaError):
        VerifyDecoder([300], [40], 12, "bf16", tree=True).run(
            torch.zeros((40, 12, 576), dtype=torch.bfloat16, device="cuda"), batch.kv.cuda(), dev(batch.table),
            torch.empty((40, 12, 512), dtype=torch.bfloat16, device="cuda"), tree_masks=torch.zeros((40, 1), dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------------------- verify
NEAR = 2e-5  # decisions nearer than this, relative, may fall either way: fp32 exponentials, sums and quotients


class Draft:
    """Trees with logits: the target's, the draft's (near it), and tokens drawn or the draft's best."""

    def __init__(self, sizes, vocab, dtype, drawn, seed, width=3, roots=0.0, pad=0):
        g = torch.Generator().manual_seed(seed)
        r = np.random.default_rng(seed)
        self.sizes, self.vocab = list(sizes), vocab
        self.trees = [tref.random_tree(r, n, width, roots) if n else [] for n in sizes]
        total = sum(sizes)
        x = torch.randn((total, vocab + pad), generator=g) * 2
        x[torch.arange(total), torch.randint(0, vocab, (total,), generator=g)] += 8
        self.logits = x.to(dtype)
        self.draft = (x + 0.5 * torch.randn(x.shape, generator=g)).to(dtype)
        self.temp = torch.where(torch.rand(len(sizes), generator=g) < 0.15, 0.0, 0.4 + torch.rand(len(sizes), generator=g))
        cu, self.tokens = cu_of(sizes), torch.zeros(total, dtype=torch.int32)
        for b, t in enumerate(self.trees):
            for i, p in enumerate(t):
                row = self.draft[cu[b] + max(p, 0), :vocab].float()
                if drawn:
                    pr = torch.softmax(row / max(float(self.temp[b]), 0.05), 0)
                    self.tokens[cu[b] + i] = int(torch.multinomial(pr, 1, generator=g))
                else:
                    self.tokens[cu[b] + i] = int(row.topk(min(vocab, width)).indices[t[:i].count(p) % min(vocab, width)])
        self.drawn = drawn
        self.uniforms = torch.rand(total, generator=g)
        self.noise = torch.empty((len(sizes), vocab)).exponential_(generator=g)

    def want(self, width, greedy=False):
        cu = cu_of(self.sizes)
        for b, t in enumerate(self.trees):
            s = slice(cu[b], cu[b + 1])
            if not t:
                yield [], [], 1.0
                continue
            x = self.logits[s, :self.vocab].float().numpy()
            q = self.draft[s, :self.vocab].float().numpy() if self.drawn else None
            yield tref.verify(x, q, self.tokens[s].tolist(), t, 0.0 if greedy else float(self.temp[b]),
                              self.uniforms[s].numpy(), self.noise[b].double().numpy(), width)

    def run(self, width, greedy=False, stream=None, max_nodes=None):
        batch = len(self.sizes)
        path, out = (torch.full((batch, width), 99, dtype=torch.int32, device="cuda") for _ in range(2))
        accepted, status = i32([99] * batch), i32([0])
        view = lambda t: t.cuda()[:, :self.vocab]  # noqa: E731
        kw = {} if greedy else dict(temperature=self.temp.cuda(), uniforms=self.uniforms.cuda(), noise=self.noise.cuda())
        args = (view(self.logits), self.tokens.cuda(), dev(flat(self.trees)), dev(cu_of(self.sizes)), path, out, accepted)
        kw["draft_logits"] = view(self.draft) if self.drawn else None
        torch.cuda.synchronize()
        tree.verify(*args, max_nodes=max_nodes or max(self.sizes), status=status, stream=stream, **kw)
        torch.cuda.synchronize()
        return path.cpu().numpy(), out.cpu().numpy(), accepted.cpu().numpy(), int(status.item())

    def check(self, width, greedy=False):
        path, out, accepted, status = self.run(width, greedy)
        assert status == 0
        near = 0
        for b, (p, o, margin) in enumerate(self.want(width, greedy)):
            if margin < NEAR:
                near += 1
                continue
            assert accepted[b] == len(p), b
            assert path[b].tolist() == p + [-1] * (width - len(p)), b
            assert out[b].tolist() == o + [-1] * (width - len(o)), b
        assert near <= max(1, len(self.sizes) // 20)


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes,vocab,pad", [([1], 1, 0), ([5], 2, 0), ([4, 1, 0, 9], 7, 1), ([12] * 20, 1000, 0), ([30, 64], 4099, 0),
                                             ([6] * 160, 333, 3), ([5], 131072, 0), ([8, 8], 50001, 7), ([3] * 330, 64, 0)])
def test_verify(sizes, vocab, pad, dtype, drawn):
    Draft(sizes, vocab, dtype, drawn, seed=vocab + len(sizes), pad=pad).check(width=max(sizes))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes,vocab", [([1], 1), ([40], 5), ([20] * 12, 257), ([64, 3], 65536)])
def test_verify_greedy(sizes, vocab, dtype):
    """bf16 logits tie often: the lowest index is the token."""
    d = Draft(sizes, vocab, dtype, False, seed=vocab)
    d.check(max(sizes), greedy=True)
    d.temp.zero_()
    d.check(max(sizes))


def test_verify_greedy_looks_at_no_draft_distribution():
    d = Draft([20] * 12, 257, torch.bfloat16, True, seed=15)
    got = d.run(20, greedy=True)
    d.draft.fill_(float("nan"))
    assert all(np.array_equal(a, b) for a, b in zip(got[:3], d.run(20, greedy=True)[:3]))
    d.check(20, greedy=True)


def test_verify_of_nothing():
    """Requests without nodes, and a batch of them alone; a draft that is the target's own distribution is accepted."""
    d = Draft([0, 3, 0], 30, torch.float32, False, seed=16)
    d.check(4)
    d = Draft([0, 0], 30, torch.float32, False, seed=16)
    path, out, accepted, status = d.run(4, max_nodes=1)
    assert status == 0 and (path == -1).all() and (out == -1).all() and (accepted == 0).all()
    d = Draft([6] * 40, 100, torch.float32, True, seed=17, width=1)
    d.draft = d.logits.clone()
    d.temp.fill_(0.8)
    assert (d.run(6)[2] == 6).all()


def test_verify_long_chains_and_padding():
    d = Draft([1024, 900], 50, torch.float32, False, seed=3, width=1)
    d.temp[0], d.temp[1] = 2.0, 0.5
    d.uniforms[:1024] = 0.0  # a token is accepted wherever it has any probability
    d.check(width=1024)
    assert d.run(1024)[2][0] == 1024
    Draft([40] * 6, 300, torch.bfloat16, True, seed=4, roots=0.3).check(width=40)


def test_a_full_path_ends_the_walk():
    d = Draft([30] * 8, 40, torch.float32, False, seed=5)
    d.temp.fill_(0.3)
    for width in (1, 2, 3):
        d.check(width)


def test_many_siblings():
    """64 children of one node, drawn with replacement (repeats among them), and certain ones with repeats."""
    for drawn in (True, False):
        d = Draft([65] * 12, 20, torch.float32, drawn, seed=6, width=64)
        d.trees = [[-1] + [0] * 64 for _ in d.sizes]
        d.uniforms = d.uniforms.clamp(min=0.9)
        d.check(width=3)


def test_verify_special_values():
    """Masked vocabulary (-inf), NaN, infinite logits, rows with nothing finite, the type's lowest
    value, tokens outside the vocabulary, noise of zero, a draft of nothing."""
    for dtype in (torch.bfloat16, torch.float32):
        for drawn in (False, True):
            d = Draft([6] * 12, 40, dtype, drawn, seed=8)
            d.temp[:2] = 0.0
            d.logits[:, 5:30:2] = float("-inf")
            d.draft[:, 6:30:2] = float("-inf")
            d.logits[3::7, 2] = float("nan")
            d.logits[5::11, 3] = float("inf")
            d.logits[9::13, 4] = torch.finfo(dtype).min
            d.logits[12] = float("-inf")       # request 2's root
            d.logits[18] = float("nan")        # request 3's
            d.draft[24] = float("-inf")        # request 4's
            d.logits[30] = torch.finfo(dtype).min
            d.logits[36, 7], d.logits[36, 9] = float("inf"), float("inf")
            d.tokens[25], d.tokens[26], d.tokens[32] = -1, 40, 2 ** 31 - 1
            d.noise[5, ::3], d.noise[6, ::5], d.noise[7, 1] = 0.0, float("nan"), float("inf")
            d.check(width=6)


def test_temperatures():
    d = Draft([5] * 9, 100, torch.float32, True, seed=9)
    d.temp[:] = torch.tensor([float("nan"), -1.0, 1e-7, 2e-6, 0.01, 1.0, 50.0, 1e9, float("inf")])
    want = torch.tensor([0.0, 0.0, 0.0, 2e-6, 0.01, 1.0, 50.0, 2.0 ** 20, 2.0 ** 20])
    path, out, accepted, status = d.run(5)
    d.temp = want
    for b, (p, o, margin) in enumerate(d.want(5)):
        if margin >= NEAR:
            assert path[b, :len(p)].tolist() == p and out[b, :len(o)].tolist() == o, b


def test_verify_bad_trees():
    d = Draft([4, 4, 4], 30, torch.float32, False, seed=10)
    d.trees[1][2] = 2  # its own parent
    path, out, accepted, status = d.run(4)
    assert status == binding.MLA_DEVICE_BAD_TREE
    d.trees[1][2] = -1
    for b, (p, o, _) in enumerate(d.want(4)):
        assert accepted[b] == len(p) and path[b, :len(p)].tolist() == p and out[b, :len(o)].tolist() == o
    path, out, accepted, status = d.run(4, max_nodes=3)
    assert status == binding.MLA_DEVICE_PLAN_MISMATCH | 0 and (accepted == 0).all() and (path == -1).all() and (out == -1).all()


def test_the_result_is_distributed_as_the_target():
    """65536 requests with the same logits, drafts drawn from the draft's distribution (two children of
    the root, one below each): the first token, and the second where the first is given, have the target's
    distribution. A frequency over n is off by at most 5 sqrt(0.25 / n)."""
    n, vocab = 65536, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x, y = (torch.randn((vocab + 1, vocab), generator=g, device="cuda") * 1.3 for _ in range(2))  # by the last token
    q = torch.softmax(y, 1)
    first = torch.multinomial(q[vocab], 2 * n, True, generator=g).view(n, 2)
    below = torch.multinomial(q[first.view(-1)], 1, generator=g).view(n, 2)
    last = torch.cat([torch.full((n, 1), vocab, device="cuda"), first, below], 1).view(-1)  # a node's own token
    tokens = torch.cat([torch.zeros((n, 1), device="cuda", dtype=torch.long), first, below], 1).view(-1).int()
    path, out = (torch.zeros((n, 3), dtype=torch.int32, device="cuda") for _ in range(2))
    accepted = torch.zeros(n, dtype=torch.int32, device="cuda")
    tree.verify(x[last], tokens, i32([-1, 0, 0, 1, 2]).repeat(n), torch.arange(n + 1, dtype=torch.int32, device="cuda") * 5, path,
                out, accepted, uniforms=torch.rand(5 * n, generator=g, device="cuda"),
                noise=torch.empty((n, vocab), device="cuda").exponential_(generator=g), draft_logits=y[last])
    torch.cuda.synchronize()
    p = torch.softmax(x.double(), 1)
    a = out[:, 0].long()
    assert (torch.bincount(a, minlength=vocab) / n - p[vocab]).abs().max() < 5 * (0.25 / n) ** 0.5
    for t in range(vocab):
        rows = (a == t) & (accepted > 1)
        k = int(rows.sum())
        assert (torch.bincount(out[rows, 1].long(), minlength=vocab) / k - p[t]).abs().max() < 5 * (0.25 / k) ** 0.5


def test_verify_rows_far_apart():
    """Rows whose offsets pass 2^31 elements, unaligned rows, rows of other strides."""
    rows, stride = 5, (1 << 29) + 3
    big = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda").as_strided((rows, 1000), (stride, 1))
    d = Draft([5], 1000, torch.bfloat16, False, seed=12, width=1)
    big.copy_(d.logits)
    path, out, accepted = torch.zeros((1, 5), dtype=torch.int32, device="cuda"), torch.zeros((1, 5), dtype=torch.int32, device="cuda"), i32([0])
    d.temp[:] = 0.7
    tree.verify(big, d.tokens.cuda(), dev(flat(d.trees)), i32([0, 5]), path, out, accepted, d.temp.cuda(), d.uniforms.cuda(),
                d.noise.cuda())
    torch.cuda.synchronize()
    (p, o, margin), = d.want(5)
    assert margin >= NEAR and path[0, :len(p)].tolist() == p and out[0, :len(o)].tolist() == o


def test_verify_refuses_tensors():
    d = Draft([4], 30, torch.float32, True, seed=11)
    x, cu = d.logits.cuda(), i32([0, 4])
    good = dict(logits=x, tokens=d.tokens.cuda(), parents=dev(flat(d.trees)), cu_nodes=cu, path=i32([[0] * 4]), out_tokens=i32([[0] * 4]),
                accepted=i32([0]), uniforms=d.uniforms.cuda(), noise=d.noise.cuda(), draft_logits=d.draft.cuda())
    tree.verify(**good)
    wide_x = torch.zeros((4, 60), device="cuda")
    for name, bad in (("logits", x.double()), ("logits", wide_x[:, ::2]), ("logits", x[:1].expand(4, 30)), ("logits", x[0]),
                      ("draft_logits", x.bfloat16()), ("draft_logits", x[:3]), ("tokens", d.tokens.cuda().long()), ("cu_nodes", cu[:1]),
                      ("path", i32([0] * 4)), ("out_tokens", i32([[0] * 3])), ("accepted", i32([0, 0])), ("noise", d.noise.cuda()[:, :29]),
                      ("uniforms", d.uniforms), ("temperature", torch.ones(2, device="cuda"))):
        with pytest.raises((ValueError, binding.MlaError)):
            tree.verify(**{**good, name: bad})
    for left_out in ("uniforms", "noise"):
        with pytest.raises(binding.MlaError):
            tree.verify(**{**good, left_out: None})
    with pytest.raises(binding.MlaError):  # written over what other requests still read
        tree.verify(**{**good, "accepted": good["tokens"][:1]})


# ------------------------------------------------------------------------------- commit
def commit_case(lens, nodes, layers, kind, block, seed=0):
    g, r = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    batch = ref.Batch(1, np.maximum(lens, 1), np.ones(len(lens)), "bf16", seed=seed, extra_pages=2, poison=False)
    x = torch.randn((layers, batch.pages, PAGE, D), generator=g)
    if kind == "bf16":
        kv, scales = x.to(torch.bfloat16), None
    else:
        kv = (x * 60).clamp(-448, 448).to(F8).view(torch.uint8)
        scales = torch.exp2(torch.randint(-9, -3, (layers, batch.pages, PAGE // block), generator=g).float()) if block else None
    paths = []
    for q in nodes:
        k = int(r.integers(1, q + 1)) if q else 0
        paths.append([0] + sorted((r.permutation(q - 1)[:k - 1] + 1).tolist()) if q else [])
    return batch, kv, scales, paths


def run_commit(batch, kv, scales, lens, nodes, paths, width=None, stream=None):
    width = width or max([1] + [len(p) for p in paths])
    path = np.full((len(lens), width), -1, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    kv, scales = kv.clone().cuda(), None if scales is None else scales.clone().cuda()
    new_lens, status = torch.full((len(lens),), 99, dtype=torch.int32, device="cuda"), i32([0])
    args = (dev(batch.table), i32(lens), dev(cu_of(nodes)), dev(path), i32([len(p) for p in paths]))
    torch.cuda.synchronize()
    cache.commit(kv, *args, new_lens, scales, status, stream)
    torch.cuda.synchronize()
    return kv, scales, new_lens.tolist(), int(status.item())


def check_commit(batch, kv, scales, lens, nodes, paths, block, **kw):
    got, got_s, new_lens, status = run_commit(batch, kv, scales, lens, nodes, paths, **kw)
    assert status == 0 and new_lens == [n - q + len(p) for n, q, p in zip(lens, nodes, paths)]
    for l in range(kv.shape[0]):
        values = kv[l].double().numpy() if kv.dtype == torch.bfloat16 else ref.code_values(kv[l])
        s = None if scales is None else scales[l].double().numpy()
        for b, (n, q, p) in enumerate(zip(lens, nodes, paths)):
            tref.commit(values, s, batch.table[b], n, q, p, block)
        now = got[l].cpu().double() if kv.dtype == torch.bfloat16 else got[l].cpu().view(F8).double()
        assert np.array_equal(now.numpy(), values, equal_nan=True)
        if s is not None:
            assert np.array_equal(got_s[l].cpu().double().numpy(), s)


@pytest.mark.parametrize("kind,block", [("bf16", 0), ("e4m3", 0)] + [("e4m3", 2 ** k) for k in range(7)])
@pytest.mark.parametrize("lens,nodes,layers", [([1], [1], 1), ([8], [8], 2), ([70, 64, 130, 9], [8, 1, 66, 0], 3),
                                               ([200] * 9, [30] * 9, 5), ([400, 3], [300, 3], 2), ([65, 129], [64, 128], 40)])
def test_commit(lens, nodes, layers, kind, block):
    batch, kv, scales, paths = commit_case(lens, nodes, layers, kind, block, seed=len(lens) + block)
    check_commit(batch, kv, scales, lens, nodes, paths, block)


@pytest.mark.parametrize("block", [1, 16, 64])
def test_commit_where_scales_grow_or_vanish(block):
    """A large draft row enters a block of small older ones; blocks of zeros with the scale 0."""
    batch, kv, scales, _ = commit_case([100, 90, 80], [20, 20, 20], 2, "e4m3", block, seed=5)
    scales[:] = 2.0 ** -8
    last = batch.table[0, 1]
    scales[:, last, 30 // block:] = 2.0 ** 3        # position 94 on
    zero = batch.table[1, 1]
    scales[1, zero], kv[1, zero] = 0.0, 0
    scales[0, batch.table[2, 1]] = torch.tensor(0.37)  # no power of two
    check_commit(batch, kv, scales, [100, 90, 80], [20, 20, 20], [[0, 1, 15, 18], [0, 5, 7], [0, 2, 19]], block)


def test_commit_many_rows_and_layers():
    """More (layer, row) pairs than a CTA holds at a time."""
    lens, nodes = [700, 650], [600, 640]
    batch, kv, scales, _ = commit_case(lens, nodes, 4, "e4m3", 8, seed=6)
    paths = [list(range(0, 600, 2)), [0] + list(range(39, 640))]
    check_commit(batch, kv, scales, lens, nodes, paths, 8)
    batch, kv, _, _ = commit_case(lens, nodes, 4, "bf16", 0, seed=6)
    check_commit(batch, kv, None, lens, nodes, paths, 0)


def test_commit_of_lengths_that_pass_32_bits():
    """A negative length minus the nodes passes the lowest int32 and comes out positive."""
    batch, kv, _, _ = commit_case([100], [20], 1, "bf16", 0, seed=8)
    k, new_lens, status = kv.cuda().clone(), i32([7]), i32([0])
    cache.commit(k, dev(batch.table), i32([-5]), i32([0, 2 ** 31 - 1]), i32([[0, 3, 7]]), i32([3]), new_lens, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == binding.MLA_DEVICE_PLAN_MISMATCH and int(new_lens.item()) == -5
    assert torch.equal(k, kv.cuda())


def test_commit_bad_requests_stay():
    lens, nodes = [100, 90, 80], [20, 20, 20]
    good = [0, 3, 7]
    batch, kv, scales, _ = commit_case(lens, nodes, 2, "e4m3", 16, seed=7)
    for bad, bit in (([0, 3, 3], 8), ([0, 5, 4], 8), ([0, 20], 8), ([-1, 2], 8), ([2, 1], 8)):
        got, got_s, new_lens, status = run_commit(batch, kv, scales, lens, nodes, [good, bad, good])
        assert status == bit and new_lens == [83, 90, 63], bad
        only = run_commit(batch, kv, scales, lens, nodes, [good, [0], good])
        assert torch.equal(got, only[0]) and torch.equal(got_s, only[1])
    # more accepted than nodes; more nodes than tokens; pages that the table has no room for
    for l, n, paths in (([100, 90, 80], [20, 2, 20], [good, good, good]), ([100, 19, 80], [20, 20, 20], [good] * 3),
                        ([100, 64 * batch.table.shape[1] + 1, 80], [20, 20, 20], [good] * 3)):
        got, got_s, new_lens, status = run_commit(batch, kv, scales, l, n, paths)
        assert status == binding.MLA_DEVICE_PLAN_MISMATCH and new_lens == [83, l[1], 63]
    table = batch.table.copy()
    table[1, 1] = batch.pages
    b2 = type("B", (), {"table": table})
    got, _, new_lens, status = run_commit(b2, kv, scales, lens, nodes, [good] * 3)
    assert status == binding.MLA_DEVICE_BAD_PAGE and new_lens == [83, 73, 63]
    only = run_commit(batch, kv, scales, lens, nodes, [good, [0], good])
    assert torch.equal(got, only[0])


def test_commit_rows_beyond_32_bits():
    """The last layer's rows lie behind 2^32 bytes (and behind 2^31 16-byte pieces' indices of bytes)."""
    layers, pages = 70, 1024
    kv = torch.zeros((layers, pages, PAGE, D), dtype=torch.bfloat16, device="cuda")
    kv[:, 1000] = torch.arange(PAGE, device="cuda")[:, None].to(torch.bfloat16)
    kv[-1, 1000] += 64
    new_lens = i32([0])
    cache.commit(kv, i32([[1000]]), i32([40]), i32([0, 10]), i32([[0, 4, 9]]), i32([3]), new_lens)
    torch.cuda.synchronize()
    want = list(range(64))
    want[31], want[32] = 34, 39
    assert new_lens.item() == 33
    for l, add in ((0, 0), (33, 0), (layers - 1, 64)):
        assert kv[l, 1000, :, 5].tolist() == [w + add for w in want]


def test_one_layer_and_other_forms_of_a_call():
    lens, nodes = [70, 64], [8, 5]
    batch, kv, scales, paths = commit_case(lens, nodes, 1, "e4m3", 16, seed=8)
    got, got_s, new_lens, _ = run_commit(batch, kv, scales, lens, nodes, paths)
    flat_kv, flat_s, flat_lens, _ = run_commit(batch, kv[0], scales[0], lens, nodes, paths)
    assert torch.equal(got[0], flat_kv) and torch.equal(got_s[0], flat_s) and new_lens == flat_lens
    typed, _, _, _ = run_commit(batch, kv.view(F8), scales, lens, nodes, paths)
    assert torch.equal(typed.view(torch.uint8), got)
    for kw in (dict(kv=kv.cuda()[:, :, :, :288]), dict(scales=scales.cuda()[0]), dict(scales=torch.ones((1, batch.pages, 3), device="cuda")),
               dict(kv=kv.cuda().view(-1)), dict(scales=scales.double().cuda())):
        a = dict(kv=kv.cuda(), scales=scales.cuda(), **{}) | kw
        with pytest.raises(ValueError):
            cache.commit(a["kv"], dev(batch.table), i32(lens), dev(cu_of(nodes)), i32([[0], [0]]), i32([1, 1]), i32([0, 0]), a["scales"])


# ------------------------------------------------------------------------------- together
class Step:
    """One serving step over a block-scaled cache of some layers: masks, append and decode in each
    layer, verification, commit. Everything stays on the GPU, so the step can be captured."""

    def __init__(self, seed, layers=2, heads=12, block=16, vocab=500):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = np.random.default_rng(seed)
        self.layers, self.heads, self.block = layers, heads, block
        self.prefix, self.nodes = np.array([100, 63, 1]), np.array([13, 5, 1])
        self.lens = self.prefix + self.nodes
        self.trees = [tref.random_tree(r, int(n)) for n in self.nodes]
        self.total = int(self.nodes.sum())
        per = [3, 3, 2]
        perm = r.permutation(sum(per) + 1).astype(np.int32)
        self.host_table = np.zeros((3, 3), np.int32)
        for b, k in enumerate(per):
            self.host_table[b, :k] = perm[sum(per[:b]):sum(per[:b]) + k]
        self.table = dev(self.host_table)
        self.kv = torch.zeros((layers, sum(per) + 1, PAGE, D), dtype=torch.uint8, device="cuda")
        self.scales = torch.ones((layers, sum(per) + 1, PAGE // block), device="cuda")
        prompt = torch.randn((layers, int(self.prefix.sum()), D), generator=g, device="cuda").to(torch.bfloat16)
        for l in range(layers):
            cache.append(prompt[l], self.kv[l], self.scales[l], self.table, i32(self.prefix.tolist()),
                         dev(cu_of(self.prefix)), int(self.prefix.max()))
        self.rows = torch.randn((layers, self.total, D), generator=g, device="cuda").to(torch.bfloat16)
        self.q = torch.randn((layers, self.total, heads, D), generator=g, device="cuda").to(torch.bfloat16)
        self.parents, self.cu = dev(flat(self.trees)), dev(cu_of(self.nodes))
        self.tokens = torch.randint(0, 3, (self.total,), generator=g, device="cuda").int()
        self.temp = torch.full((3,), 2.0, device="cuda")
        self.uniforms = torch.rand(self.total, generator=g, device="cuda")
        self.noise = torch.empty((3, vocab), device="cuda").exponential_(generator=g)
        self.masks, self.depths = torch.zeros((self.total, 1), dtype=torch.int32, device="cuda"), i32([0] * self.total)
        self.decoder = VerifyDecoder(self.lens, self.nodes, heads, "fp8", tree=True)
        self.out = torch.zeros((layers, self.total, heads, 512), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.zeros((layers, self.total, heads), device="cuda")
        self.logits = torch.zeros((self.total, vocab), device="cuda")
        self.path, self.tok = torch.zeros((3, 8), dtype=torch.int32, device="cuda"), torch.zeros((3, 8), dtype=torch.int32, device="cuda")
        self.accepted, self.new_lens, self.status = i32([0] * 3), i32([0] * 3), i32([0])
        self.len_dev = i32(self.lens.tolist())

    def run(self, keep=False):
        tree.masks(self.parents, self.cu, self.masks, self.depths, 13, self.status)
        for l in range(self.layers):
            cache.append(self.rows[l], self.kv[l], self.scales[l], self.table, self.len_dev, self.cu, 13, self.status)
            self.decoder.run(self.q[l], self.kv[l], self.table, self.out[l], self.lse[l], kv_scales=self.scales[l],
                             tree_masks=self.masks, status=self.status)
        # (elementwise: graphs that are replayed at once must not hold a library's product, whose workspace they share)
        self.logits.copy_(self.out[-1].view(self.total, -1)[:, :self.logits.shape[1]]).mul_(30.0)
        self.logits[:, :3] += 20.0  # (three tokens that the drafts are made of)
        tree.verify(self.logits, self.tokens, self.parents, self.cu, self.path, self.tok, self.accepted, self.temp,
                    self.uniforms, self.noise, max_nodes=13, status=self.status)
        if keep:
            self.before = self.kv.clone(), self.scales.clone()
        cache.commit(self.kv, self.table, self.len_dev, self.cu, self.path, self.accepted, self.new_lens, self.scales, self.status)

    def results(self):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        return [t.clone() for t in (self.kv, self.scales, self.out, self.lse, self.path, self.tok, self.accepted, self.new_lens)]


    def batch(self, l, kv, scales, lens, q_lens, q):
        """Layer l as the plain forms take it."""
        b = ref.Batch.__new__(ref.Batch)
        b.H, b.kind, b.block, b.table, b.kv_scale = self.heads, "e4m3", self.block, self.host_table, 1.0
        b.seq_lens, b.q_lens = np.asarray(lens, np.int32), np.asarray(q_lens, np.int32)
        b.kv, b.scales, b.q = kv[l].cpu(), scales[l].cpu(), q.cpu()
        return b


def test_a_serving_step():
    """Each operator's result follows from the one before; after the step the cache is a chain, over
    which a causal decode and the key weights of the accepted path's queries run."""
    s = Step(1)
    s.run(keep=True)
    kv, scales, out, lse, path, tok, accepted, new_lens = s.results()
    words, depths = tref.words(s.trees, 1)
    assert np.array_equal(s.masks.cpu().numpy(), words) and np.array_equal(s.depths.cpu().numpy(), depths)
    acc = accepted.tolist()
    paths = [path[b, :acc[b]].tolist() for b in range(3)]
    assert max(acc) > 1 and new_lens.tolist() == [p + a for p, a in zip(s.prefix.tolist(), acc)]
    for b, p in enumerate(paths):  # the path climbs the tree, and tokens are its nodes' own
        assert p == tref.lines(s.trees[b])[p[-1]]
        at = int(s.nodes[:b].sum())
        assert tok[b, :acc[b] - 1].tolist() == s.tokens[at:at + 13][p[1:]].tolist()
    chosen = [int(s.nodes[:b].sum()) + i for b in range(3) for i in paths[b]]
    d = VerifyDecoder(new_lens.cpu().numpy(), acc, s.heads, "fp8")
    for l in range(s.layers):
        check(s.batch(l, *s.before, s.lens, s.nodes, s.q[l]), words, out[l], lse[l])
        values, want_s = ref.code_values(s.before[0][l].cpu()), s.before[1][l].cpu().double().numpy()
        for b, p in enumerate(paths):
            tref.commit(values, want_s, s.host_table[b], int(s.lens[b]), int(s.nodes[b]), p, s.block)
        same = np.array_equal(ref.code_values(kv[l].cpu()), values) and np.array_equal(scales[l].cpu().double().numpy(), want_s)
        assert same
        q = s.q[l][chosen].contiguous()
        o, e = torch.empty((sum(acc), s.heads, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((sum(acc), s.heads), device="cuda")
        d.run(q, kv[l], s.table, o, e, kv_scales=scales[l])
        w = torch.zeros((3, 192), device="cuda")
        d.key_weights(q, kv[l], s.table, e, w, kv_scales=scales[l])
        torch.cuda.synchronize()
        chain, _ = tref.words([list(range(-1, a - 1)) for a in acc], 1)
        check(s.batch(l, kv, scales, new_lens.tolist(), acc, q), chain, o, e)
        assert torch.allclose(w.sum(1), torch.tensor(acc, device="cuda").float() * s.heads, rtol=1e-4)


def test_a_serving_step_over_bf16_keeps_every_bit():
    """With a bf16 cache the moved rows are the same, so the chain's decode differs from the tree's by the
    order of sums alone: two bf16 outputs within a rounding each (2^-8) and the partials' (2^-8 each)."""
    g = torch.Generator(device="cuda").manual_seed(2)
    r = np.random.default_rng(2)
    parents = tref.random_tree(r, 21)
    path = tref.lines(parents)[-1]
    kv = torch.randn((3, PAGE, D), generator=g, device="cuda").to(torch.bfloat16)
    table, q = i32([[2, 0, 1]]), torch.randn((21, 12, D), generator=g, device="cuda").to(torch.bfloat16)
    masks = dev(tref.words([parents], 1)[0])
    out, lse = torch.empty((21, 12, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((21, 12), device="cuda")
    VerifyDecoder([150], [21], 12, "bf16", tree=True).run(q, kv, table, out, lse, tree_masks=masks)
    new_lens = i32([0])
    cache.commit(kv, table, i32([150]), i32([0, 21]), i32([path]), i32([len(path)]), new_lens)
    torch.cuda.synchronize()
    n = int(new_lens.item())
    assert n == 129 + len(path) and len(path) > 1
    o, e = torch.empty((len(path), 12, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((len(path), 12), device="cuda")
    VerifyDecoder([n], [len(path)], 12, "bf16").run(q[path].contiguous(), kv, table, o, e)
    torch.cuda.synchronize()
    assert torch.allclose(e, lse[path], rtol=0, atol=1e-5)
    scale = kv.float().abs().max()
    assert (o.float() - out[path].float()).abs().max() <= 4 * 2.0 ** -8 * scale


def test_a_captured_step_and_streams():
    """The step from a graph, replayed on refilled buffers, and on another stream: the same results."""
    want = Step(3)
    want.run()
    want = want.results()
    s = Step(3)
    kv, scales = s.kv.clone(), s.scales.clone()
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for _ in range(2):
        s.kv.copy_(kv)
        s.scales.copy_(scales)
        for t in (s.out, s.lse, s.path, s.tok, s.accepted, s.new_lens, s.masks):
            t.fill_(5)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(s.results(), want))
    other = Step(3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        other.run()
    assert all(torch.equal(a, b) for a, b in zip(other.results(), want))


def test_two_graphs_at_once():
    steps = [Step(4), Step(5)]
    want, graphs = [], []
    for s in steps:
        first = (s.kv.clone(), s.scales.clone())
        s.run()
        want.append(s.results())
        s.kv.copy_(first[0])
        s.scales.copy_(first[1])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.run()
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for graph, stream in zip(graphs, streams):
        with torch.cuda.stream(stream):
            graph.replay()
    for s, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(s.results(), w))


def test_explicit_streams():
    """The stream argument of each operator, with another one current."""
    side = torch.cuda.Stream()
    d = Draft([6] * 4, 100, torch.float32, True, seed=13)
    a, b = d.run(6), d.run(6, stream=side)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))
    batch, kv, scales, paths = commit_case([70, 64], [8, 5], 2, "e4m3", 16, seed=8)
    a, b = (run_commit(batch, kv, scales, [70, 64], [8, 5], paths, stream=st) for st in (None, side))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[2:] == b[2:]
    batch = ref.Batch(12, [700], [9], "bf16", seed=30)
    masks, _ = tref.words([tref.random_tree(np.random.default_rng(1), 9)], 1)
    assert all(torch.equal(x, y) for x, y in zip(decode(batch, masks), decode(batch, masks, stream=side)))
    out, parents, cu = torch.zeros((9, 1), dtype=torch.int32, device="cuda"), i32([-1, 0, 0, 1, 2, 2, 3, 4, 5]), i32([0, 9])
    torch.cuda.synchronize()
    tree.masks(parents, cu, out, stream=side)
    torch.cuda.synchronize()
    assert out[:, 0].tolist() == [1, 3, 5, 11, 21, 37, 75, 149, 293]
