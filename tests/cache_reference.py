"""Plain 64-bit forms of the cache operators for their tests: numpy and torch on the CPU, a
request and a block at a time, written from the definitions in include/mla_decode.h."""
import math

import numpy as np
import torch

from mla_speculative_verify_gb300 import inputs

D, DV, PAGE = 576, 512, 64
F8 = torch.float8_e4m3fn


def code_values(codes: torch.Tensor) -> np.ndarray:
    """e4m3 codes (uint8) as their values."""
    return codes.view(F8).to(torch.float64).numpy()


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """Values on the e4m3 grid next to x: ties to even, beyond 448 cut, NaN kept."""
    x = np.clip(np.asarray(x, np.float64), -448.0, 448.0)
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(x / step) * step


def block_scale(amax: float) -> float:
    e = -60
    while e < 60 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(rows, values, scales, table, seq_lens, cu, block):
    """values [pages, 64, 576] float64 on the e4m3 grid and scales, both changed in place."""
    rows = rows.to(torch.float64).numpy()
    for b, end in enumerate(seq_lens):
        n = cu[b + 1] - cu[b]
        for k in range((end - n) // block, -(-end // block) if n else 0):
            at = k * block
            page, slot = table[b, at // PAGE], at % PAGE
            new = [p for p in range(at, at + block) if end - n <= p < end]
            x = rows[[cu[b] + p - (end - n) for p in new]]
            amax = np.abs(x[np.isfinite(x)]).max(initial=0.0)
            old = scales[page, slot // block]
            s = block_scale(amax)
            if new[0] > at:  # older rows before the new ones
                s = max(s, old)
                sl = slice(slot, slot + new[0] - at)
                values[page, sl] = to_e4m3(np.float32(values[page, sl]) * np.float32(old / s))
            for p, r in zip(new, x):
                values[page, p % PAGE] = to_e4m3(np.float32(r / s))
            scales[page, slot // block] = s


def keep(weights, n, budget, first, last):
    """Indices that an eviction keeps, in order."""
    if n <= budget:
        return np.arange(n)
    mid = np.arange(first, n - last)
    w = weights[mid].astype(np.float64) + 0.0
    w[np.isnan(w)] = -np.inf
    low = np.isnan(weights[mid])  # NaN below everything, -inf too
    best = mid[np.lexsort((mid, -w, low))][:budget - first - last]
    return np.sort(np.concatenate([np.arange(first), best, np.arange(n - last, n)])).astype(np.int64)


def evict(weights, lens, budget, first, last, values, scales, table, values_dst, scales_dst, table_dst, block):
    """Moves rows in the float64 arrays values_dst (and scales_dst); returns the kept indices."""
    kept = []
    for b, n in enumerate(lens):
        k = keep(weights[b], n, budget, first, last)
        kept.append(k)
        src = [(table[b, j // PAGE], j % PAGE) for j in k]
        if scales is None:
            for r, (p, s) in enumerate(src):
                values_dst[table_dst[b, r // PAGE], r % PAGE] = values[p, s]
            continue
        for r0 in range(0, len(k), block):
            members = src[r0:r0 + block]
            old = [scales[p, s // block] for p, s in members]
            new = max(old)
            scales_dst[table_dst[b, r0 // PAGE], r0 % PAGE // block] = new
            for i, (p, s) in enumerate(members):
                r = r0 + i
                v = values[p, s] if old[i] == new else to_e4m3(np.float32(values[p, s]) * (np.float32(old[i]) / np.float32(new)))
                values_dst[table_dst[b, r // PAGE], r % PAGE] = v
    return kept


class Batch:
    """A seeded paged batch in host memory: bf16 cache, e4m3 cache with one scale, or (block > 0)
    with a scale for each block, whose scales spread over 2^-spread .. 2^spread."""

    def __init__(self, heads, seq_lens, q_lens, kind, block=0, spread=3.0, seed=0, extra_pages=0, poison=True):
        self.H, self.kind, self.block = heads, kind, block
        self.seq_lens, self.q_lens = np.asarray(seq_lens, np.int32), np.asarray(q_lens, np.int32)
        g = torch.Generator().manual_seed(seed)
        per = (self.seq_lens + PAGE - 1) // PAGE
        self.pages = int(per.sum()) + extra_pages
        perm = torch.randperm(self.pages, generator=g).numpy().astype(np.int32)
        self.table = np.zeros((len(per), max(1, int(per.max(initial=1)))), np.int32)
        at = 0
        for b, k in enumerate(per):
            self.table[b, :k] = perm[at:at + k]
            at += int(k)
        self.free = perm[at:]
        x = torch.randn((self.pages, PAGE, D), generator=g)
        self.scales, self.kv_scale = None, 1.0
        if kind == "bf16":
            self.kv = x.to(torch.bfloat16)
        elif block == 0:
            self.kv_scale = float(x.abs().max()) / 448.0
            self.kv = (x / self.kv_scale).clamp(-448, 448).to(F8).view(torch.uint8)
        else:
            per_page = PAGE // block
            s = torch.exp2(spread * (2.0 * torch.rand((self.pages, per_page), generator=g) - 1.0)) / 100.0
            mult = torch.exp2(torch.rand((self.pages, per_page), generator=g) * 2.0)
            self.scales = s.contiguous()
            y = x.view(self.pages, per_page, -1) * (100.0 / mult[:, :, None])
            self.kv = y.clamp(-448, 448).to(F8).view(torch.uint8).view(self.pages, PAGE, D)
        self.q = torch.randn((int(self.q_lens.sum()), heads, D), generator=g).to(torch.bfloat16)
        if poison:  # what lies behind a request's last key may be anything
            for b, n in enumerate(self.seq_lens):
                if n % PAGE:
                    page, s = self.table[b, n // PAGE], n % PAGE
                    self.kv[page, s:] = float("nan") if kind == "bf16" else 0x7F
                    if self.scales is not None:
                        self.scales[page, -(-s // block):] = float("nan")

    def key_scales(self, b):
        n = int(self.seq_lens[b])
        j = np.arange(n)
        page = self.table[b, j // PAGE]
        if self.scales is None:
            return np.full(n, self.kv_scale)
        return self.scales.double().numpy()[page, j % PAGE // self.block]

    def codes(self, b):
        n = int(self.seq_lens[b])
        j = np.arange(n)
        kv = self.kv[torch.from_numpy(self.table[b, j // PAGE].astype(np.int64)), torch.from_numpy(j % PAGE)]
        return kv.double().numpy() if self.kind == "bf16" else code_values(kv)

    def rows(self, b):
        """For each verify token of request b: (global token, its q [H, 576], keys it sees)."""
        t0, q, n = int(self.q_lens[:b].sum()), int(self.q_lens[b]), int(self.seq_lens[b])
        for i in range(q):
            yield t0 + i, self.q[t0 + i].double().numpy(), n - q + i + 1


def score_error(batch, q, k):
    """How far a score of fp32-accumulated products may be off, [H, keys]: each of the 576 sums
    rounds by at most 2^-23 of the magnitudes' sum (the tensor cores may cut instead of round);
    on an e4m3 cache q is held as two e4m3 parts, off by at most 2^-18 of the row's largest."""
    err = 576 * 2.0 ** -23 * (np.abs(q) @ np.abs(k).T)
    if batch.kind != "bf16":
        err = err + 2.0 ** -17 * np.abs(q).max(1, keepdims=True) * np.abs(k).sum(1)
    return inputs.SM_SCALE * err


def attend(batch):
    """out, lse and the bounds of their errors.

    P of a key enters the e4m3 products as two parts: off by 2^-8 of itself, or, where it is
    small, by 2^-10 where the row's largest is at least 2^4. The partial results of a split
    round to bf16, and so does the output: 2^-8 each."""
    total = batch.q.shape[0]
    out, bound = np.zeros((total, batch.H, DV)), np.zeros((total, batch.H, DV))
    lse, lse_bound = np.zeros((total, batch.H)), np.zeros((total, batch.H))
    for b in range(len(batch.seq_lens)):
        codes, v = batch.codes(b), batch.key_scales(b)
        k = codes * v[:, None]
        for t, q, n in batch.rows(b):
            s = inputs.SM_SCALE * (q @ k[:n].T)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(1, keepdims=True)
            p /= l
            lse[t] = (m + np.log(l))[:, 0]
            ds = score_error(batch, q, k[:n])
            lse_bound[t] = ds.max(1) + 1e-6 * (1 + np.abs(lse[t]))
            out[t] = p @ k[:n, :DV]
            mag = p @ np.abs(k[:n, :DV])
            term = p * v[:n]
            top = term.max(1, keepdims=True)
            small = 2.0 ** -14 * top * (term < 2.0 ** -4 * top)
            bound[t] = (3 * 2.0 ** -8 + 2 * ds.max(1, keepdims=True)) * mag + small @ np.abs(codes[:n, :DV]) + 1e-30
    return out, bound, lse, lse_bound


def weights(batch, lse, decay, old, counted=None):
    """The sums [B, stride] and the bounds of their errors, for the given lse (float64)."""
    w, bound = old.astype(np.float64).copy(), np.zeros(old.shape)
    for b, n in enumerate(batch.seq_lens):
        w[b, :n] = w[b, :n] * decay if decay else 0.0
        bound[b, :n] += 2.0 ** -23 * np.abs(w[b, :n])
        k = batch.codes(b) * batch.key_scales(b)[:, None]
        rows = batch.H * int(batch.q_lens[b])
        for i, (t, q, seen) in enumerate(batch.rows(b)):
            if counted is not None and i >= counted[b]:
                break
            p = np.exp(inputs.SM_SCALE * (q @ k[:seen].T) - lse[t][:, None])
            ds = score_error(batch, q, k[:seen])
            w[b, :seen] += p.sum(0)
            # exp2 approximated to 2^-22; its argument and lse round to 2^-23 of their sizes
            size = np.where(np.isfinite(lse[t]), np.abs(lse[t]), 0.0)[:, None] + 2.0 * math.log(2.0) * 40
            rel = ds + 2.0 ** -21 + 2.0 ** -22 * size + rows * 2.0 ** -23
            bound[b, :seen] += (p * rel).sum(0)
    return w, bound + 1e-37
