"""The paged 8-bit KV cache on the CPU, from its definition (include/kvcache.h)."""
import math

import torch

from tests import window_ref

F8 = torch.float8_e4m3fn


def page_exp(amax: float) -> int:
    """Smallest e >= -126 with amax <= 448 * 2^e."""
    if amax == 0.0:
        return -126
    m, e = math.frexp(amax / 448.0)
    return max(e if m > 0.5 else e - 1, -126)


def round_e4m3(x):
    """fp64 -> the nearest e4m3 value as fp64, clamped to +-448, NaN kept."""
    return x.clamp(-448, 448).float().to(F8).double()


def append(new, pages, scales, table, lens, n_new):
    """new [B, H, T, D] into copies of pages (e4m3) and scales; returns both."""
    B, H, T, D = new.shape
    P = pages.shape[2]
    raw, scales = pages.view(torch.uint8).clone(), scales.clone()
    for b in range(B):
        n, ln = int(n_new[b]), int(lens[b])
        for t in range(n):
            pos = ln - n + t
            pid, r = int(table[b, pos // P]), pos % P
            fresh = t == 0 and r > 0   # the page already holds tokens
            if t == 0 or r == 0:       # first new token of a page: the page's new tokens together
                cnt = min(n - t, P - r)
                x = new[b, :, t:t + cnt].double()
                for h in range(H):
                    fin = x[h][torch.isfinite(x[h])]
                    e = page_exp(float(fin.abs().max()) if fin.numel() else 0.0)
                    s = 2.0 ** e
                    if fresh:
                        old = float(scales[pid, h])
                        s = max(s, old)
                        held = raw[pid, h, :r].view(F8).double() * (old / s)
                        raw[pid, h, :r] = held.float().to(F8).view(torch.uint8)
                    raw[pid, h, r:r + cnt] = round_e4m3(x[h] / s).float().to(F8).view(torch.uint8)
                    scales[pid, h] = s
    return raw.view(F8), scales


def dense(pages, scales, row, length):
    """[H, length, D] fp64 values of one sequence."""
    P = pages.shape[2]
    ids = row[: -(-length // P)].long()
    x = pages.view(torch.uint8)[ids].view(F8).double() * scales[ids].double()[:, :, None, None]
    return x.transpose(0, 1).reshape(pages.shape[1], -1, pages.shape[3])[:, :length]


def attention(q, kp, vp, ks, vs, table, lens, window=0, sinks=0, scale=None):
    """out and lse [B, Hq, Nq, ...] as fp64; evicted or missing pages only where no query looks."""
    B, Hq, Nq, D = q.shape
    P = kp.shape[2]
    G = Hq // kp.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:3], float("-inf"), dtype=torch.float64)
    for b in range(B):
        n = int(lens[b])
        rows = min(Nq, n)   # queries before the first position see nothing
        if rows == 0:
            continue
        row = table[b].clone()
        seen = window_ref.visible(rows, n, window, sinks).any(0)
        for j in range(-(-n // P)):
            if not seen[j * P:(j + 1) * P].any():
                row[j] = int(row[(n - 1) // P])   # any readable page
        k, v = dense(kp, ks, row, n), dense(vp, vs, row, n)
        k[:, ~seen] = 0.0
        v[:, ~seen] = 0.0
        for h in range(Hq):
            o, l = window_ref.head(q[b, h, Nq - rows:], k[h // G], v[h // G], window, sinks, scale)
            out[b, h, Nq - rows:], lse[b, h, Nq - rows:] = o, l
    return out, lse


class Pages:
    """Tables, lengths and holder counts as Python lists."""

    def __init__(self, table, lens, refs, page):
        self.table, self.lens, self.refs = table.tolist(), lens.tolist(), refs.tolist()
        self.page = page

    def cols(self, n):
        return -(-n // self.page)

    def free(self):
        return [i for i, r in enumerate(self.refs) if r == 0]

    def drop(self, i):
        if i >= 0:
            self.refs[i] -= 1

    def reserve(self, n_new, window=0, sinks=0):
        saved = [r[:] for r in self.table], self.lens[:], self.refs[:]
        before = len(self.free())
        need, ok = [], True
        for c, n in enumerate(n_new):
            ln = self.lens[c]
            if n and self.cols(ln + n) > len(self.table[c]):
                ok = False
            need.append(self.cols(ln + n) - self.cols(ln) if n else 0)
            if n and window > 0:
                for j in range(self.cols(sinks), min(max(ln - window + 1, 0) // self.page, len(self.table[c]))):
                    self.drop(self.table[c][j])
                    self.table[c][j] = -1
        free = self.free()
        if not ok or sum(need) > len(free):
            self.table, self.lens, self.refs = saved
            return [0, 0, 0, before]
        back = len(free) - before
        ids = iter(free)
        for c, n in enumerate(n_new):
            first = self.cols(self.lens[c])
            for k in range(need[c]):
                i = next(ids)
                self.table[c][first + k] = i
                self.refs[i] = 1
            self.lens[c] += n
        return [1, sum(need), back, len(free) - sum(need)]

    def reassign(self, parents):
        old, lens = [r[:] for r in self.table], self.lens[:]
        saved = self.refs[:]
        before = len(self.free())
        pairs, seen = [], set(c for c, q in enumerate(parents) if c == q)
        for c, q in enumerate(parents):
            if q == c:
                continue
            for i in old[c]:
                self.drop(i)
        want = []
        for c, q in enumerate(parents):
            if q == c:
                continue
            row, ln = ([-1] * len(old[c]), 0) if q < 0 else (old[q][:], lens[q])
            tail = -1
            if q >= 0 and ln % self.page:
                if q in seen:
                    tail = ln // self.page
                seen.add(q)
            for j, i in enumerate(row):
                if i >= 0 and j != tail:
                    self.refs[i] += 1
            if tail >= 0:
                want.append((c, tail))
            self.table[c], self.lens[c] = row, ln
        free = self.free()
        if len(want) > len(free):
            self.table, self.lens, self.refs = old, lens, saved
            return [0, 0, 0, before], []
        for (c, tail), i in zip(want, free):
            pairs.append((self.table[c][tail], i))
            self.table[c][tail] = i
            self.refs[i] = 1
        return [1, len(want), len(free) - before, len(free) - len(want)], pairs

    def compact(self):
        held = sum(r > 0 for r in self.refs)
        holes = [i for i in range(held) if self.refs[i] == 0]
        movers = [i for i in range(held, len(self.refs)) if self.refs[i] > 0]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[to.get(i, i) for i in r] for r in self.table]
        return [1, len(movers), held, len(self.refs) - held], list(zip(movers, holes))
