"""Plain 64-bit references of the speculative-decoding operators (test-side only): tree attention
over pages, draft verification, and a list-of-lists model of the page operations."""
import numpy as np

PAGE = 64


def ancestors(parents):
    """seen[i, k]: draft k is node i or an ancestor of it."""
    n = len(parents)
    seen = np.eye(n, dtype=bool)
    for i in range(1, n):
        seen[i] |= seen[parents[i]]
    return seen


def mask_words(seen, words=None):
    """Boolean [n, k] masks as int32 words, bit k % 32 of word k // 32."""
    n, k = seen.shape
    words = max(1, (k + 31) // 32) if words is None else words
    wide = np.zeros((n, words * 32), bool)
    wide[:, :k] = seen
    return np.packbits(wide, axis=1, bitorder="little").view(np.int32)


def tree_attention(q, rows, seen, ctx, scale):
    """q [n, H, 576], rows [ctx + n, 576], seen [n, n] -> O, lse and the bounds' ingredients: A = sum p |v|
    per output and s_abs = max over visible rows of scale * sum |q| |k| per (node, head)."""
    n, H = q.shape[:2]
    O, L = np.zeros((n, H, 512)), np.full((n, H), -np.inf)
    A, S = np.zeros((n, H, 512)), np.zeros((n, H))
    for i in range(n):
        see = np.concatenate([np.arange(ctx), ctx + np.nonzero(seen[i])[0]])
        if len(see) == 0:
            continue
        k = rows[see]
        s = scale * (q[i] @ k.T)
        S[i] = (scale * (np.abs(q[i]) @ np.abs(k).T)).max(1)
        m = s.max(1)
        p = np.exp(s - m[:, None])
        L[i] = m + np.log(p.sum(1))
        p /= p.sum(1)[:, None]
        O[i] = p @ k[:, :512]
        A[i] = p @ np.abs(k[:, :512])
    return O, L, A, S


def verify(target, draft, tokens, parents, r, max_path):
    """One request's walk and next token, in 64 bits, from the definition."""
    n, u, depth = len(tokens), 0, [0]
    if n == 0:
        return 0, [], -1
    target = np.clip(np.nan_to_num(np.asarray(target, np.float64), nan=0.0, posinf=1.0), 0.0, 1.0)
    if draft is not None:
        draft = np.clip(np.nan_to_num(np.asarray(draft, np.float64), nan=0.0, posinf=1.0), 0.0, 1.0)
    w, S = target[0].copy(), 1.0
    V = target.shape[1]
    i = 0
    while len(depth) < max_path:
        i += 1
        if i >= n:
            break
        if parents[i] != u or not 0 <= parents[i] < i or not 0 <= tokens[i] < V:
            continue
        x = tokens[i]
        q = np.zeros(V) if draft is None else draft[u]
        if draft is None:
            q[x] = 1.0
        if float(r[i]) * q[x] * S < w[x]:
            u = i
            depth.append(i)
            w, S = target[u].copy(), 1.0
        elif draft is None:
            S -= w[x]
            w[x] = 0.0
        else:
            w = np.maximum(w - q * S, 0.0)
            S = w.sum()
    if w.sum() <= 0:
        w = target[u]
    if w.sum() <= 0:
        return len(depth), depth, -1
    c = np.cumsum(w)
    token = int((c <= min(max(float(r[0]), 0.0), 1.0) * c[-1]).sum())
    return len(depth), depth, min(token, int(np.nonzero(w > 0)[0][-1]))


class Pages:
    """The page operations, request by request and page by page."""

    def __init__(self, n_slots, max_pages, n_pages):
        self.seq = [0] * n_slots
        self.table = [[-1] * max_pages for _ in range(n_slots)]
        self.ref = [0] * n_pages
        self.status = set()

    @staticmethod
    def pages(rows):
        return -(-rows // PAGE)

    def _free(self):
        return [p for p, c in enumerate(self.ref) if c == 0]

    def resize(self, new):
        most = len(self.table[0]) * PAGE
        refused = set()
        for s, now in enumerate(new):
            if not (0 <= now <= most and 0 <= self.seq[s] <= most):
                self.status.add("bounds")
                refused.add(s)
                continue
            for i in range(self.pages(now), self.pages(self.seq[s])):
                p, self.table[s][i] = self.table[s][i], -1
                if 0 <= p < len(self.ref) and self.ref[p] > 0:
                    self.ref[p] -= 1
                else:
                    self.status.add("bounds")
        want = []
        for s, now in enumerate(new):
            if s in refused or now <= self.seq[s]:
                continue
            if self.seq[s] % PAGE:
                p = self.table[s][self.seq[s] // PAGE]
                if not 0 <= p < len(self.ref) or self.ref[p] > 1:
                    self.status.add("bounds" if not 0 <= p < len(self.ref) else "shared")
                    refused.add(s)
                    continue
            want += [(s, i) for i in range(self.pages(self.seq[s]), self.pages(now))]
        free = self._free()
        enough = len(want) <= len(free)
        if enough:
            for (s, i), p in zip(want, free):
                self.table[s][i] = p
                self.ref[p] = 1
        else:
            self.status.add("pages")
        for s, now in enumerate(new):
            if s not in refused and (enough or now <= self.seq[s]):
                self.seq[s] = now

    def fork(self, src, dst):
        """Returns the page copies [(from, to, rows)]."""
        ok = [self.seq[d] == 0 for d in dst]
        if not all(ok):
            self.status.add("bounds")
        need = [k for k, (s, d) in enumerate(zip(src, dst)) if ok[k] and self.seq[s] % PAGE]
        free = self._free()
        if len(need) > len(free):
            self.status.add("pages")
            return []
        fresh, copies = dict(zip(need, free)), []
        for k, (s, d) in enumerate(zip(src, dst)):
            if not ok[k]:
                continue
            full = self.seq[s] // PAGE
            for i in range(full):
                self.table[d][i] = self.table[s][i]
                self.ref[self.table[s][i]] += 1
            if k in fresh:
                self.table[d][full] = fresh[k]
                self.ref[fresh[k]] = 1
                copies.append((self.table[s][full], fresh[k], self.seq[s] % PAGE))
            self.seq[d] = self.seq[s]
        return copies
