"""A paged latent cache on the GPU for tests, its plain model on lists, and
the attention it answers in 64 bits."""
import numpy as np
import torch

import edge_moe_serving_gb300 as moe

DEV = "cuda"


class Paged:
    """Cache arrays of a test: every page starts as NaN, so whatever reads a place no token was stored in shows."""

    def __init__(self, n_pages, page, rank, rope, max_seqs, max_blocks, layers=1, device=DEV):
        self.page, self.rank, self.rope, self.row = page, rank, rope, rank + rope
        self.pages = torch.full((layers, n_pages, page, self.row), float("nan"), dtype=torch.bfloat16, device=device)
        self.table = torch.full((max_seqs, max_blocks), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(max_seqs, dtype=torch.int32, device=device)
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.handle = moe.moe_kv_cache(self.pages.data_ptr(), self.table.data_ptr(), self.lens.data_ptr(),
                                       self.refs.data_ptr(), layers, n_pages, page, rank, rope, max_seqs, max_blocks, 0)
        n = moe.moe_kv_workspace_size(self.handle, max_seqs)
        self.ws = torch.empty(max(n, 256), dtype=torch.uint8, device=device)

    def bits(self):
        b = int(self.status.item())
        self.status.zero_()
        return b

    def fill(self, lens, seed=0, layer=0, shared_blocks=0, spread=1.0):
        """Gives sequence i lens[i] random rows on pages scattered over the pool (the first shared_blocks blocks of
        all sequences are sequence 0's), without the library.  Returns the rows in 64 bits, per sequence."""
        g = torch.Generator().manual_seed(seed)
        order = torch.randperm(self.refs.numel(), generator=g).tolist()
        table = np.full(tuple(self.table.shape), -1, np.int32)
        refs = np.zeros(self.refs.numel(), np.int32)
        rows = []
        for i, n in enumerate(lens):
            x = (torch.randn(n, self.row, generator=g) * spread).to(torch.bfloat16)
            for b in range(-(-n // self.page)):
                if i and b < shared_blocks:
                    p = int(table[0, b])
                    x[b * self.page:(b + 1) * self.page] = rows[0][b * self.page:min(n, (b + 1) * self.page)]
                else:
                    p = order.pop()
                    part = x[b * self.page:(b + 1) * self.page]
                    self.pages[layer, p, :len(part)] = part.to(self.pages.device)
                table[i, b] = p
                refs[p] += 1
            rows.append(x)
        self.table.copy_(torch.from_numpy(table))
        self.refs.copy_(torch.from_numpy(refs))
        self.lens[:len(lens)] = torch.tensor(lens, dtype=torch.int32)
        return [x.double() for x in rows]


def attend64(q, k, v, scale, limit):
    """softmax(scale q k^T over t < limit[r]) v in 64 bits, and sum p |v|, log-sum-exp.  A row with no token: 0, 0, -inf."""
    z = (q @ k.T) * scale
    t = torch.arange(k.shape[0])
    z = z.masked_fill(t[None] >= torch.as_tensor(limit)[:, None], -float("inf"))
    lse = torch.logsumexp(z, -1) if k.shape[0] else torch.full((q.shape[0],), -float("inf"), dtype=torch.float64)
    p = torch.exp(z - torch.where(lse == -float("inf"), torch.zeros_like(lse), lse)[:, None])
    return p @ v, p @ v.abs(), lse


class Model:
    """The page calls on lists: refs, tables and lengths as the header states them, pages as sets of rows moved."""

    def __init__(self, n_pages, page, max_seqs, max_blocks):
        self.page, self.max_blocks = page, max_blocks
        self.refs = [0] * n_pages
        self.table = [[] for _ in range(max_seqs)]
        self.lens = [0] * max_seqs
        self.data = {}          # (page, slot) -> row id

    def blocks(self, n):
        return -(-n // self.page)

    def free_pages(self):
        return [i for i, r in enumerate(self.refs) if r == 0]

    def reserve(self, seqs, n_new):
        todo, seen = [], set()
        for s, n in zip(seqs, n_new):
            if 0 <= s < len(self.lens) and n >= 0 and s not in seen:
                todo.append((s, n))
            seen.add(s)
        free = self.free_pages()
        need = [self.blocks(self.lens[s] + n) - self.blocks(self.lens[s]) for s, n in todo]
        if sum(need) > len(free) or any(self.blocks(self.lens[s] + n) > self.max_blocks for s, n in todo):
            return False
        for (s, n), k in zip(todo, need):
            for _ in range(k):
                p = free.pop(0)
                self.refs[p] = 1
                self.table[s].append(p)
            self.lens[s] += n
        return True

    def append(self, s, pos, row):
        self.data[(self.table[s][pos // self.page], pos % self.page)] = row

    def rows(self, s):
        return [self.data.get((self.table[s][t // self.page], t % self.page)) for t in range(self.lens[s])]

    def fork(self, src, dst):
        seen, pairs = set(), []
        for a, b in zip(src, dst):
            ok = 0 <= a < len(self.lens) and 0 <= b < len(self.lens) and b not in seen
            if 0 <= b < len(self.lens):
                seen.add(b)
            if ok and a != b:
                pairs.append((a, b))
        free = self.free_pages()
        if sum(self.lens[a] % self.page != 0 for a, _ in pairs) > len(free):
            return False
        old_t, old_l, old_d = [list(t) for t in self.table], list(self.lens), dict(self.data)
        for a, b in pairs:
            for p in old_t[b]:
                self.refs[p] -= 1
            new, n = list(old_t[a]), old_l[a]
            if n % self.page:
                p = free.pop(0)
                for j in range(n % self.page):
                    self.data[(p, j)] = old_d.get((new[-1], j))
                new[-1] = p
            for p in new:
                self.refs[p] += 1
            self.table[b], self.lens[b] = new, n
        return True

    def free(self, seqs):
        for s in seqs:
            if 0 <= s < len(self.lens):
                for p in self.table[s]:
                    self.refs[p] -= 1
                self.table[s], self.lens[s] = [], 0

    def compact(self):
        live = [i for i, r in enumerate(self.refs) if r]
        n = len(live)
        move = dict(zip([i for i in live if i >= n], [i for i in range(n) if self.refs[i] == 0]))
        for a, b in move.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            for j in range(self.page):
                if (a, j) in self.data:
                    self.data[(b, j)] = self.data[(a, j)]
        self.table = [[move.get(p, p) for p in t] for t in self.table]
        return n
