"""Plain references of the streaming operators: the plan one sequence after
another, the attention and the norm in 64 bits, and packed test batches."""
import math

import torch

D = 64


def plan(cached, new, free, n_free, table, page, n_rows):
    """(table, cu_rows, kv_lens, slots, counts) as lists, one sequence after another."""
    n_free = max(0, min(n_free, len(free)))
    table = [list(r) for r in table]
    width = len(table[0])
    cu, kv, slots, refused, row, asked, taken = [0], [], [], 0, 0, 0, 0
    for b, (c, n) in enumerate(zip(cached, new)):
        c, n = max(0, c), max(0, n)
        row += n
        have, want = -(-c // page), -(-(c + n) // page)
        ok = row <= n_rows and want <= width
        if ok:
            asked += want - have
            ok = want == have or asked <= n_free
        if ok:
            for i in range(have, want):
                table[b][i] = free[n_free - 1 - taken]
                taken += 1
            slots += [table[b][t // page] * page + t % page for t in range(c, c + n)]
            kv.append(c + n)
        else:
            refused += 1
            kv.append(c)
            slots += [-1] * max(0, min(n, n_rows - cu[-1]))
        cu.append(min(row, n_rows))
    slots += [-1] * (n_rows - len(slots))
    return table, cu, kv, slots, [n_free - taken, refused]


def limit(kv, pos, unit):
    if unit == 0:
        return kv
    return 0 if pos < 0 else min(kv, (pos // unit + 1) * unit)


def attention(q, k_seqs, v_seqs, cu, kv, unit, scale=None):
    """64-bit (o, lse, sum of p |v| over l) of packed rows; k_seqs[b]: [kv, Hkv, 64]."""
    scale = 1 / math.sqrt(D) if scale is None else scale
    rows, heads, _ = q.shape
    o = torch.zeros(rows, heads, D, dtype=torch.float64, device=q.device)
    spread = torch.zeros_like(o)
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64, device=q.device)
    for b in range(len(kv)):
        n = cu[b + 1] - cu[b]
        if n == 0 or kv[b] == 0:
            continue
        r = slice(cu[b], cu[b + 1])
        lim = torch.tensor([limit(kv[b], kv[b] - n + i, unit) for i in range(n)], device=q.device)
        seen = torch.arange(kv[b], device=q.device)[None, :] < lim[:, None]
        some = lim > 0
        group = heads // k_seqs[b].shape[1]
        for h in range(heads):
            k, v = k_seqs[b][:kv[b], h // group].double(), v_seqs[b][:kv[b], h // group].double()
            s = (q[r, h].double() @ k.T) * scale
            s = s.masked_fill(~seen, -math.inf)[some]
            p = torch.softmax(s, -1)
            o[r, h] = torch.zeros(n, D, dtype=torch.float64, device=q.device).index_copy(
                0, some.nonzero()[:, 0], p @ v)
            spread[r, h] = torch.zeros(n, D, dtype=torch.float64, device=q.device).index_copy(
                0, some.nonzero()[:, 0], p @ v.abs())
            lse[r, h] = lse[r, h].index_copy(0, some.nonzero()[:, 0], torch.logsumexp(s, -1))
    return o, lse, spread


def normed(t, kind, eps, w, b):
    if kind == "layer":
        t = t - t.mean(-1, keepdim=True)
    t = t / (t.square().mean(-1, keepdim=True) + eps).sqrt()
    t = t if w is None else t * w.double()
    return t if b is None else t + b.double()


class Batch:
    """Sequences of given lengths in a paged cache whose other contents are NaN."""

    def __init__(self, kv, new, page, heads, kv_heads, seed=0, layout="head", extra=3, pad=0, q_scale=1.0,
                 device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.kv, self.new, self.page = list(kv), list(new), page
        self.cu = [sum(new[:b]) for b in range(len(new) + 1)]
        self.rows = self.cu[-1] + pad
        held = [-(-n // page) for n in kv]
        n_pages = sum(held) + extra
        width = max(held + [1]) + 2
        order = torch.randperm(n_pages, generator=g).tolist()
        nan = float("nan")
        if layout == "head":     # [pages, heads, page, 64]
            k_pages, v_pages = (torch.full((n_pages, kv_heads, page, D), nan).bfloat16() for _ in range(2))
        elif layout == "token":  # [pages, page, heads, 64]
            k_pages, v_pages = (torch.full((n_pages, page, kv_heads, D), nan).bfloat16().transpose(1, 2)
                                for _ in range(2))
        else:                    # K and V of a page side by side
            both = torch.full((n_pages, 2, kv_heads, page, D), nan).bfloat16()
            k_pages, v_pages = both[:, 0], both[:, 1]
        self.k_seqs = [torch.randn(n, kv_heads, D, generator=g).bfloat16() for n in kv]
        self.v_seqs = [torch.randn(n, kv_heads, D, generator=g).bfloat16() for n in kv]
        table = torch.full((len(kv), width), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(kv):
            for i in range(held[b]):
                table[b, i] = order[at]
                part = slice(i * page, min(n, (i + 1) * page))
                m = part.stop - part.start
                k_pages[order[at], :, :m] = self.k_seqs[b][part].transpose(0, 1)
                v_pages[order[at], :, :m] = self.v_seqs[b][part].transpose(0, 1)
                at += 1
        self.q = (q_scale * torch.randn(self.rows, heads, D, generator=g)).bfloat16().to(device)

        def move(t):  # keeps the strides
            if device == "cpu":
                return t
            base = t if t._base is None else t._base
            moved = base.to(device)
            return moved.as_strided(t.shape, t.stride(), t.storage_offset())

        if layout == "both":
            both = both.to(device)
            self.k_pages, self.v_pages = both[:, 0], both[:, 1]
        else:
            self.k_pages, self.v_pages = move(k_pages), move(v_pages)
        self.table = table.to(device)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=device)  # noqa: E731
        self.cu_rows, self.kv_lens = i32(self.cu), i32(self.kv)
        self.k_seqs = [x.to(device) for x in self.k_seqs]
        self.v_seqs = [x.to(device) for x in self.v_seqs]

    def reference(self, unit, scale=None):
        return attention(self.q, self.k_seqs, self.v_seqs, self.cu, self.kv, unit, scale)
