"""Plain 64-bit forms of the tree-speculation calls, for their tests (CPU, torch float64)."""
import math

import torch


def parents_of(kind: str, batch: int, T: int, seed: int = 0) -> torch.Tensor:
    """Parent indices (batch, T): a chain, a star (all nodes follow the cache) or random trees."""
    g = torch.Generator().manual_seed(seed)
    p = torch.full((batch, T), -1, dtype=torch.int32)
    for t in range(1, T):
        if kind == "chain":
            p[:, t] = t - 1
        elif kind == "random":
            p[:, t] = torch.randint(-1, t, (batch,), generator=g, dtype=torch.int32)
    return p


def seen_of(parents: torch.Tensor) -> torch.Tensor:
    """(batch, T, T) truth values: node t's ancestors and itself, by walking up."""
    batch, T = parents.shape
    seen = torch.zeros((batch, T, T), dtype=torch.bool)
    for b in range(batch):
        for t in range(T):
            a = t
            while a >= 0:
                seen[b, t, a] = True
                a = int(parents[b, a])
    return seen


def words_of(seen: torch.Tensor) -> torch.Tensor:
    """Truth values (batch, T, T) as int32 words (batch * T, ceil(T / 32))."""
    batch, T, _ = seen.shape
    n = (T + 31) // 32
    out = torch.zeros((batch * T, n), dtype=torch.int64)
    for j in range(T):
        out[:, j // 32] |= seen[:, :, j].reshape(-1).long() << (j % 32)
    return torch.where(out >= 1 << 31, out - (1 << 32), out).int()


def attend(q, rows, seen, w_uv, r: int, scale: float):
    """One sequence in 64 bits: q (T, H, D), rows (L, D) with the T drafted ones last, seen (T, T).

    Returns o (T, H, d_v), lse (T, H), `size` (T, H, d_v): the sums with every term taken absolute,
    which rounding errors are relative to, and `dot` (T, H): the largest sum of absolute
    products of a score.
    """
    T, H, _ = q.shape
    L = rows.shape[0]
    q, rows, w_uv = q.double(), rows.double(), w_uv.double()
    vis = torch.ones((T, L), dtype=torch.bool)
    vis[:, L - T:] = seen
    keep = vis.any(0)  # a row that nobody sees may hold anything
    rows, vis = rows[keep], vis[:, keep]
    s = torch.einsum("thd,jd->thj", q, rows) * scale
    s = torch.where(vis[:, None], s, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(torch.isinf(lse)[..., None], 0.0, torch.exp(s - lse[..., None]))
    v = torch.where(vis.any(0)[:, None], rows[:, :r], 0.0)
    o = torch.einsum("hvr,thr->thv", w_uv, torch.einsum("thj,jr->thr", p, v))
    size = torch.einsum("hvr,thr->thv", w_uv.abs(), torch.einsum("thj,jr->thr", p, v.abs()))
    dots = torch.einsum("thd,jd->thj", q.abs(), rows.abs()) * scale
    dot = torch.where(vis[:, None], dots, 0.0).amax(-1) if L else torch.zeros(T, H)
    return o, lse, size, dot


def tolerances(dtype, o, size, dot, D: int, L: int):
    """(o, lse) tolerances. One rounding to bf16 is off by 2^-8 of the value at most; fp32 sums of n
    terms by n 2^-23 of the sum of the terms' sizes (2^-23 and not 2^-24: a tensor core may
    truncate).

    lse: a score by D 2^-23 of `dot`, the exponentials, their sum and the logarithm by
    (8 + L) 2^-23. The weights carry twice the scores' error. o: in bf16 the weights are rounded
    (2^-8 of `size`) and o is (2^-8 of o); the latent sums' two bf16 terms leave 2^-16."""
    fp = 2.0 ** -23
    lse_tol = D * fp * dot + (8 + L) * fp
    rel = 2 * lse_tol.amax() + (L + 512) * fp
    if dtype == torch.bfloat16:
        return (2.0 ** -8 + 2.0 ** -16 + rel) * size + 2.0 ** -8 * o.abs() + 1e-30, lse_tol
    return rel * size + 2.0 ** -24 * o.abs() + 1e-30, lse_tol


def tables(bs, lens, new, table, held, free, count, num_blocks, max_tokens):
    """mla_build_tables request by request: (table, held, free, count, cu, seq, pos, slots, bits)."""
    OOB, LEN, FULL = 1, 8, 32
    table = [list(row) for row in table]
    free, held, width, bits = list(free), list(held), len(table[0]), 0
    ok = [0 <= n <= width * bs and 0 <= m and (m <= n or n == 0) and 0 <= h <= width
          for n, m, h in zip(lens, new, held)]
    want = [-(-n // bs) if good else h for n, h, good in zip(lens, held, ok)]
    if not all(ok):
        bits |= LEN
    back = sum(max(h - w, 0) for h, w in zip(held, want))
    moves = 0 <= count <= num_blocks and back <= num_blocks - count
    out, n = list(held), count
    if moves:
        for b, row in enumerate(table):
            for i in range(want[b], held[b]):
                free[n] = row[i]
                n += 1
            out[b] = min(held[b], want[b])
    else:
        bits |= LEN
    served, full = [], not moves
    for b, row in enumerate(table):
        due = max(want[b] - held[b], 0)
        full = full or due > n
        served.append(due == 0 or not full)
        if due and full:
            bits |= FULL
        elif due:
            for i in range(held[b], want[b]):
                n -= 1
                row[i] = free[n]
                if not 0 <= row[i] < num_blocks:
                    bits |= OOB
            out[b] = want[b]
    cu, seq, pos, slots = [0], [], [], []
    for b, row in enumerate(table):
        m = new[b] if ok[b] else 0
        cu.append(min(cu[-1] + m, max_tokens) if cu[-1] + m <= max_tokens else max_tokens)
        if len(seq) + m > max_tokens:
            bits |= LEN
        for p in range(lens[b] - m, lens[b]):
            if len(seq) == max_tokens:
                break
            if lens[b] == 0:  # padding
                seq.append(-1)
                pos.append(0)
                slots.append(-1)
                continue
            blk = row[p // bs]
            seq.append(b)
            pos.append(p)
            if served[b] and 0 <= blk < num_blocks:
                slots.append(blk * bs + p % bs)
            else:
                slots.append(-1)
                if served[b]:
                    bits |= OOB
    pad = max_tokens - len(seq)
    return (table, out, free, n, cu, seq + [-1] * pad, pos + [0] * pad, slots + [-1] * pad, bits)
