"""Workloads of speculative decoding with a tree of drafted tokens over the paged latent cache.

Five operators that one serving step calls one after another:

* ``tables``: block tables and slot maps of a step, built on the GPU from request lengths
* ``masks``: ancestor masks and RoPE positions of a tree given by its parent indices
* ``append``: cache rows written through a slot map (a drafted token's RoPE position is its
  depth's, its slot its own)
* ``tree``: attention of every drafted token over its sequence's cache and its ancestors, then
  the value up-projection
* ``commit``: the accepted path's rows moved together at the end of the sequence

``run`` computes them in elementary torch operations (32-bit floats, 64-bit angles), or, with
``own`` set, by this repository's kernels. ``exact`` gives the results in 64 bits.
"""
import math

import torch

own = False

# Model shapes: the DeepSeek-V2 attention shape (with 128 heads, or a tensor-parallel shard's
# 64, 32 or 16) and its scaled-down variant.
_SHAPES = {
    "dsv2": dict(r=512, dr=64, dh=128, bs=64),
    "small": dict(r=64, dr=32, dh=64, bs=64),
}


def listed():
    return [
        # one decode step of the benchmark batch: a block falls due every 64 tokens, a few
        # requests have ended and give theirs back
        dict(name="tables decode", op="tables", batch=64, longest=8192, prompts=0, tokens=64),
        # a step that admits prompts beside running requests: the slot map is what is long
        dict(name="tables prompts", op="tables", batch=128, longest=8192, prompts=32,
             tokens=131072),
        # four drafted tokens for each of 32 sequences
        dict(name="masks 32x4", op="masks", batch=32, tree=4),
        # wide trees for a large batch
        dict(name="masks 128x64", op="masks", batch=128, tree=64),
        # the drafted rows of one step
        dict(name="append 32x4", op="append", dtype="bf16", shape="dsv2", tokens=128,
             longest=16384),
        # a step's prompts: 4 x 4096 tokens
        dict(name="append prompts", op="append", dtype="bf16", shape="dsv2", tokens=16384,
             longest=4096),
        # the scaled-down model in fp32, odd tree
        dict(name="tree small f32", op="tree", dtype="f32", shape="small", heads=16, batch=8,
             cached=1024, ragged=False, tree=5),
        # one request, a short cache: what counts is latency
        dict(name="tree one request", op="tree", dtype="bf16", shape="dsv2", heads=128, batch=1,
             cached=1000, ragged=False, tree=8),
        # long contexts, few drafted tokens: the cache's bytes against the tensor cores
        dict(name="tree 32x16384x4", op="tree", dtype="bf16", shape="dsv2", heads=128, batch=32,
             cached=16384, ragged=False, tree=4),
        # ragged lengths, wide trees: the largest
        dict(name="tree ragged 64x16", op="tree", dtype="bf16", shape="dsv2", heads=128,
             batch=64, cached=8192, ragged=True, tree=16),
        # the accepted rows of one step
        dict(name="commit 32x4", op="commit", dtype="bf16", shape="dsv2", batch=32, tree=4,
             cached=1000),
        # wide trees, large batch
        dict(name="commit 256x64", op="commit", dtype="bf16", shape="dsv2", batch=256, tree=64,
             cached=500),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "masks", "append", "tree", "tree", "tree", "commit"])
    if op == "tables":
        batch = _log_int(rng, 1, 512)
        prompts = rng.randint(0, batch // 4)
        return dict(op=op, batch=batch, longest=_log_int(rng, 64, 8192), prompts=prompts,
                    tokens=batch + (_log_int(rng, 256, 131072) if prompts else 0))
    if op == "masks":
        return dict(op=op, batch=_log_int(rng, 1, 256), tree=_log_int(rng, 1, 128))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    shape = "dsv2" if dtype == "bf16" and rng.random() < 0.75 else "small"
    if op == "append":
        return dict(op=op, dtype=dtype, shape=rng.choice(["dsv2", "small"]),
                    tokens=_log_int(rng, 1, 16384), longest=_log_int(rng, 16, 32768))
    if op == "commit":
        return dict(op=op, dtype=dtype, shape=rng.choice(["dsv2", "small"]),
                    batch=_log_int(rng, 1, 256), tree=_log_int(rng, 1, 64),
                    cached=_log_int(rng, 1, 1024))
    if shape == "small":
        return dict(op=op, dtype=dtype, shape=shape, heads=rng.choice([8, 16]),
                    batch=_log_int(rng, 1, 16), cached=_log_int(rng, 1, 2048),
                    ragged=rng.random() < 0.5, tree=_log_int(rng, 1, 16))
    heads = rng.choice([16, 32, 64, 128, 128])
    batch, tree = _log_int(rng, 1, 64), _log_int(rng, 1, 32)
    # scores of all (head, token, row) triples: at most those of the largest listed case
    most = 64 * 4096 * 16 * 128 // (batch * tree * heads)
    return dict(op=op, dtype=dtype, shape=shape, heads=heads, batch=batch,
                cached=_log_int(rng, 1, max(2, min(32768, most))), ragged=rng.random() < 0.5,
                tree=tree)


# ------------------------------------------------------------------------------------ inputs

def _dims(case):
    d = dict(_SHAPES[case["shape"]])
    d["dt"] = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    d["D"] = d["r"] + d["dr"]
    d["scale"] = 1.0 / math.sqrt(d["dh"] + d["dr"])
    return d


def _ints(g, lo, hi, shape):
    """Whole numbers in [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _parents(g, batch, tree):
    """Random trees: node 0 follows the cache, every other node some earlier node."""
    t = torch.arange(tree, device="cuda")
    u = torch.rand((batch, tree), generator=g, device="cuda")
    p = (u * t).floor().clamp(max=(t - 1).clamp(min=0)).to(torch.int32)
    p[:, 0] = -1
    return p


def _ancestors(parents):
    """(batch, T, T) truth values: node t's ancestors and itself."""
    batch, tree = parents.shape
    at = torch.arange(tree, device=parents.device)
    reach = (parents[:, :, None] == at) | (at[:, None] == at)
    for _ in range(max(1, tree - 1).bit_length()):
        reach = torch.matmul(reach.float(), reach.float()) > 0
    return reach


def _words(reach):
    """Truth values (batch, T, T) as 32-bit words, bit j % 32 of word j / 32 for node j."""
    batch, tree, _ = reach.shape
    n = (tree + 31) // 32
    bits = torch.zeros((batch, tree, 32 * n), dtype=torch.int64, device=reach.device)
    bits[:, :, :tree] = reach
    w = (bits.view(batch, tree, n, 32) << torch.arange(32, device=reach.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).view(batch * tree, n)


def _table(g, batch, longest, bs):
    """Block table whose blocks lie anywhere in the pool, and the pool's block count."""
    most = -(-longest // bs)
    ids = torch.randperm(batch * most, generator=g, device="cuda").to(torch.int32)
    return ids.view(batch, most), batch * most


def _prepare_tables(case, g):
    bs, batch, longest = 64, case["batch"], case["longest"]
    most = -(-longest // bs)
    lens = _ints(g, 1, longest, (batch,))
    new = torch.ones_like(lens)
    kind = torch.randperm(batch, generator=g, device="cuda")
    n = case["prompts"]
    first = torch.zeros(batch, dtype=torch.bool, device="cuda")
    first[kind[:n]] = True
    if n:  # prompts admitted by this step, all their tokens new, fitted to the step's budget
        room = case["tokens"] - batch
        share = lens[first].double()
        lens[first] = (share * min(1.0, room / float(share.sum()))).floor().clamp(min=1).int()
    new = torch.where(first, lens, new)
    ended = torch.zeros_like(first)
    ended[kind[n: n + (batch - n) // 16]] = True
    held = torch.where(first, 0, (lens - new + bs - 1) // bs).int()
    new = torch.where(ended, 0, new).int()
    lens = torch.where(ended, 0, lens).int()
    total = batch * most
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(most, device="cuda")
    rank = (torch.cumsum(held, 0) - held)[:, None] + col
    has = col < held[:, None]
    table = torch.where(has, ids[rank.clamp(max=total - 1)], -1).int().contiguous()
    used = int(held.sum())
    free = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    free[: total - used] = ids[used:]
    dev = dict(device="cuda")
    return dict(bs=bs, lens=lens, new=new, table=table, held=held, free=free,
                count=torch.tensor([total - used], dtype=torch.int32, **dev),
                held_out=torch.empty(batch, dtype=torch.int32, **dev),
                count_out=torch.empty(1, dtype=torch.int32, **dev),
                cu=torch.empty(batch + 1, dtype=torch.int32, **dev),
                seq=torch.empty(case["tokens"], dtype=torch.int32, **dev),
                pos=torch.empty(case["tokens"], dtype=torch.int32, **dev),
                slots=torch.empty(case["tokens"], dtype=torch.int64, **dev))


def _prepare_masks(case, g):
    batch, tree = case["batch"], case["tree"]
    return dict(parents=_parents(g, batch, tree), lens=_ints(g, tree, 32768, (batch,)), tree=tree,
                mask=torch.empty((batch * tree, (tree + 31) // 32), dtype=torch.int32,
                                 device="cuda"),
                pos=torch.empty(batch * tree, dtype=torch.int32, device="cuda"))


def _prepare_append(case, g):
    d = _dims(case)
    n, bs = case["tokens"], d["bs"]
    blocks = -(-n // bs) + 2
    rows = blocks * bs
    # the last row takes what has no slot; it is not part of the pool
    flat = torch.zeros((rows + 1, d["D"]), dtype=d["dt"], device="cuda")
    at = torch.randperm(rows, generator=g, device="cuda")[:n].to(torch.int64)
    at[n - n // 32:] = -1  # the padding of a step's fixed token count
    return dict(d, flat=flat, pool=flat[:rows].view(blocks, bs, d["D"]), slots=at,
                ckv=torch.randn((n, d["r"]), generator=g, device="cuda").to(d["dt"]),
                kr=torch.randn((n, d["dr"]), generator=g, device="cuda").to(d["dt"]),
                gamma=1 + 0.1 * torch.randn(d["r"], generator=g, device="cuda"),
                pos=_ints(g, 0, case["longest"] - 1, (n,)))


def _prepare_tree(case, g):
    d = _dims(case)
    batch, tree, H = case["batch"], case["tree"], case["heads"]
    if case["ragged"]:
        lens = _ints(g, 1, case["cached"], (batch,)) + tree
    else:
        lens = torch.full((batch,), case["cached"] + tree, dtype=torch.int32, device="cuda")
    table, blocks = _table(g, batch, case["cached"] + tree, d["bs"])
    # rows as an append leaves them: unit RMS latent, rotated key of unit variance
    pool = torch.randn((blocks, d["bs"], d["D"]), generator=g, device="cuda", dtype=d["dt"])
    q = torch.randn((batch * tree, H, d["D"]), generator=g, device="cuda")
    q[..., : d["r"]] *= math.sqrt(d["dh"] / d["r"])  # what W_UK of variance 1 / r gives
    w_uv = torch.randn((H, d["dh"], d["r"]), generator=g, device="cuda") / math.sqrt(d["r"])
    return dict(d, heads=H, tree=tree, lens=lens, table=table, pool=pool, q=q.to(d["dt"]),
                w_uv=w_uv.to(d["dt"]), mask=_words(_ancestors(_parents(g, batch, tree))),
                o=torch.empty((batch * tree, H, d["dh"]), dtype=d["dt"], device="cuda"),
                lse=torch.empty((batch * tree, H), device="cuda"))


def _prepare_commit(case, g):
    d = _dims(case)
    batch, tree = case["batch"], case["tree"]
    lens = _ints(g, 0, case["cached"], (batch,)) + tree
    table, blocks = _table(g, batch, case["cached"] + tree, d["bs"])
    pool = torch.randn((blocks, d["bs"], d["D"]), generator=g, device="cuda", dtype=d["dt"])
    # accepted paths: the first nodes of the tree, then nodes of the levels behind the path's
    # own length (a path of k nodes moves nodes from behind its k rows)
    most = max(1, min(16, tree // 2))
    count = _ints(g, 0, most, (batch,))
    head = (torch.rand(batch, generator=g, device="cuda") * (count + 1)).int()
    col = torch.arange(most, device="cuda", dtype=torch.int32)
    jump = torch.rand((batch, tree), generator=g, device="cuda")
    node = torch.arange(tree, device="cuda")
    jump = torch.where(node >= count[:, None], jump, 2.0)
    tail = jump.argsort(-1)[:, :most]
    have = (tree - count)[:, None]
    want = (count - head)[:, None]
    tail = torch.where((col < want) & (col < have), tail, tree + 1).sort(-1).values
    at = (col - head[:, None]).clamp(min=0)
    path = torch.where(col < head[:, None], col, tail.gather(1, at.long())).int()
    count = torch.where((path < tree) & (col < count[:, None]), 1, 0).cumprod(1).sum(1).int()
    path = torch.where(col < count[:, None], path, -1).int().contiguous()
    return dict(d, tree=tree, lens=lens, table=table, pool=pool, path=path, count=count,
                lens_out=torch.empty_like(lens))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"tables": _prepare_tables, "masks": _prepare_masks, "append": _prepare_append,
         "tree": _prepare_tree, "commit": _prepare_commit}[case["op"]](case, g)
    s["op"] = case["op"]
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------------- one pass

def _config(s):
    import mla_latent_kv_44_b200 as mla

    return mla.Config(num_heads=s.get("heads", 16), head_dim=s.get("dh", 64),
                      kv_rank=s.get("r", 64), rope_dim=s.get("dr", 32), block_size=s["bs"],
                      dtype="bf16" if s.get("dt") == torch.bfloat16 else "f32")


def _own(s):
    import mla_latent_kv_44_b200 as mla

    op = s["op"]
    if "bs" in s and "cfg" not in s:
        s["cfg"] = _config(s)
    if op == "tables":
        mla.build_tables(s["cfg"], s["lens"], s["new"], s["table"], s["held"], s["free"],
                         s["count"], s["held_out"], s["count_out"], s["cu"], s["seq"], s["pos"],
                         s["slots"], s["err"])
        return [s[k] for k in ("table", "held_out", "free", "count_out", "cu", "seq", "pos",
                               "slots")]
    if op == "masks":
        mla.tree_masks(s["parents"], s["lens"], s["mask"], s["pos"], s["err"])
        return [s["mask"], s["pos"]]
    if op == "append":
        mla.append_slots(s["cfg"], s["ckv"], s["kr"], s["gamma"], s["pos"], s["slots"],
                         s["pool"], s["err"])
        return [s["pool"]]
    if op == "tree":
        if "ws" not in s:
            s["ws"] = torch.empty(mla.decode_tree_workspace_size(s["cfg"], s["lens"].numel(),
                                                                 s["tree"]),
                                  dtype=torch.uint8, device="cuda")
        mla.decode_tree(s["cfg"], s["q"], s["pool"], s["table"], s["lens"], s["tree"], s["mask"],
                        s["w_uv"], s["ws"], s["o"], s["lse"], s["err"])
        return [s["o"], s["lse"]]
    mla.commit_tree(s["cfg"], s["path"], s["count"], s["tree"], s["table"], s["pool"], s["lens"],
                    s["lens_out"], s["err"])
    return [s["pool"], s["lens_out"]]


def _plain_tables(s):
    bs, lens, new, held, table, free = (s[k] for k in ("bs", "lens", "new", "held", "table",
                                                       "free"))
    want = (lens + bs - 1) // bs
    back, grow = (held - want).clamp(min=0), (want - held).clamp(min=0)
    col = torch.arange(table.shape[1], device="cuda")
    end = free.numel()
    # blocks given back go on the free stack in order
    to = s["count"] + (back.cumsum(0) - back)[:, None] + (col - want[:, None])
    gone = (col >= want[:, None]) & (col < held[:, None])
    stack = torch.cat([free, free[:1]])
    stack[torch.where(gone, to, end).flatten().long()] = table.flatten()
    count = s["count"] + back.sum()
    # blocks taken come off its top, whole sequences first come first served
    taken = grow.cumsum(0)
    served = (grow == 0) | (taken <= count)
    k = (taken - grow)[:, None] + (col - held[:, None])
    due = (col >= held[:, None]) & (col < want[:, None]) & served[:, None]
    table = torch.where(due, stack[(count - 1 - k).clamp(0, end - 1).long()], table)
    held_out = torch.where(served, want, held).int()
    count_out = (count - (grow * served).sum()).int()
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)]).int()
    i = torch.arange(s["seq"].numel(), device="cuda", dtype=torch.int32)
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True).clamp(max=lens.numel() - 1)
    real = i < cu[-1]
    pos = torch.where(real, (lens - new - cu[:-1])[b] + i, 0).int()
    slot = table[b, (pos // bs).long()].long() * bs + pos % bs
    return [table, held_out, stack[:-1], count_out, cu, torch.where(real, b, -1).int(), pos,
            torch.where(real & served[b], slot, -1)]


def _plain_masks(s):
    reach = _ancestors(s["parents"])
    pos = (s["lens"] - s["tree"])[:, None] + reach.sum(-1) - 1
    return [_words(reach), pos.flatten().int()]


def _plain_append(s):
    x = s["ckv"].float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["gamma"]
    i = torch.arange(s["dr"] // 2, device="cuda", dtype=torch.float64)
    angle = s["pos"].double()[:, None] * 10000.0 ** (-2.0 * i / s["dr"])
    c, sn = angle.cos(), angle.sin()
    k = s["kr"].double()
    turned = torch.stack([k[:, 0::2] * c - k[:, 1::2] * sn, k[:, 0::2] * sn + k[:, 1::2] * c], -1)
    row = torch.cat([y, turned.flatten(1).float()], -1).to(s["dt"])
    s["flat"][torch.where(s["slots"] < 0, s["flat"].shape[0] - 1, s["slots"])] = row
    return [s["pool"]]


def _plain_tree(s):
    batch, tree, H, r = s["lens"].numel(), s["tree"], s["heads"], s["r"]
    rows = s["pool"][s["table"].long()].float().flatten(1, 2)
    L = rows.shape[1]
    q = s["q"].float().view(batch, tree * H, -1)
    score = torch.matmul(q, rows.transpose(1, 2)).view(batch, tree, H, L) * s["scale"]
    j = torch.arange(L, device="cuda")
    node = j - (s["lens"] - tree)[:, None]
    word = s["mask"].view(batch, tree, -1).long()
    in_tree = (node >= 0) & (node < tree)
    at = node.clamp(0, tree - 1)
    bit = word.gather(2, (at // 32)[:, None].expand(-1, tree, -1)) >> (at % 32)[:, None] & 1
    seen = (node < 0)[:, None] | (in_tree[:, None] & (bit == 1))
    score = torch.where(seen[:, :, None], score, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top)
    del score
    total = p.sum(-1, keepdim=True)
    lat = torch.matmul(p.view(batch, tree * H, L), rows[..., :r])
    lat = (lat.view(batch * tree, H, r) / total.view(batch * tree, H, 1).clamp(min=1e-30))
    o = torch.matmul(lat.transpose(0, 1), s["w_uv"].float().transpose(1, 2)).transpose(0, 1)
    lse = (top + total.log()).view(batch * tree, H)
    return [o.to(s["dt"]).contiguous(), lse]


def _plain_commit(s):
    batch, bs, tree = s["lens"].numel(), s["bs"], s["tree"]
    flat = s["pool"].view(-1, s["pool"].shape[-1])
    first = (s["lens"] - tree)[:, None]
    d = torch.arange(s["path"].shape[1], device="cuda")
    real = d < s["count"][:, None]
    b = torch.arange(batch, device="cuda")[:, None]
    most = s["table"].shape[1] * bs - 1

    def slot(row):
        row = row.clamp(0, most).long()
        return s["table"][b, row // bs].long() * bs + row % bs

    # rows that are not accepted stay: each of those writes itself where it is
    own_row = slot(first + d)
    moved = flat[torch.where(real, slot(first + s["path"]), own_row)]
    keep = (first + d) <= most
    to = torch.where(keep, own_row, own_row[:, :1])
    flat[to] = torch.where(keep[..., None], moved, moved[:, :1])
    return [s["pool"], (s["lens"] - tree + s["count"]).int()]


def run(s):
    if own:
        return _own(s)
    return {"tables": _plain_tables, "masks": _plain_masks, "append": _plain_append,
            "tree": _plain_tree, "commit": _plain_commit}[s["op"]](s)


# ------------------------------------------------------------------------ what a pass is worth

def work(case):
    op = case["op"]
    if op == "tables":
        tokens = case["tokens"]
        # lengths, counts and offsets per request; a block id per 64 tokens in and out; a token's
        # sequence, position and slot out
        return {"bytes": 20 * case["batch"] + 8 * (tokens // 64 + 1) + 16 * tokens, "flops": 0}
    if op == "masks":
        n = case["batch"] * case["tree"]
        return {"bytes": 4 * case["batch"] + n * (4 + 4 + 4 * ((case["tree"] + 31) // 32)),
                "flops": 0}
    d = _dims(case)
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "append":
        n = case["tokens"]
        return {"bytes": n * (2 * d["D"] * size + 12) + 4 * d["r"],
                "flops": n * (4 * d["r"] + 6 * d["dr"])}
    if op == "commit":
        moved = max(1, min(16, case["tree"] // 2)) / 4  # on average, without those in place
        return {"bytes": case["batch"] * (moved * 2 * d["D"] * size + 16), "flops": 0}
    n, H = case["batch"] * case["tree"], case["heads"]
    rows = case["batch"] * (case["cached"] / 2 if case["ragged"] else case["cached"])
    return {"bytes": rows * d["D"] * size + n * H * (d["D"] + d["dh"]) * size
            + H * d["dh"] * d["r"] * size + 4 * n * H,
            "flops": 2.0 * rows * case["tree"] * H * (d["D"] + d["r"])
            + 2.0 * n * H * d["r"] * d["dh"]}


# ------------------------------------------------------------------------------- in 64 bits

def _exact_tables(s):
    bs = s["bs"]
    lens, new, held = (s[k].tolist() for k in ("lens", "new", "held"))
    table, free, n = s["table"].tolist(), s["free"].tolist(), int(s["count"])
    for b, row in enumerate(table):
        for i in range(-(-lens[b] // bs), held[b]):
            free[n] = row[i]
            n += 1
    full, got, out = False, [], list(held)
    for b, row in enumerate(table):
        due = -(-lens[b] // bs) - held[b]
        full = full or due > n
        got.append(due <= 0 or not full)
        if got[-1]:
            out[b] = held[b] + due
            for i in range(held[b], out[b]):
                n -= 1
                row[i] = free[n]
    cu, seq, pos, slots = [0], [], [], []
    for b, row in enumerate(table):
        cu.append(cu[-1] + new[b])
        for p in range(lens[b] - new[b], lens[b]):
            seq.append(b)
            pos.append(p)
            slots.append(row[p // bs] * bs + p % bs if got[b] else -1)
    pad = s["seq"].numel() - len(seq)
    i32 = dict(dtype=torch.int32)
    return [torch.tensor(table, **i32), torch.tensor(out, **i32), torch.tensor(free, **i32),
            torch.tensor([n], **i32), torch.tensor(cu, **i32),
            torch.tensor(seq + [-1] * pad, **i32), torch.tensor(pos + [0] * pad, **i32),
            torch.tensor(slots + [-1] * pad)]


def _exact_masks(s):
    words, pos = [], []
    for b, parents in enumerate(s["parents"].tolist()):
        seen = []
        for t, p in enumerate(parents):
            seen.append((seen[p] if p >= 0 else 0) | 1 << t)
            for w in range((s["tree"] + 31) // 32):
                v = seen[t] >> 32 * w & 0xffffffff
                words.append(v - (1 << 32) if v >> 31 else v)
            pos.append(int(s["lens"][b]) - s["tree"] + bin(seen[t]).count("1") - 1)
    n = (s["tree"] + 31) // 32
    return [torch.tensor(words, dtype=torch.int32).view(-1, n),
            torch.tensor(pos, dtype=torch.int32)]


def _exact_append(s):
    pool = s["pool"].double().view(-1, s["D"])
    x, k = s["ckv"].double(), s["kr"].double()
    norm = x / (x.pow(2).sum(1) / s["r"] + 1e-6).sqrt()[:, None] * s["gamma"].double()
    pair = torch.view_as_complex(k.view(len(k), -1, 2))
    freq = torch.tensor([10000.0 ** (-2 * i / s["dr"]) for i in range(s["dr"] // 2)],
                        dtype=torch.float64, device="cuda")
    angle = s["pos"].double()[:, None] * freq
    turned = torch.view_as_real(pair * torch.polar(torch.ones_like(angle), angle)).flatten(1)
    at = (s["slots"] >= 0).nonzero()[:, 0]
    pool[s["slots"][at]] = torch.cat([norm, turned], 1)[at]
    return [pool.view(s["pool"].shape)]


def _exact_tree(s):
    H, tree, r = s["heads"], s["tree"], s["r"]
    w_uv = s["w_uv"].double()
    os, lses = [], []
    for b, L in enumerate(s["lens"].tolist()):
        rows = s["pool"][s["table"][b].long()].double().view(-1, s["D"])[:L]
        q = s["q"][b * tree: (b + 1) * tree].double()
        score = torch.einsum("thd,jd->thj", q, rows) * s["scale"]
        words = s["mask"][b * tree: (b + 1) * tree].tolist()
        seen = torch.tensor([[w[j // 32] >> j % 32 & 1 for j in range(tree)] for w in words],
                            dtype=torch.bool, device="cuda")
        score[:, :, L - tree:].masked_fill_(~seen[:, None], -math.inf)
        lse = score.logsumexp(-1)
        lat = torch.einsum("thj,jr->thr", (score - lse[..., None]).exp_(), rows[:, :r])
        os.append(torch.einsum("thr,hvr->thv", lat, w_uv))
        lses.append(lse)
    return [torch.cat(os), torch.cat(lses)]


def _exact_commit(s):
    pool = s["pool"].double()
    flat, was = pool.view(-1, s["D"]), s["pool"].double().view(-1, s["D"])
    table, bs = s["table"].tolist(), s["bs"]
    to, come = [], []
    for b, (L, n) in enumerate(zip(s["lens"].tolist(), s["count"].tolist())):
        for d, a in enumerate(s["path"][b, :n].tolist()):
            for row, out in ((L - s["tree"] + d, to), (L - s["tree"] + a, come)):
                out.append(table[b][row // bs] * bs + row % bs)
    flat[torch.tensor(to, device="cuda", dtype=torch.long)] = was[
        torch.tensor(come, device="cuda", dtype=torch.long)]
    return [pool, (s["lens"] - s["tree"] + s["count"]).int()]


def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "masks": _exact_masks, "append": _exact_append,
            "tree": _exact_tree, "commit": _exact_commit}[s["op"]](s)
