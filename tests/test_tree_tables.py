"""mla_build_tables, mla_tree_masks, mla_append_slots and mla_commit_tree against plain forms, and the
refusals of all tree calls."""
import copy
import ctypes
import math
import pickle

import pytest
import torch

from tests import tree_util as tu

GPU = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    from mla_latent_kv_44_b200 import build

    build.build()
    import mla_latent_kv_44_b200 as m

    return m


# ------------------------------------------------------------------------------------- refusals

def _ref(mla, **kw):
    base = dict(num_heads=128, head_dim=128, kv_rank=512, rope_dim=64, block_size=64)
    base.update(kw)
    return mla.Config(**base).ref()


A, ODD = 4096, 4104  # an aligned and a misaligned address; no call here gets as far as using one


def _tables(mla, cfg, **kw):
    a = dict(lens=A, new=A, batch=2, table=A, width=4, held=A, free=A, count=A, blocks=8, held_out=A,
             count_out=A, cu=A, seq=A, pos=A, slots=A, tokens=4, err=A)
    a.update(kw)
    return mla.lib.mla_build_tables(cfg, *a.values(), None)


def test_build_tables_refusals(mla):
    c = _ref(mla)
    for name in ("lens", "new", "table", "held", "free", "count", "held_out", "count_out", "cu", "seq",
                 "pos", "slots", "err"):
        assert _tables(mla, c, **{name: None}) == mla.MLA_ERR_INVALID_ARG, name
    for kw in (dict(batch=-1), dict(tokens=-1), dict(width=0), dict(blocks=0)):
        assert _tables(mla, c, **kw) == mla.MLA_ERR_INVALID_ARG, kw
    assert _tables(mla, None) == mla.MLA_ERR_INVALID_ARG
    for kw in (dict(batch=mla.MAX_TABLE_BATCH + 1), dict(tokens=(1 << 26) + 1),
               dict(batch=4096, width=(1 << 18) + 1)):
        assert _tables(mla, c, **kw) == mla.MLA_ERR_UNSUPPORTED, kw
    assert _tables(mla, c, batch=0) == mla.MLA_OK


def test_tree_masks_refusals(mla):
    f = mla.lib.mla_tree_masks
    good = [A, 2, A, 2, 4, A, A, A]
    for i in (0, 2, 5, 6, 7):
        assert f(*good[:i], None, *good[i + 1:], None) == mla.MLA_ERR_INVALID_ARG, i
    assert f(A, 3, A, 2, 4, A, A, A, None) == mla.MLA_ERR_INVALID_ARG
    assert f(A, 2, A, -1, 4, A, A, A, None) == mla.MLA_ERR_INVALID_ARG
    assert f(A, 2, A, 2, 0, A, A, A, None) == mla.MLA_ERR_INVALID_ARG
    assert f(A, 2, A, 2, mla.MAX_TREE + 1, A, A, A, None) == mla.MLA_ERR_UNSUPPORTED
    assert f(A, 2, A, 0, 4, A, A, A, None) == mla.MLA_OK


def test_append_slots_refusals(mla):
    c, f = _ref(mla), mla.lib.mla_append_slots
    good = [A, A, A, A, A, A, 8, 4, A]
    for i in (0, 1, 2, 3, 4, 5, 8):
        assert f(c, *good[:i], None, *good[i + 1:], None) == mla.MLA_ERR_INVALID_ARG, i
    for i in (0, 2, 5):
        assert f(c, *good[:i], ODD, *good[i + 1:], None) == mla.MLA_ERR_INVALID_ARG, i
    assert f(c, A, A, A, A, A, A, 0, 4, A, None) == mla.MLA_ERR_INVALID_ARG
    assert f(c, A, A, A, A, A, A, 8, -1, A, None) == mla.MLA_ERR_INVALID_ARG
    assert f(c, A, A, A, A, A, A, 8, (1 << 26) + 1, A, None) == mla.MLA_ERR_UNSUPPORTED
    assert f(c, A, A, A, A, A, A, 8, 0, A, None) == mla.MLA_OK


def _tree(mla, cfg, **kw):
    a = dict(q=A, pool=A, table=A, width=4, blocks=8, lens=A, batch=2, T=4, mask=A, w_uv=A, ws=A,
             size=1 << 40, o=A, lse=A, err=A)
    a.update(kw)
    return mla.lib.mla_decode_tree(cfg, *a.values(), None)


def test_decode_tree_refusals(mla):
    c = _ref(mla)
    for name in ("q", "pool", "table", "lens", "w_uv", "ws", "o", "err"):
        assert _tree(mla, c, **{name: None}) == mla.MLA_ERR_INVALID_ARG, name
    for name in ("q", "pool", "w_uv", "o"):
        assert _tree(mla, c, **{name: ODD}) == mla.MLA_ERR_INVALID_ARG, name
    for kw in (dict(batch=-1), dict(T=0), dict(width=0), dict(blocks=0)):
        assert _tree(mla, c, **kw) == mla.MLA_ERR_INVALID_ARG, kw
    assert _tree(mla, c, T=mla.MAX_TREE + 1) == mla.MLA_ERR_UNSUPPORTED
    need = mla.lib.mla_decode_tree_workspace_size(c, 2, 4)
    assert need > 0 and need % 256 == 0
    assert _tree(mla, c, size=need - 1) == mla.MLA_ERR_WORKSPACE
    assert _tree(mla, c, ws=ODD) == mla.MLA_ERR_WORKSPACE
    # tensor-core kernels only: another rank or fp32 has none
    for kw in (dict(kv_rank=256), dict(dtype="f32"), dict(block_size=96)):
        odd = _ref(mla, decode_kernel=mla.DECODE_TENSOR, **kw)
        assert _tree(mla, odd) == mla.MLA_ERR_UNSUPPORTED, kw
    assert _tree(mla, c, batch=0) == mla.MLA_OK


def test_decode_tree_refuses_what_32_bits_cannot_number(mla):
    """The tensor-core kernel's pool rows and 64-row pieces; the CUDA cores' are 64-bit."""
    c, size = _ref(mla), 1 << 40
    assert _tree(mla, c, blocks=1 << 25, size=size) == mla.MLA_ERR_UNSUPPORTED  # 2^31 rows
    assert _tree(mla, c, batch=1 << 16, width=1 << 15, size=size) == mla.MLA_ERR_UNSUPPORTED
    assert _tree(mla, c, T=1, batch=1 << 24, width=128, size=size) == mla.MLA_ERR_UNSUPPORTED
    # heads and tokens: 2^28 query rows at most
    assert _tree(mla, c, T=256, batch=(1 << 13) + 1, size=size) == mla.MLA_ERR_UNSUPPORTED
    # one below the limits: refused for its workspace only
    for kw in (dict(blocks=(1 << 25) - 1), dict(batch=1 << 16, width=(1 << 15) - 1)):
        assert _tree(mla, c, size=0, **kw) == mla.MLA_ERR_WORKSPACE, kw


def test_commit_tree_refusals(mla):
    c, f = _ref(mla), mla.lib.mla_commit_tree
    good = [A, A, 4, 4, A, 4, A, 8, A, A, 2, A]
    for i in (0, 1, 4, 6, 8, 9, 11):
        assert f(c, *good[:i], None, *good[i + 1:], None) == mla.MLA_ERR_INVALID_ARG, i
    for i, v in ((2, 0), (3, 0), (5, 0), (7, 0), (10, -1), (6, ODD)):
        assert f(c, *good[:i], v, *good[i + 1:], None) == mla.MLA_ERR_INVALID_ARG, i
    assert f(c, A, A, 4, mla.MAX_TREE + 1, *good[4:], None) == mla.MLA_ERR_UNSUPPORTED
    assert f(c, *good[:10], 0, A, None) == mla.MLA_OK


def test_workspace_sizes_are_host_arithmetic(mla):
    size = mla.lib.mla_decode_tree_workspace_size
    c = _ref(mla)
    assert size(c, 0, 4) == 0 and size(c, 1, 0) == 0 and size(c, 1, mla.MAX_TREE + 1) == 0
    assert size(None, 1, 4) == 0
    # two bf16 terms of every latent sum, and the partial results
    n = 32 * 4 * 128 * 512
    assert size(c, 32, 4) >= 4 * n + 148 * 128 * 512 * 4
    f32 = _ref(mla, num_heads=16, head_dim=64, kv_rank=64, rope_dim=32, dtype="f32")
    assert size(f32, 8, 5) >= 8 * 5 * 16 * 64 * 4


@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c))],
                         ids=["copy", "deepcopy", "pickle"])
def test_a_used_config_copies_and_pickles(mla, again):
    cfg = mla.Config(16, 64, 64, 32, 64)
    at = cfg.address()
    other = again(cfg)
    assert other == cfg and other.address() != at and cfg.address() == at
    other.num_heads = 8
    assert mla.MlaConfig.from_address(other.address()).num_heads == 8
    cfg.num_heads = 4  # the first struct stays as it was, and where it was
    assert mla.MlaConfig.from_address(cfg.address()).num_heads == 4
    assert mla.MlaConfig.from_address(at).num_heads == 16
    cfg.num_heads = 16
    assert cfg.address() == at


def test_binding_refuses_what_a_pointer_cannot_carry(mla):
    cfg = mla.Config(16, 64, 64, 32, 64, dtype="f32")
    i32 = torch.int32
    cpu = [torch.zeros(1, 4, dtype=i32), torch.zeros(1, dtype=i32), torch.zeros(4, 1, dtype=i32),
           torch.zeros(4, dtype=i32), torch.zeros(1, dtype=i32)]
    with pytest.raises(mla.MlaError, match="not on a GPU"):
        mla.tree_masks(*cpu)
    with pytest.raises(mla.MlaError, match="dimensions"):
        mla.tree_masks(torch.zeros(4, dtype=i32), *cpu[1:])
    pool = torch.zeros(2, 64, 96)
    with pytest.raises(mla.MlaError, match="not on a GPU"):
        mla.append_slots(cfg, torch.zeros(3, 64), torch.zeros(3, 32), torch.ones(64),
                         torch.zeros(3, dtype=i32), torch.zeros(3, dtype=torch.int64), pool,
                         torch.zeros(1, dtype=i32))


@GPU
def test_binding_names_the_wrong_tensor(mla):
    i32, d = torch.int32, "cuda"
    parents, lens = torch.zeros(2, 4, dtype=i32, device=d), torch.full((2,), 9, dtype=i32, device=d)
    mask, pos = torch.zeros(8, 1, dtype=i32, device=d), torch.zeros(8, dtype=i32, device=d)
    err = torch.zeros(1, dtype=i32, device=d)
    for args, name in (((parents.long(), lens, mask, pos, err), "parents"),
                       ((parents, lens, mask[:7], pos, err), "mask"),
                       ((parents, lens, mask, pos.repeat_interleave(2)[::2], err), "pos"),
                       ((parents, lens.cpu(), mask, pos, err), "seq_lens")):
        with pytest.raises(mla.MlaError, match=name):
            mla.tree_masks(*args)


@GPU
def test_binding_takes_no_number_modulo_2_to_32(mla):
    i32, d = torch.int32, "cuda"
    cfg = mla.Config(16, 64, 64, 32, 64, dtype="f32")
    pool, table = torch.zeros(2, 64, 96, device=d), torch.zeros(1, 1, dtype=i32, device=d)
    path, one = torch.zeros(1, 4, dtype=i32, device=d), torch.ones(1, dtype=i32, device=d)
    lens, out = torch.full((1,), 9, dtype=i32, device=d), torch.full((1,), -7, dtype=i32, device=d)
    for T in (2 ** 32 + 4, -2 ** 32 + 4):
        with pytest.raises(mla.MlaError):
            mla.commit_tree(cfg, path, one, T, table, pool, lens, out, torch.zeros_like(one))
    with pytest.raises((TypeError, OverflowError)):
        mla.commit_tree(cfg, path, one, 4.0, table, pool, lens, out, torch.zeros_like(one))
    torch.cuda.synchronize()
    assert int(out) == -7


# --------------------------------------------------------------------------------- build_tables

def _run_tables(mla, bs, lens, new, table, held, free, count, tokens, in_place=False, odd=False):
    d, i32 = "cuda", torch.int32
    cfg = mla.Config(16, 64, 64, 32, bs)
    t = [torch.tensor(x, dtype=i32, device=d) for x in (lens, new, table, held, free, [count])]
    held_out = t[3] if in_place else torch.full((len(lens),), -7, dtype=i32, device=d)
    count_out = t[5] if in_place else torch.full((1,), -7, dtype=i32, device=d)
    cu = torch.full((len(lens) + 1,), -7, dtype=i32, device=d)
    off = 1 if odd else 0  # outputs that are not 16-byte aligned
    seq, pos = (torch.full((tokens + off,), -7, dtype=i32, device=d)[off:] for _ in range(2))
    slots = torch.full((tokens + off,), -7, dtype=torch.int64, device=d)[off:]
    err = torch.zeros(1, dtype=i32, device=d)
    mla.build_tables(cfg, t[0], t[1], t[2], t[3], t[4], t[5], held_out, count_out, cu, seq, pos,
                     slots, err)
    torch.cuda.synchronize()
    got = (t[2].tolist(), held_out.tolist(), t[4].tolist(), int(count_out), cu.tolist(),
           seq.tolist(), pos.tolist(), slots.tolist(), int(err))
    want = tu.tables(bs, lens, new, table, held, free, count, len(free), tokens)
    for name, g, w in zip(("table", "held", "free", "count", "cu", "seq", "pos", "slots", "err"),
                          got, want):
        assert g == w, name


def _requests(seed, batch, width, bs, spare, growth=8):
    """Running, new and ended requests with blocks anywhere in the pool."""
    g = torch.Generator().manual_seed(seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    lens, new, held, used = [], [], [], 0
    for _ in range(batch):
        kind = r(0, 3)
        n = r(1, width * bs)
        m = n if kind == 0 else 0 if kind == 1 else min(n, r(0, growth))
        held.append(0 if kind == 0 else r(0, width) if kind == 1 else -(-(n - m) // bs))
        lens.append(0 if kind == 1 else n)
        new.append(m)
    total = sum(held) + spare
    ids = torch.randperm(total, generator=g).tolist()
    table = []
    for h in held:
        table.append(ids[used:used + h] + [-1] * (width - h))
        used += h
    return lens, new, table, held, ids[used:] + [-1] * used, total - used


@GPU
@pytest.mark.parametrize("batch,width,bs,spare,tokens,seed", [
    (1, 1, 1, 1, 1, 0), (1, 3, 64, 3, 200, 1), (5, 4, 16, 30, 64, 2), (7, 5, 24, 40, 1000, 3),
    (64, 9, 64, 600, 40000, 4), (33, 7, 1, 300, 5, 5), (130, 3, 8, 2, 700, 6),
    (1500, 2, 4, 4000, 9001, 7), (3, 4, 64, 0, 300, 8), (40, 6, 32, 90, 0, 9)])
@pytest.mark.parametrize("in_place,odd", [(False, False), (True, True)])
def test_tables_match_the_plain_form(mla, batch, width, bs, spare, tokens, seed, in_place, odd):
    args = _requests(seed, batch, width, bs, spare)
    _run_tables(mla, bs, *args, tokens, in_place, odd)


@GPU
@pytest.mark.parametrize("batch,width,bs,spare,tokens,seed", [
    (512, 2, 8, 900, 512, 11), (512, 2, 8, 900, 513, 12), (300, 2, 8, 500, 2048, 13),
    (513, 2, 8, 900, 2049, 14), (1024, 3, 4, 2500, 4096, 15), (1025, 2, 4, 2000, 4097, 16),
    (700, 2, 16, 1200, 33000, 17), (1100, 2, 16, 1200, 33000, 18), (8192, 2, 4, 15000, 32768, 19),
    (600, 2, 4, 100, 3000, 20)])
def test_tables_at_the_sizes_where_the_launch_changes(mla, batch, width, bs, spare, tokens, seed):
    lens, new, table, held, free, count = _requests(seed, batch, width, bs, spare)
    _run_tables(mla, bs, lens, new, table, held, free, count, tokens, in_place=seed % 2 == 0)


@GPU
@pytest.mark.parametrize("batch,T,bs,tokens", [(4, 6, 64, 24), (4, 6, 64, 40), (9, 4, 16, 36),
                                               (300, 8, 8, 2400), (1200, 5, 16, 6000),
                                               (500, 70, 64, 35000), (7, 3, 1, 20)])
@pytest.mark.parametrize("full", [True, False])
def test_tables_of_a_padded_batch(mla, batch, T, bs, tokens, full):
    """T tokens for every place, the empty ones too: token t of request b is b * T + t."""
    g = torch.Generator().manual_seed(batch + T)
    width = -(-400 // bs)
    lens = torch.randint(T, 400, (batch,), generator=g)
    lens[torch.rand(batch, generator=g) < 0.4] = 0
    lens[0] = 0
    held = [int(h) for h in torch.randint(0, 2, (batch,), generator=g)]
    need = int(((lens + bs - 1) // bs).sum()) // (1 if full else 2)
    total = need + sum(held) + 1
    ids = torch.randperm(total, generator=g).tolist()
    table = [[ids.pop() if i < h else -1 for i in range(width)] for h in held]
    count = len(ids)
    _run_tables(mla, bs, lens.tolist(), [T] * batch, table, held, ids + [-1] * (total - count), count,
                tokens)


@GPU
def test_tables_of_bad_input(mla):
    table = [[0, 1, -1], [2, -1, -1], [3, 4, 5]]
    good = dict(lens=[130, 64, 192], new=[3, 1, 0], held=[2, 1, 3], free=[6, 7, -1, -1, -1, -1, -1, -1],
                count=2)
    for kw in (dict(lens=[-1, 64, 192]), dict(lens=[193, 64, 192]), dict(new=[3, 65, 0]),
               dict(new=[-1, 1, 0]), dict(held=[2, 4, 3]), dict(held=[-1, 1, 3]), dict(count=-1),
               dict(count=9), dict(free=[6, 99, -1, -1, -1, -1, -1, -1]),
               dict(free=[6, -5, -1, -1, -1, -1, -1, -1]), dict(lens=[130, 64, 0], count=7),
               dict(count=0), dict(lens=[130, 128, 64], count=0)):
        a = dict(good, **kw)
        _run_tables(mla, 64, a["lens"], a["new"], table, a["held"], a["free"], a["count"], 6)
    _run_tables(mla, 64, [130, 64, 64], [3, 1, 1], [[0, 1, 2], [77, -1, -1], [-3, 4, 5]], [3, 1, 3],
                [6, 7, 8, 9, -1, -1, -1, -1], 4, 8)


@GPU
def test_tables_of_very_many_new_rows(mla):
    """New rows whose count passes 32 bits: the first max_tokens of them are right."""
    n, width, bs = 6000, 2, 1 << 20
    lens = [2 << 20] * n
    table = torch.arange(2 * n).view(n, 2).tolist()
    d, i32 = "cuda", torch.int32
    cfg = mla.Config(16, 64, 64, 32, bs)
    t = lambda x: torch.tensor(x, dtype=i32, device=d)  # noqa: E731
    tokens = (1 << 21) + 5
    cu, seq, pos = t([0] * (n + 1)), t([0] * tokens), t([0] * tokens)
    slots, err = torch.zeros(tokens, dtype=torch.int64, device=d), t([0])
    held = t([2] * n)
    mla.build_tables(cfg, t(lens), t(lens), t(table), held, t([-1] * (2 * n)), t([0]), held, t([0]), cu,
                     seq, pos, slots, err)
    assert int(err) == mla.DEV_BAD_LENGTH
    i = torch.arange(tokens)
    assert torch.equal(seq.cpu(), (i >> 21).int())
    assert torch.equal(pos.cpu(), (i & ((1 << 21) - 1)).int())
    assert torch.equal(slots.cpu(), i)
    assert cu.tolist() == [min(k << 21, tokens) for k in range(n + 1)]


# ----------------------------------------------------------------------------------- tree_masks

@GPU
@pytest.mark.parametrize("batch,T,kind", [(1, 1, "star"), (3, 4, "chain"), (5, 7, "random"),
                                          (2, 31, "random"), (4, 32, "chain"), (2, 33, "random"),
                                          (3, 64, "random"), (2, 65, "star"), (2, 128, "random"),
                                          (1, 129, "chain"), (2, 256, "chain"), (3, 256, "random"),
                                          (300, 5, "random")])
@pytest.mark.parametrize("shared", [False, True])
def test_masks_and_positions(mla, batch, T, kind, shared):
    d, i32 = "cuda", torch.int32
    parents = tu.parents_of(kind, 1 if shared else batch, T, seed=T)
    lens = torch.randint(T, 70000, (batch,), generator=torch.Generator().manual_seed(1), dtype=i32)
    lens[0] = T
    if batch > 2:
        lens[1] = 0  # an empty place
    mask = torch.full((batch * T, (T + 31) // 32), -7, dtype=i32, device=d)
    pos, err = torch.full((batch * T,), -7, dtype=i32, device=d), torch.zeros(1, dtype=i32, device=d)
    mla.tree_masks(parents.to(d), lens.to(d), mask, pos, err)
    seen = tu.seen_of(parents).expand(batch, T, T)
    assert int(err) == 0
    assert torch.equal(mask.cpu(), tu.words_of(seen))
    want = (lens[:, None] - T) + seen.sum(-1).int() - 1
    want[lens == 0] = 0
    assert torch.equal(pos.cpu().view(batch, T), want.int())


@GPU
def test_masks_of_bad_trees(mla):
    d, i32 = "cuda", torch.int32
    for bad in ([-2, 0, 1, 2], [0, 0, 1, 2], [-1, 0, 3, 2], [-1, 0, 1, 7]):
        mask = torch.zeros(4, 1, dtype=i32, device=d)
        pos, err = torch.zeros(4, dtype=i32, device=d), torch.zeros(1, dtype=i32, device=d)
        mla.tree_masks(torch.tensor([bad], dtype=i32, device=d),
                       torch.tensor([10], dtype=i32, device=d), mask, pos, err)
        mended = [[p if -1 <= p < t else -1 for t, p in enumerate(bad)]]
        assert int(err) == mla.DEV_BAD_TREE
        assert torch.equal(mask.cpu(), tu.words_of(tu.seen_of(torch.tensor(mended))))
    err.zero_()
    mla.tree_masks(torch.tensor([[-1, 0, 1, 2]], dtype=i32, device=d),
                   torch.tensor([3], dtype=i32, device=d), mask, pos, err)
    assert int(err) == mla.DEV_BAD_LENGTH and pos.tolist() == [0] * 4


# --------------------------------------------------------------------------------- append_slots

def _row(ckv, kr, gamma, pos, base=10000.0, eps=1e-6):
    """The rows in 64 bits, and what their values' rounding errors are relative to."""
    x, k = ckv.double(), kr.double()
    norm = x / (x.pow(2).mean(1, keepdim=True) + eps).sqrt() * gamma.double()
    dr = kr.shape[1]
    theta = base ** (-2.0 * torch.arange(dr // 2, dtype=torch.float64) / max(dr, 1))
    a = pos.double()[:, None] * theta
    c, s = a.cos(), a.sin()
    x0, x1 = k[:, 0::2], k[:, 1::2]
    rot = torch.stack([x0 * c - x1 * s, x0 * s + x1 * c], -1).flatten(1)
    size = torch.stack([x0.abs() + x1.abs()] * 2, -1).flatten(1)
    return torch.cat([norm, rot], 1), torch.cat([norm.abs(), size], 1)


@GPU
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("r,dr,bs,n", [(512, 64, 64, 1), (512, 64, 64, 333), (64, 32, 16, 100),
                                       (32, 0, 7, 50), (96, 8, 5, 64), (1024, 256, 3, 40),
                                       (256, 34 + 6, 64, 2000)])
def test_append_by_slots(mla, dtype, r, dr, bs, n):
    d = "cuda"
    cfg = mla.Config(16, 64, r, dr, bs, dtype=dtype)
    dt, g = cfg.torch_dtype, torch.Generator().manual_seed(r + n)
    ckv = torch.randn(n, r, generator=g).to(dt)
    kr = torch.randn(n, dr, generator=g).to(dt)
    gamma = 1 + 0.1 * torch.randn(r, generator=g)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32)
    pos[0] = 0
    blocks = -(-n // bs) + 2
    slots = torch.randperm(blocks * bs, generator=g)[:n]
    slots[n // 3:n // 3 + n // 8] = -1 - torch.arange(n // 8)  # a step's padding
    pool = torch.full((blocks, bs, r + dr), 7.5).to(dt)
    out, err = pool.to(d), torch.zeros(1, dtype=torch.int32, device=d)
    mla.append_slots(cfg, ckv.to(d), kr.to(d) if dr else None, gamma.to(d), pos.to(d), slots.to(d),
                     out, err)
    assert int(err) == 0
    want, size = _row(ckv, kr, gamma, pos)
    # fp32: the mean of squares and its root 2^-20 at most, the angle in fp32 2^-22 of the pair
    tol = 2.0 ** -20 * size + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * want.abs()
    got = out.cpu().view(-1, r + dr).double()
    at = slots >= 0
    assert ((got[slots[at]] - want[at]).abs() <= tol[at]).all()
    rest = torch.ones(blocks * bs, dtype=torch.bool)
    rest[slots[at]] = False
    assert torch.equal(got[rest], torch.full_like(got[rest], 7.5))


@GPU
def test_append_by_slots_equals_append_through_the_table(mla):
    """The same rows by mla_append_latent: equal but for values that round the other way."""
    d, i32 = "cuda", torch.int32
    cfg = mla.Config(128, 128, 512, 64, 64)
    g = torch.Generator().manual_seed(3)
    n, lens, new = 70, [40, 66, 200], [40, 20, 10]
    ckv, kr = torch.randn(n, 512, generator=g).bfloat16().to(d), torch.randn(n, 64, generator=g).bfloat16().to(d)
    gamma = torch.ones(512, device=d)
    t = lambda x: torch.tensor(x, dtype=i32, device=d)  # noqa: E731
    table, held, count = t([[-1] * 4] * 3), t([0, 1, 3]), t([5])
    table[1, 0], table[2, :3] = 9, t([6, 7, 8])
    free = t([0, 1, 2, 3, 4, -1, -1, -1, -1, -1])
    cu, seq, pos = t([0] * 4), t([0] * n), t([0] * n)
    slots, err = torch.zeros(n, dtype=torch.int64, device=d), t([0])
    mla.build_tables(cfg, t(lens), t(new), table, held, free, count, held, count, cu, seq, pos, slots,
                     err)
    assert held.tolist() == [1, 2, 4] and int(count) == 2 and int(err) == 0
    pools = [torch.zeros(10, 64, 576, dtype=torch.bfloat16, device=d) for _ in range(2)]
    mla.append_slots(cfg, ckv, kr, gamma, pos, slots, pools[0], err)
    mla.append_latent(cfg, ckv, kr, gamma, seq, pos, table, pools[1], err)
    assert int(err) == 0
    a, b = (p.double() for p in pools)
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-6).all()  # one step of bf16
    assert float((a != b).double().mean()) < 1e-3
    assert int((a.view(-1, 576).abs().sum(1) > 0).sum()) == n


@GPU
def test_append_slots_outside_the_pool(mla):
    d = "cuda"
    cfg = mla.Config(16, 64, 64, 32, 8, dtype="f32")
    pool = torch.zeros(3, 8, 96, device=d)
    err = torch.zeros(1, dtype=torch.int32, device=d)
    slots = torch.tensor([24, 5, 1 << 40, -(1 << 40)], device=d)
    mla.append_slots(cfg, torch.ones(4, 64, device=d), torch.ones(4, 32, device=d),
                     torch.ones(64, device=d), torch.zeros(4, dtype=torch.int32, device=d), slots, pool,
                     err)
    assert int(err) == mla.DEV_OOB_BLOCK
    assert (pool.view(24, 96).abs().sum(1) > 0).nonzero().flatten().tolist() == [5]


# ---------------------------------------------------------------------------------- commit_tree

def _commit(mla, dtype, bs, T, lens, paths, in_place=False, width=None, seed=0):
    d, i32 = "cuda", torch.int32
    r, dr = 64, 32
    cfg = mla.Config(16, 64, r, dr, bs, dtype=dtype)
    g = torch.Generator().manual_seed(seed)
    B, most = len(lens), max(1, -(-max(lens) // bs))
    table = torch.randperm(B * most + 3, generator=g)[:B * most].view(B, most).int()
    pool = torch.randn(B * most + 3, bs, r + dr, generator=g).to(cfg.torch_dtype)
    width = width or max(1, max(len(p) for p in paths))
    path = torch.full((B, width), -9, dtype=i32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p, dtype=i32)
    count = torch.tensor([len(p) for p in paths], dtype=i32)
    L = torch.tensor(lens, dtype=i32, device=d)
    out = L if in_place else torch.full((B,), -7, dtype=i32, device=d)
    got, err = pool.to(d), torch.zeros(1, dtype=i32, device=d)
    mla.commit_tree(cfg, path.to(d), count.to(d), T, table.to(d), got, L, out, err)
    flat = pool.clone().view(-1, r + dr)
    ends = []
    for b, (n, p) in enumerate(zip(lens, paths)):
        bad = n != 0 and (n < T or len(p) > T or any(not 0 <= a < T for a in p) or
                          any(x >= y for x, y in zip(p, p[1:])))
        ends.append(n if bad or n == 0 else n - T + len(p))
        if bad or n == 0:
            continue
        slot = lambda row: int(table[b, row // bs]) * bs + row % bs  # noqa: E731
        keep = [pool.view(-1, r + dr)[slot(n - T + a)].clone() for a in p]
        for i, row in enumerate(keep):
            flat[slot(n - T + i)] = row
    assert torch.equal(got.cpu().view(-1, r + dr), flat)
    assert out.tolist() == ends
    return int(err)


@GPU
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bs,T,lens,paths", [
    (64, 4, [10, 64, 67, 4], [[0, 1, 3], [], [0, 2], [3]]),
    (4, 16, [16, 33, 21, 0], [[0, 3, 4, 9, 15], [1, 2, 3, 4, 5, 6, 7, 8, 9], [0], [0, 1]]),
    (8, 40, [61, 40], [list(range(40)), list(range(1, 40))]),
    (64, 256, [300], [[5 * i for i in range(50)]]),
    (1, 3, [3, 9], [[0, 2], [2]]),
    (64, 1, [1, 65, 128], [[0], [], [0]])])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit_moves_the_accepted_rows(mla, dtype, bs, T, lens, paths, in_place):
    assert _commit(mla, dtype, bs, T, lens, paths, in_place) == 0


@GPU
def test_commit_of_random_paths(mla):
    g = torch.Generator().manual_seed(7)
    T, B = 64, 200
    lens = (torch.randint(0, 300, (B,), generator=g) + T).tolist()
    paths = [sorted(torch.randperm(T, generator=g)[:int(torch.randint(0, T + 1, (1,), generator=g))].tolist())
             for _ in range(B)]
    assert _commit(mla, "bf16", 16, T, lens, paths) == 0


@GPU
def test_commit_of_bad_paths(mla):
    assert _commit(mla, "f32", 8, 4, [10, 20], [[0, 0], [0, 1]]) == mla.DEV_BAD_TREE
    assert _commit(mla, "f32", 8, 4, [10, 20], [[0, 1], [0, 4]]) == mla.DEV_BAD_TREE
    assert _commit(mla, "f32", 8, 4, [10, 20], [[2, 1], [-1]]) == mla.DEV_BAD_TREE
    assert _commit(mla, "f32", 8, 4, [10, 20], [[0, 1, 2, 3, 5], [0]]) == mla.DEV_BAD_TREE
    assert _commit(mla, "f32", 8, 4, [3, 20], [[0], [0, 3]]) == mla.DEV_BAD_LENGTH
