"""Tree calls at sizes and inputs where they can go wrong apart from their values: limits that a launch
depends on, empty places of a padded batch, calls from two threads."""
import json
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from tests import tree_util as tu
from tests.test_tree_attention import Case

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GPU = pytest.mark.gpu
D_ = "cuda"


@pytest.fixture(scope="module")
def mla():
    from mla_latent_kv_44_b200 import build

    build.build()
    import mla_latent_kv_44_b200 as m

    return m


# ------------------------------------------------------------------------------- build_tables

TABLES = r"""
import json, sys
sys.path.insert(0, ROOT)
import torch
import mla_latent_kv_44_b200 as mla
from tests import tree_util as tu
B, d, i32 = BATCH, "cuda", torch.int32
g = torch.Generator().manual_seed(B)
lens = torch.randint(0, 9, (B,), generator=g).tolist()
held = [int(n > 4) for n in lens]
total = 3 * B
ids = torch.randperm(total, generator=g).tolist()
table = [[ids.pop() if i < h else -1 for i in range(2)] for h in held]
count = len(ids)
free = ids + [-1] * (total - count)
new = [min(n, 1) for n in lens]
t = [torch.tensor(x, dtype=i32, device=d) for x in (lens, new, table, held, free, [count])]
cu, seq, pos = (torch.zeros(n, dtype=i32, device=d) for n in (B + 1, B, B))
slots, err = torch.zeros(B, dtype=torch.int64, device=d), torch.zeros(1, dtype=i32, device=d)
mla.build_tables(mla.Config(16, 64, 64, 32, 4), *t, t[3], t[5], cu, seq, pos, slots, err)
got = [x.tolist() for x in (t[2], t[3], t[4], t[5][0], cu, seq, pos, slots, err[0])]
want = tu.tables(4, lens, new, table, held, free, count, total, B)
print(json.dumps([list(g) == list(w) if isinstance(g, list) else g == w for g, w in zip(got, want)]))
"""


@GPU
@pytest.mark.parametrize("batch", [3046, 3047, 3071, 3080])
def test_tables_where_shared_memory_passes_the_default_limit(batch):
    """In a process of its own: a larger call before would have raised the kernel's limit."""
    out = subprocess.run([sys.executable, "-c",
                          TABLES.replace("ROOT", repr(ROOT)).replace("BATCH", str(batch))],
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert json.loads(out.stdout.splitlines()[-1]) == [True] * 9


# --------------------------------------------------------------------------------- tree_masks

@GPU
@pytest.mark.parametrize("T", [1, 5, 33, 100, 256])
def test_parents_of_an_empty_place_are_not_flagged(mla, T):
    """Unused places of a captured step hold whatever was there: no error, whatever their parents; a
    live place's bad parents are flagged as before."""
    i32, junk = torch.int32, 0x7ADE7ADE
    parents = tu.parents_of("random", 4, T, seed=T)
    parents[1], parents[3] = junk, -junk
    lens = torch.tensor([T + 7, 0, T, 0], dtype=i32)
    mask = torch.full((4 * T, (T + 31) // 32), -7, dtype=i32, device=D_)
    pos, err = torch.full((4 * T,), -7, dtype=i32, device=D_), torch.zeros(1, dtype=i32, device=D_)
    mla.tree_masks(parents.to(D_), lens.to(D_), mask, pos, err)
    assert int(err) == 0
    mended = parents.clone()
    mended[[1, 3]] = -1                                # a bad parent counts as -1
    seen = tu.seen_of(mended)
    assert torch.equal(mask.cpu(), tu.words_of(seen))
    want = lens[:, None] - T + seen.sum(-1).int() - 1
    want[[1, 3]] = 0
    assert torch.equal(pos.cpu().view(4, T), want)
    mla.tree_masks(parents.to(D_), torch.full_like(lens, T).to(D_), mask, pos, err)
    assert int(err) == mla.DEV_BAD_TREE


@GPU
def test_a_shared_tree_is_flagged_only_where_it_is_used(mla):
    i32 = torch.int32
    bad = torch.tensor([[-1, 5, 1]], dtype=i32, device=D_)
    mask, pos = torch.zeros(6, 1, dtype=i32, device=D_), torch.zeros(6, dtype=i32, device=D_)
    for lens, bits in (([0, 0], 0), ([0, 9], mla.DEV_BAD_TREE)):
        err = torch.zeros(1, dtype=i32, device=D_)
        mla.tree_masks(bad, torch.tensor(lens, dtype=i32, device=D_), mask, pos, err)
        assert int(err) == bits


# -------------------------------------------------------------------------------- decode_tree

@GPU
@pytest.mark.parametrize("kw", [dict(r=64, dr=128), dict(r=128, dr=64), dict(r=256, dr=256),
                                dict(r=512, dr=256, dv=200), dict(r=1024, dr=256),
                                dict(r=1024, dr=0, dv=600, T=60)], ids=str)
def test_cuda_cores_at_each_kernels_largest_rows(mla, kw):
    kw = dict(dict(T=20, dv=64), **kw)
    Case(mla, 3, lens=[kw["T"] + 70, 0, kw["T"]], dtype="f32", dh=64, bs=16, kernel=mla.DECODE_SIMT,
         **kw).run(mla)


@GPU
def test_calls_from_two_threads_at_sizes_of_their_own(mla):
    """Two models whose calls use the same kernels with other amounts of shared memory, a thread, a
    stream and a workspace each. Called without the interpreter's lock, as a C program would."""
    cases = [Case(mla, 4, 2, [70], dtype="f32", r=256, dr=dr, dh=16, dv=dv, kernel=1, seed=dr)
             for dr, dv in ((0, 45), (256, 60))]
    ready = [c.device(mla) for c in cases]
    mla.lib.mla_decode_tree  # loaded before the threads start
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    bad = [[], []]

    def calls(k):
        c, t = cases[k], ready[k]
        args = (c.cfg.ref(), t["q"].data_ptr(), t["pool"].data_ptr(), t["table"].data_ptr(),
                c.table.shape[1], c.pool.shape[0], t["lens"].data_ptr(), 1, 2, t["mask"].data_ptr(),
                t["w_uv"].data_ptr(), t["ws"].data_ptr(), t["ws"].numel(), t["o"].data_ptr(),
                t["lse"].data_ptr(), t["err"].data_ptr(), streams[k].cuda_stream)
        for _ in range(5000):
            st = mla.lib.mla_decode_tree(*args)
            if st:
                bad[k].append(st)

    threads = [threading.Thread(target=calls, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert bad == [[], []], (len(bad[0]), len(bad[1]))
    for c, t in zip(cases, ready):
        assert int(t["err"]) == 0
        c.check(t["o"], t["lse"])


FIRST_CHUNK = r"""
#include <cstdio>
#include "tree.cuh"
int main() {
  const int counts[] = {1, 2, 73, 74, 75, 1000, 28999999, 29020050, 33554431, 33554432, 2147483647};
  for (int C : counts)
    for (int R = 1; R <= mla::kRanges && R <= C; ++R)
      for (int q = 0; q <= R; ++q)
        if (mla::first_chunk(q, R, C) != (int)((long long)q * C / R))
          return std::printf("q %d R %d C %d: %d\n", q, R, C, mla::first_chunk(q, R, C)), 1;
  return 0;
}
"""


def test_ranges_begin_where_they_should_at_any_number_of_chunks(mla, tmp_path):
    """On the host, with signed overflow trapped: 74 ranges of 2^25 chunks pass 2^31 on the way."""
    from mla_latent_kv_44_b200 import build

    src, exe = tmp_path / "first_chunk.cu", tmp_path / "first_chunk"
    src.write_text(FIRST_CHUNK)
    trap = "-fsanitize=signed-integer-overflow,-fsanitize-undefined-trap-on-error"
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-O1", "--expt-relaxed-constexpr", "-Xcompiler",
                    trap, "-I", build.INCLUDE, "-I", build.CSRC, str(src), "-o", str(exe)],
                   check=True, capture_output=True, timeout=300)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, (out.returncode, out.stdout)


@GPU
@pytest.mark.parametrize("kernel,bs", [(1, 64), (1, 16), (2, 64), (2, 128), (2, 320)])
def test_rows_of_a_block_outside_the_pool_are_left_out(mla, kernel, bs):
    """Flagged, and attended by nobody: no other request's rows come in their place (block 0 holds NaN
    here), in the prefix or among the drafted rows, for one block or for all."""
    T = 6
    c = Case(mla, 16, T, [900, 700, 64, 330, 2000], bs=bs, kernel=kernel, seed=3)
    spare = sorted(set(range(c.pool.shape[0])) - set(c.table.flatten().tolist()))[0]
    c.table[c.table == 0] = spare                    # nobody's block 0
    c.pool[0] = float("nan")
    gone = [{0}, {2, 700 // bs}, {63 // bs}, set(), set(range(-(-2000 // bs)))]
    ids = [c.pool.shape[0], -1, 2 ** 31 - 1, -2 ** 31]
    was = c.table.clone()
    for b, blocks in enumerate(gone):
        for i, k in enumerate(sorted(blocks)):
            c.table[b, k] = ids[(b + i) % 4]
    t = c.device(mla)
    c.call(mla, t)
    assert int(t["err"]) == mla.DEV_OOB_BLOCK
    o, lse = t["o"].cpu().double(), t["lse"].cpu().double()
    for b, n in enumerate(c.lens):
        rows = c.pool[was[b].long()].reshape(-1, c.D)[:n]
        out = torch.tensor([j // bs in gone[b] for j in range(n)])
        seen = c.seen[b] & ~out[n - T:]
        keep = ~out
        keep[n - T:] = True
        at = slice(b * T, (b + 1) * T)
        if out.all():
            assert (lse[at] == -float("inf")).all() and (o[at] == 0).all(), b
            continue
        want, wl, size, dot = tu.attend(c.q[at], rows[keep], seen, c.w_uv, c.r, c.scale)
        tol, tol_l = tu.tolerances(c.cfg.torch_dtype, want, size, dot, c.D, n)
        none = torch.isinf(wl)
        assert (lse[at][none] == -float("inf")).all() and (o[at][none] == 0).all(), b
        assert ((o[at] - want).abs() <= tol).all(), b
        assert ((lse[at] - wl).abs() <= tol_l)[~none].all(), b


# ------------------------------------------------------------------------------- append_slots

def _rotated(kr, pos, base):
    """Rotated keys in the host's longest floating type, and the angles."""
    dr = kr.shape[1]
    i = np.arange(dr // 2, dtype=np.longdouble)
    theta = np.longdouble(base) ** (-2 * i / dr)
    a = pos.numpy().astype(np.longdouble)[:, None] * theta
    x = kr.double().numpy().astype(np.longdouble)
    x0, x1 = x[:, 0::2], x[:, 1::2]
    out = np.stack([x0 * np.cos(a) - x1 * np.sin(a), x0 * np.sin(a) + x1 * np.cos(a)], -1)
    size = np.repeat(abs(x0) + abs(x1), 2, axis=1)
    return out.reshape(kr.shape), size, np.repeat(abs(a), 2, axis=1)


@GPU
@pytest.mark.parametrize("dr,base", [(64, 10000.0), (256, 10000.0), (32, 500000.0), (8, 10000.0)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rotated_keys_at_near_and_far_positions(mla, dr, base, dtype):
    """The angle is a product in double: off by 2^-53 for the frequency's rounding and 2^-53 for its
    own, of its size. An fp32 pool holds the key rounded once from double, as mla_append_latent writes
    it; for a bf16 pool sine and cosine are taken in fp32 (2^-23 for the angle's rounding there, 2^-22
    for CUDA's sincosf, of 2 ulp at most) and combined in two roundings, 2^-23."""
    n, r, bs = 96, 32, 8
    cfg = mla.Config(16, 64, r, dr, bs, dtype=dtype, rope_base=base)
    dt, g = cfg.torch_dtype, torch.Generator().manual_seed(dr)
    ckv, kr = torch.randn(n, r, generator=g).to(dt), torch.randn(n, dr, generator=g).to(dt)
    top = torch.tensor([0, 1, 2 ** 31 - 1, 2 ** 31 - 2, 2 ** 24 + 1, 2 ** 30 + 7])
    pos = torch.cat([top, torch.randint(0, 2 ** 17, (n - 6,), generator=g)]).int()
    d = lambda x: x.to(D_)  # noqa: E731
    err, gamma = torch.zeros(1, dtype=torch.int32, device=D_), torch.ones(r, device=D_)
    pool = torch.zeros(n // bs, bs, r + dr, dtype=dt, device=D_)
    mla.append_slots(cfg, d(ckv), d(kr), gamma, d(pos), torch.arange(n, device=D_), pool, err)
    assert int(err) == 0
    got = pool.view(n, r + dr)[:, r:].cpu().double().numpy()
    want, size, angle = _rotated(kr, pos, base)
    work = 2.0 ** -23 + 2.0 ** -22 + 2.0 ** -23 if dtype == "bf16" else 0.0
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    tol = step * abs(want) + (angle * 2.0 ** -52 + 2.0 ** -32 + work) * size
    assert (abs(got - want) <= tol).all(), float((abs(got - want) / tol).max())
    # the same rows through a table
    short = pos.clone()
    short[:6] = torch.arange(6) + 2 ** 17
    table = torch.zeros(n, 2 ** 17 // bs + 1, dtype=torch.int32, device=D_)
    table[:] = d(torch.arange(n // bs).repeat_interleave(bs).int())[:, None]
    short = (short // bs * bs + torch.arange(n) % bs).int()  # row n % bs of block n / bs
    pools = [torch.zeros_like(pool) for _ in range(2)]
    mla.append_slots(cfg, d(ckv), d(kr), gamma, d(short), torch.arange(n, device=D_), pools[0], err)
    mla.append_latent(cfg, d(ckv), d(kr), gamma, torch.arange(n, dtype=torch.int32, device=D_), d(short),
                      table, pools[1], err)
    assert int(err) == 0
    a, b = (p.view(n, r + dr)[:, r:].cpu() for p in pools)
    if dtype == "f32":  # both round one double, whose last bit may differ: one value in 10^8
        assert int((a != b).sum()) <= 1


# ------------------------------------------------------------------------------------ binding

@GPU
def test_a_stream_that_is_none_launches_nothing(mla):
    """A handle that no pointer holds: refused before the launch, by every call."""
    i32, bad = torch.int32, 1 << 70
    z = lambda *s, t=i32: torch.full(s, -7, dtype=t, device=D_)  # noqa: E731
    one, cfg = torch.ones(1, dtype=i32, device=D_), mla.Config(2, 32, 64, 32, 8, dtype="f32")
    f32 = torch.float32
    pool, table, err = z(2, 8, 96, t=f32), torch.zeros(1, 1, dtype=i32, device=D_), torch.zeros_like(one)
    ws = torch.zeros(mla.decode_tree_workspace_size(cfg, 1, 1), dtype=torch.uint8, device=D_)
    outs = dict(cu=z(2), seq=z(1), pos=z(1), slots=z(1, t=torch.int64), held=z(1), count=z(1), mask=z(1, 1),
                tpos=z(1), pool=pool, o=z(1, 2, 32, t=f32), lens=z(1))
    was = {k: v.clone() for k, v in outs.items()}
    for call in (
            lambda: mla.build_tables(cfg, one, one, table, one, z(2), one, outs["held"], outs["count"],
                                     outs["cu"], outs["seq"], outs["pos"], outs["slots"], err, bad),
            lambda: mla.tree_masks(z(1, 1), one, outs["mask"], outs["tpos"], err, bad),
            lambda: mla.append_slots(cfg, z(1, 64, t=f32), z(1, 32, t=f32), z(64, t=f32), one,
                                     torch.zeros(1, dtype=torch.int64, device=D_), pool, err, bad),
            lambda: mla.decode_tree(cfg, z(1, 2, 96, t=f32), pool, table, one, 1, None, z(2, 32, 64, t=f32),
                                    ws, outs["o"], None, err, bad),
            lambda: mla.commit_tree(cfg, torch.zeros(1, 1, dtype=i32, device=D_), one, 1, table, pool, one,
                                    outs["lens"], err, bad)):
        with pytest.raises(OverflowError):
            call()
    torch.cuda.synchronize()
    assert int(err) == 0 and all(torch.equal(outs[k], was[k]) for k in outs)


def test_no_workspace_size_for_what_the_call_refuses(mla):
    size, cfg = mla.decode_tree_workspace_size, mla.Config(1, 32, 64, 32, 8)
    assert size(cfg, 1 << 24, 1) > 0 and size(cfg, 1 << 16, 256) > 0
    assert size(cfg, (1 << 24) + 1, 1) == 0 and size(cfg, 1 << 17, 256) == 0
    for n in (2 ** 32 + 1, -2 ** 32 + 1, 2 ** 63):      # not taken modulo 2^32
        assert size(cfg, n, 4) == 0 and size(cfg, 1, n) == 0


# ----------------------------------------------------------------------------- far offsets

@GPU
def test_tables_whose_slots_pass_32_bits(mla):
    bs, blocks, i32 = 1 << 12, 1 << 20, torch.int32
    cfg = mla.Config(16, 64, 64, 32, bs)
    t = lambda *x: torch.tensor(x, dtype=i32, device=D_)  # noqa: E731
    free = torch.arange(blocks, dtype=i32, device=D_)
    for tokens in (6, 40000):                        # one launch, and a slot map of its own
        lens, count, held = t(bs + 5, 0, 30000), t(blocks), t(0, 0, 0)
        table, err = torch.full((3, 8), -1, dtype=i32, device=D_), t(0)
        new = t(3, 0, 3) if tokens == 6 else t(bs + 5, 0, 30000)
        cu, seq, pos = torch.zeros(4, dtype=i32, device=D_), *torch.zeros(2, tokens, dtype=i32, device=D_)
        slots = torch.zeros(tokens, dtype=torch.int64, device=D_)
        mla.build_tables(cfg, lens, new, table, held, free, count, held, count, cu, seq, pos, slots, err)
        assert int(err) == 0 and held.tolist() == [2, 0, 8] and int(count) == blocks - 10
        n = int(cu[-1])
        assert n == int(new.sum())
        want = table[seq[:n].long(), (pos[:n] // bs).long()].long() * bs + pos[:n] % bs
        assert torch.equal(slots[:n], want) and int(slots.max()) > 1 << 31
        assert (slots[n:] == -1).all() and table[0, :2].tolist() == [blocks - 1, blocks - 2]


@GPU
@pytest.mark.parametrize("dtype,kernel", [("bf16", 1), ("bf16", 2), ("f32", 1)])
def test_a_pool_of_more_than_2_to_31_values(mla, dtype, kernel):
    """Rows written, attended and moved at the pool's end, in a sequence that also has its begin."""
    bs, T, H, n = 64, 5, 4, 700
    cfg = mla.Config(H, 64, 512, 64, bs, dtype=dtype, decode_kernel=kernel)
    dt, i32, blocks = cfg.torch_dtype, torch.int32, 2 ** 31 // (64 * 576) + 50
    c = Case(mla, H, T, [n], dtype=dtype, dh=64, kernel=kernel, seed=4)
    pool = torch.empty(blocks, bs, 576, dtype=dt, device=D_)
    table = torch.arange(blocks - 1, blocks - 1 - c.table.shape[1], -1, dtype=i32, device=D_).view(1, -1)
    table[0, 1] = 0
    flat = pool.view(-1, 576)
    at = torch.tensor([int(table[0, j // bs]) * bs + j % bs for j in range(n)], device=D_)
    flat[at] = c.rows(0).to(D_)
    # the drafted rows again, by slots
    g = torch.Generator().manual_seed(1)
    ckv, kr = torch.randn(T, 512, generator=g).to(dt).to(D_), torch.randn(T, 64, generator=g).to(dt).to(D_)
    err, pos = torch.zeros(1, dtype=i32, device=D_), torch.arange(T, dtype=i32, device=D_)
    gamma = torch.ones(512, device=D_)
    mla.append_slots(cfg, ckv, kr, gamma, pos, at[n - T:], pool, err)
    small = torch.zeros(1, bs, 576, dtype=dt, device=D_)
    mla.append_slots(cfg, ckv, kr, gamma, pos, torch.arange(T, device=D_), small, err)
    assert torch.equal(flat[at[n - T:]], small[0, :T])
    flat[at] = c.rows(0).to(D_)
    t = c.device(mla)
    lens = torch.tensor([n], dtype=i32, device=D_)
    mla.decode_tree(cfg, t["q"], pool, table, lens, T, t["mask"], t["w_uv"], t["ws"], t["o"], t["lse"], err)
    assert int(err) == 0
    c.check(t["o"], t["lse"])
    out = torch.zeros(1, dtype=i32, device=D_)
    mla.commit_tree(cfg, torch.tensor([[0, 2, 4]], dtype=i32, device=D_),
                    torch.tensor([3], dtype=i32, device=D_), T, table, pool, lens, out, err)
    assert int(err) == 0 and int(out) == n - T + 3
    want = c.rows(0).to(D_)
    want[n - T + 1], want[n - T + 2] = want[n - T + 2].clone(), want[n - T + 4].clone()
    assert torch.equal(flat[at], want)


@GPU
@pytest.mark.parametrize("batch,tokens", [(8192, 40000), (3060, 33000), (1025, 32769)])
def test_tables_of_many_requests_with_a_slot_map_of_their_own(mla, batch, tokens):
    from tests.test_tree_tables import _requests, _run_tables

    _run_tables(mla, 4, *_requests(batch, batch, 2, 4, 2 * batch), tokens, in_place=True)
