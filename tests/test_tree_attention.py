"""mla_decode_tree against the 64-bit form: shapes, masks, padded batches, values that are not finite,
streams, graphs, and the calls of a step together."""
import json
import math
import os
import subprocess
import sys

import pytest
import torch

from tests import tree_util as tu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu
D_ = "cuda"


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_44_b200 as m

    return m


class Case:
    """Inputs of one call, on the CPU, and their device copies. lens count the drafted rows."""

    def __init__(self, mla, H, T, lens, dtype="bf16", r=512, dr=64, dh=128, dv=0, bs=64, kind="random",
                 seed=0, kernel=0, extra=1, scale_rows=None, parents=None):
        self.cfg = mla.Config(H, dh, r, dr, bs, dtype=dtype, head_dim_v=dv, decode_kernel=kernel)
        self.H, self.T, self.lens, self.r, self.D, self.bs = H, T, lens, r, r + dr, bs
        self.dv, dt = dv or dh, self.cfg.torch_dtype
        g = torch.Generator().manual_seed(1000 * seed + H + T)
        B, most = len(lens), max(1, -(-max(lens) // bs)) + extra
        total = B * most + 2
        self.table = torch.randperm(total, generator=g)[:B * most].view(B, most).int()
        self.pool = torch.randn(total, bs, self.D, generator=g).to(dt)
        if scale_rows:
            self.pool *= scale_rows(torch.arange(total * bs)).view(total, bs, 1).to(dt)
        q = torch.randn(B * T, H, self.D, generator=g)
        q[..., :r] *= math.sqrt(dh / r)
        self.q = q.to(dt)
        self.w_uv = (torch.randn(H, self.dv, r, generator=g) / math.sqrt(r)).to(dt)
        self.seen = tu.seen_of(tu.parents_of(kind, B, T, seed) if parents is None else parents)
        self.scale = 1.0 / math.sqrt(dh + dr)

    def rows(self, b):
        n = self.lens[b]
        return self.pool[self.table[b].long()].reshape(-1, self.D)[:n]

    def slot(self, b, row):
        return int(self.table[b, row // self.bs]) * self.bs + row % self.bs

    def device(self, mla):
        B, dt = len(self.lens), self.cfg.torch_dtype
        to = lambda x: x.to(D_)  # noqa: E731
        size = mla.decode_tree_workspace_size(self.cfg, B, self.T)
        return dict(q=to(self.q), pool=to(self.pool), table=to(self.table),
                    lens=torch.tensor(self.lens, dtype=torch.int32, device=D_),
                    mask=to(tu.words_of(self.seen)), w_uv=to(self.w_uv),
                    ws=torch.full((size,), 0xff, dtype=torch.uint8, device=D_),
                    o=torch.full((B * self.T, self.H, self.dv), math.nan, dtype=dt, device=D_),
                    lse=torch.full((B * self.T, self.H), math.nan, device=D_),
                    err=torch.zeros(1, dtype=torch.int32, device=D_))

    def call(self, mla, t, mask=True, lse=True, stream=None):
        mla.decode_tree(self.cfg, t["q"], t["pool"], t["table"], t["lens"], self.T,
                        t["mask"] if mask else None, t["w_uv"], t["ws"], t["o"],
                        t["lse"] if lse else None, t["err"], stream)

    def check(self, o, lse, seqs=None):
        dt = self.cfg.torch_dtype
        o, lse = o.cpu().double(), lse.cpu().double()
        for b in range(len(self.lens)) if seqs is None else seqs:
            n, at = self.lens[b], slice(b * self.T, (b + 1) * self.T)
            if n < self.T:
                assert (o[at] == 0).all() and (lse[at] == -math.inf).all(), b
                continue
            want, wl, size, dot = tu.attend(self.q[at], self.rows(b), self.seen[b], self.w_uv, self.r,
                                            self.scale)
            tol, tol_l = tu.tolerances(dt, want, size, dot, self.D, n)
            none = torch.isinf(wl)
            assert (lse[at][none] == -math.inf).all() and (o[at][none] == 0).all(), b
            assert torch.isfinite(o[at]).all(), b
            off = ((o[at] - want).abs() / tol).max()
            assert off <= 1, (b, n, float(off))
            off = ((lse[at] - wl).abs() / tol_l)[~none]
            assert off.numel() == 0 or off.max() <= 1, (b, n, float(off.max()))

    def run(self, mla, **kw):
        t = self.device(mla)
        self.call(mla, t, **kw)
        torch.cuda.synchronize()
        assert int(t["err"]) == 0
        self.check(t["o"], t["lse"])
        return t


TC = [  # tensor cores: bf16, r = 512, d_r = 64, blocks of a multiple of 64
    dict(H=128, T=1, lens=[1]), dict(H=128, T=1, lens=[64, 65, 63, 2]),
    dict(H=128, T=2, lens=[2, 300]), dict(H=128, T=5, lens=[257, 5, 1000]),
    dict(H=16, T=1, lens=[700, 30]), dict(H=16, T=8, lens=[8, 72, 511]),
    dict(H=16, T=9, lens=[200, 4000]), dict(H=8, T=3, lens=[3, 129], dh=64),
    dict(H=1, T=1, lens=[5]), dict(H=1, T=37, lens=[100, 37]), dict(H=3, T=33, lens=[33, 97, 290]),
    dict(H=64, T=32, lens=[33, 95, 96, 97]), dict(H=32, T=65, lens=[130, 65]),
    dict(H=16, T=256, lens=[256, 300]), dict(H=128, T=17, lens=[2100]),
    dict(H=128, T=3, lens=[500, 130], bs=128), dict(H=16, T=4, lens=[1000, 40], bs=320),
    dict(H=16, T=4, lens=[77, 300], dv=192), dict(H=5, T=4, lens=[77, 300], dv=33),
    dict(H=40, T=11, lens=[64 * k + k for k in range(1, 30)])]


@pytest.mark.parametrize("kw", TC, ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items())[:60])
@pytest.mark.parametrize("kind", ["random", "chain"])
def test_tensor_cores(mla, kw, kind):
    Case(mla, kind=kind, kernel=mla.DECODE_TENSOR, **kw).run(mla)


SIMT = [dict(H=16, T=5, lens=[1029, 5, 60], r=64, dr=32, dh=64), dict(H=8, T=1, lens=[1], r=64, dr=16, dh=32),
        dict(H=16, T=16, lens=[300, 17], r=64, dr=32, dh=64, bs=7),
        dict(H=3, T=33, lens=[33, 200], r=96, dr=8, dh=24, bs=16), dict(H=2, T=40, lens=[90], r=32, dr=0, dh=16),
        dict(H=4, T=3, lens=[70, 3], r=128, dr=64, dh=32, dv=48), dict(H=4, T=3, lens=[70, 35], r=256, dr=64, dh=8),
        dict(H=4, T=4, lens=[65], r=512, dr=64, dh=128, bs=40), dict(H=2, T=2, lens=[50, 2], r=1024, dr=256, dh=16),
        dict(H=2, T=2, lens=[50], r=768, dr=64, dh=16), dict(H=1, T=256, lens=[256, 400], r=64, dr=32, dh=64),
        dict(H=64, T=40, lens=[41, 90], r=64, dr=32, dh=64)]


@pytest.mark.parametrize("kw", SIMT, ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items())[:60])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cuda_cores(mla, kw, dtype):
    Case(mla, dtype=dtype, kernel=mla.DECODE_SIMT, **kw).run(mla)


@pytest.mark.parametrize("kw", [
    dict(H=16, T=32, lens=[5000]), dict(H=16, T=33, lens=[5000]), dict(H=1, T=1, lens=[20000]),
    dict(H=2, T=40, lens=[20000]), dict(H=128, T=1, lens=[64 * k for k in range(32)], dv=192),
    dict(H=128, T=1, lens=[64 * k for k in range(33)]), dict(H=24, T=4, lens=[900] * 8, dv=33),
    dict(H=128, T=16, lens=[900, 0]), dict(H=128, T=11, lens=[900, 11, 0])],
    ids=lambda k: f"H{k['H']}-T{k['T']}-B{len(k['lens'])}-L{k['lens'][0]}")
def test_partial_results_merged_with_the_output_or_before(mla, kw):
    """Up to 32 tokens the output kernel merges; items of one to 74 pieces, empty sequences."""
    Case(mla, kernel=mla.DECODE_TENSOR, **kw).run(mla)


@pytest.mark.parametrize("kernel", [1, 2])
def test_padded_batch(mla, kernel):
    """Empty places between sequences: zeros, lse -inf, no error."""
    Case(mla, 16, 6, [0, 70, 0, 0, 6, 300, 0], kernel=kernel).run(mla)
    Case(mla, 16, 6, [0, 0], kernel=kernel).run(mla)


@pytest.mark.parametrize("kernel", [1, 2])
def test_impossible_lengths_are_flagged(mla, kernel):
    c = Case(mla, 16, 6, [70, 70, 70], kernel=kernel)
    for bad in (5, -1, (c.table.shape[1] * 64) + 1):
        t = c.device(mla)
        t["lens"][1] = bad
        c.call(mla, t)
        assert int(t["err"]) == mla.DEV_BAD_LENGTH
        keep, c.lens = c.lens, [70, 0, 70]
        c.check(t["o"], t["lse"])
        c.lens = keep


@pytest.mark.parametrize("kernel", [1, 2])
def test_block_outside_the_pool_is_flagged(mla, kernel):
    c = Case(mla, 16, 2, [300, 200], kernel=kernel)
    t = c.device(mla)
    t["table"][0, 2] = c.pool.shape[0]
    c.call(mla, t)
    assert int(t["err"]) == mla.DEV_OOB_BLOCK
    c.check(t["o"], t["lse"], seqs=[1])


@pytest.mark.parametrize("kernel,kw", [(1, {}), (2, {}), (1, dict(dtype="f32", r=64, dr=32, dh=64))])
def test_nodes_that_see_nothing(mla, kernel, kw):
    """A mask of zeros, with and without rows before the tree; any bits elsewhere."""
    c = Case(mla, 16, 40, [40, 41, 104, 200], kernel=kernel, **kw)
    g = torch.Generator().manual_seed(1)
    c.seen = torch.rand(c.seen.shape, generator=g) < 0.3
    c.seen[:, ::7] = False
    t = c.run(mla)
    assert (t["lse"].view(4, 40, 16)[0, ::7] == -math.inf).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, "lowest"])
@pytest.mark.parametrize("kernel,kw", [(1, {}), (2, {}), (2, dict(bs=128)),
                                       (1, dict(dtype="f32", r=64, dr=32, dh=64))])
def test_what_masked_rows_hold_does_not_matter(mla, kernel, kw, bad):
    """A drafted row that a node does not see, and rows behind the last, never reach it."""
    c = Case(mla, 16, 35, [35, 90, 130, 256], kernel=kernel, kind="chain", **kw)
    c.seen[:, :, 20] = False           # nobody sees node 20
    c.seen[:, 20, :] = False
    c.seen[:, 20, 3] = True
    c.seen[:, 10:, 9] = False          # node 9 is seen by itself alone ...
    dt = c.cfg.torch_dtype
    v = torch.finfo(dt).min if bad == "lowest" else bad
    flat = c.pool.view(-1, c.D)
    for b, n in enumerate(c.lens):
        flat[c.slot(b, n - 35 + 20)] = v
        for row in range(n, c.table.shape[1] * c.bs):
            flat[c.slot(b, row)] = v
    t = c.run(mla)
    for b, n in enumerate(c.lens):     # ... which then has no finite result, and the others have
        t["pool"].view(-1, c.D)[c.slot(b, n - 35 + 9)] = math.nan
    c.call(mla, t)
    o = t["o"].view(4, 35, -1).cpu()
    assert torch.isnan(o[:, 9]).all()
    keep = [k for k in range(35) if k != 9]
    assert torch.isfinite(o[:, keep].float()).all()


def test_scores_that_grow_along_the_cache(mla):
    """The running maximum moves by far more than 2^8 from tile to tile."""
    for kernel in (1, 2):
        c = Case(mla, 16, 3, [900, 2000], kernel=kernel, extra=0,
                 scale_rows=lambda i: torch.ones_like(i, dtype=torch.float32))
        for b, n in enumerate(c.lens):
            rows = torch.arange(n)
            f = 1.0 + rows.float() / 40.0
            for row in range(n):
                c.pool.view(-1, c.D)[c.slot(b, row)] *= f[row]
        c.run(mla)


@pytest.mark.parametrize("H,T,lens", [(128, 4, [500, 64, 5, 700]), (16, 7, [300, 7])])
def test_a_chain_without_a_mask_is_mla_decode(mla, H, T, lens):
    c = Case(mla, H, T, lens, kind="chain")
    t = c.run(mla, mask=False)
    with_mask = c.run(mla)
    assert torch.equal(t["o"], with_mask["o"]) and torch.equal(t["lse"], with_mask["lse"])
    n = len(lens) * T
    lat = torch.empty(n, H, 512, device=D_)
    lse, o = torch.empty(n, H, device=D_), torch.empty(n, H, 128, dtype=torch.bfloat16, device=D_)
    ws = torch.empty(mla.decode_workspace_size(c.cfg, len(lens), T), dtype=torch.uint8, device=D_)
    mla.decode(c.cfg, t["q"], t["pool"], t["table"], t["lens"], T, ws, lat, lse, t["err"])
    mla.output(c.cfg, lat, t["w_uv"], o, dev_err=t["err"])
    assert int(t["err"]) == 0
    # both round the weights and o to bf16
    assert float((t["o"].double() - o.double()).norm() / o.double().norm()) < 2.0 ** -7
    assert float((t["lse"] - lse).abs().max()) < 2.0 ** -8  # mla_decode sums the rounded weights


def test_lse_may_be_left_out(mla):
    for kernel, kw in ((2, {}), (1, {}), (1, dict(dtype="f32", r=64, dr=32, dh=64))):
        c = Case(mla, 16, 5, [300, 0, 5], kernel=kernel, **kw)
        t = c.run(mla)
        u = c.device(mla)
        c.call(mla, u, lse=False)
        assert torch.equal(t["o"], u["o"]) and torch.isnan(u["lse"]).all()


def test_rows_behind_the_outputs_are_left_alone(mla):
    """The last tile of query rows reaches past the call's: nothing there is written."""
    for kernel in (1, 2):
        c = Case(mla, 5, 3, [70, 200], kernel=kernel)
        t = c.device(mla)
        big_o = torch.full((16, 5, 128), 3.0, dtype=torch.bfloat16, device=D_)
        big_l = torch.full((16, 5), 3.0, device=D_)
        t["o"], t["lse"] = big_o[:6], big_l[:6]
        c.call(mla, t)
        c.check(t["o"], t["lse"])
        assert (big_o[6:] == 3).all() and (big_l[6:] == 3).all()


def test_same_bits_again_and_on_other_streams(mla):
    """Two calls at once on streams of their own, each with its workspace, give the bits of one."""
    cases = [Case(mla, 128, 4, [900, 333], seed=1), Case(mla, 16, 31, [700] * 9, seed=2)]
    base = [c.run(mla) for c in cases]
    side = [c.device(mla) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, t, s in zip(cases, side, streams):
            c.call(mla, t, stream=s)
    torch.cuda.synchronize()
    for b, t in zip(base, side):
        assert int(t["err"]) == 0
        assert torch.equal(b["o"], t["o"]) and torch.equal(b["lse"], t["lse"])


def test_current_stream_is_the_default(mla):
    c = Case(mla, 16, 4, [500])
    base, t = c.run(mla), c.device(mla)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.call(mla, t)
    s.synchronize()
    assert torch.equal(base["o"], t["o"])


@pytest.mark.parametrize("kernel", [1, 2])
def test_captured_and_replayed_with_other_lengths(mla, kernel):
    """A graph takes its lengths from the device: replays follow them, padded places among them.
    Two graphs share one workspace, replayed one after the other."""
    c = Case(mla, 16, 6, [400, 90, 257], kernel=kernel)
    t = c.device(mla)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.call(mla, t)
    s.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        out = dict(t, o=torch.empty_like(t["o"]), lse=torch.empty_like(t["lse"]))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.call(mla, out)
        graphs.append(g)
        outs.append(out)
    for lens in ([400, 90, 257], [6, 0, 64], [0, 300, 7]):
        t["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        for g, out in zip(graphs, outs):
            out["o"].fill_(math.nan)
            g.replay()
        torch.cuda.synchronize()
        keep, c.lens = c.lens, lens
        for out in outs:
            c.check(out["o"], out["lse"])
        c.lens = keep
    assert int(t["err"]) == 0


@pytest.mark.parametrize("kernel", [1, 2])
def test_weights_written_just_before_the_call(mla, kernel):
    """W_UV, Q, the lengths and the rows come from kernels that are still queued or running."""
    c = Case(mla, 16, 3, [300, 65], kernel=kernel)
    t = c.device(mla)
    names = ("w_uv", "q", "pool", "lens", "table", "mask")
    real = {k: t[k].clone() for k in names}
    busy = torch.randn(4096, 4096, device=D_)
    for _ in range(5):
        for k in names:
            t[k].zero_()
        c.call(mla, t)
        for _ in range(3):
            busy = busy @ busy * 1e-2
        for k in reversed(names):
            t[k].copy_(real[k])
        c.call(mla, t)
        t["err"].zero_()
        c.check(t["o"], t["lse"])


def test_many_short_sequences(mla):
    """More sequences than a range's list in shared memory holds."""
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 130, (700,), generator=g).tolist()
    lens = [0 if n < 2 else n for n in lens]
    c = Case(mla, 2, 2, lens, extra=0)
    t = c.device(mla)
    c.call(mla, t)
    torch.cuda.synchronize()
    assert int(t["err"]) == 0
    c.check(t["o"], t["lse"], seqs=list(range(0, 700, 23)) + [699])


def test_long_cache(mla):
    """Offsets into the pool that pass 32 bits in bytes and, in values, come close to them."""
    bs, blocks = 64, 60000                       # 60,000 x 64 x 576 bf16: 4.4 GB
    cfg = mla.Config(16, 128, 512, 64, bs)
    L, T, H = 40000, 3, 16
    need = -(-L // bs)
    g = torch.Generator(device=D_).manual_seed(0)
    pool = torch.empty(blocks, bs, 576, dtype=torch.bfloat16, device=D_)
    table = (blocks - 1 - torch.arange(need, dtype=torch.int32, device=D_) * 7).view(1, need)
    table[0, ::2] = torch.arange(0, need, 2, dtype=torch.int32, device=D_)
    rows = torch.randn(need, bs, 576, generator=g, device=D_).bfloat16()
    pool[table[0].long()] = rows
    q = torch.randn(T, H, 576, generator=g, device=D_)
    q[..., :512] *= 0.5
    w_uv = (torch.randn(H, 128, 512, generator=g, device=D_) / 512 ** 0.5).bfloat16()
    seen = tu.seen_of(torch.tensor([[-1, 0, 0]]))
    o = torch.empty(T, H, 128, dtype=torch.bfloat16, device=D_)
    lse, err = torch.empty(T, H, device=D_), torch.zeros(1, dtype=torch.int32, device=D_)
    ws = torch.empty(mla.decode_tree_workspace_size(cfg, 1, T), dtype=torch.uint8, device=D_)
    mla.decode_tree(cfg, q.bfloat16(), pool, table, torch.tensor([L], dtype=torch.int32, device=D_), T,
                    tu.words_of(seen).to(D_), w_uv, ws, o, lse, err)
    assert int(err) == 0
    want, wl, size, dot = tu.attend(q.bfloat16().cpu(), rows.view(-1, 576)[:L].cpu(), seen[0],
                                    w_uv.cpu(), 512, 1 / math.sqrt(192))
    tol, tol_l = tu.tolerances(torch.bfloat16, want, size, dot, 576, L)
    assert ((o.cpu().double() - want).abs() <= tol).all()
    assert ((lse.cpu().double() - wl).abs() <= tol_l).all()


# --------------------------------------------------------------- the calls of a step, together

def _rope(x, pos, base=10000.0):
    dr = x.shape[-1]
    a = pos * base ** (-2.0 * torch.arange(dr // 2, dtype=torch.float64) / dr)
    x0, x1 = x[..., 0::2].double(), x[..., 1::2].double()
    return torch.stack([x0 * a.cos() - x1 * a.sin(), x0 * a.sin() + x1 * a.cos()], -1).flatten(-2)


@pytest.mark.parametrize("dtype,H,dh,r,dr,bs", [("bf16", 128, 128, 512, 64, 64),
                                                ("f32", 16, 64, 64, 32, 16)])
def test_steps_of_speculative_decoding(mla, dtype, H, dh, r, dr, bs):
    """Prompts, then steps of drafting, verifying and keeping a path, requests ending and coming:
    every node's output equals attention over its own path of tokens, positions and all."""
    cfg = mla.Config(H, dh, r, dr, bs, dtype=dtype)
    dt, i32, D, B, T, width = cfg.torch_dtype, torch.int32, r + dr, 4, 6, 12
    g = torch.Generator().manual_seed(11)
    dev = lambda x: x.to(D_)  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g).to(dt)  # noqa: E731
    w_uk, w_uv = (randn(H, dh, r) / r ** 0.5).to(dt), (randn(H, dh, r) / r ** 0.5).to(dt)
    gamma = 1 + 0.1 * torch.randn(r, generator=g)
    blocks = 40
    pool = torch.full((blocks, bs, D), math.nan, dtype=dt, device=D_)
    state = dict(table=torch.full((B, width), -1, dtype=i32, device=D_),
                 held=torch.zeros(B, dtype=i32, device=D_),
                 free=torch.randperm(blocks, generator=g).int().to(D_),
                 count=torch.tensor([blocks], dtype=i32, device=D_),
                 err=torch.zeros(1, dtype=i32, device=D_))
    kept = [[] for _ in range(B)]     # every sequence's cached rows in 64 bits, by position

    def tables(lens, new):
        n, k = dev(torch.tensor(lens, dtype=i32)), dev(torch.tensor(new, dtype=i32))
        out = [torch.empty(B + 1, dtype=i32, device=D_)] + [
            torch.empty(64, dtype=i32, device=D_) for _ in range(2)] + [
            torch.empty(64, dtype=torch.int64, device=D_)]
        mla.build_tables(cfg, n, k, state["table"], state["held"], state["free"], state["count"],
                         state["held"], state["count"], *out, state["err"])
        return n, out

    def append(ckv, kr, pos, slots):
        mla.append_slots(cfg, dev(ckv), dev(kr), dev(gamma), pos, slots, pool, state["err"])
        x = ckv.double()
        return (x / (x.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * gamma.double()).to(dt)

    def prompts(lens, new):
        n, (cu, seq, pos, slots) = tables(lens, new)
        m = sum(new)
        ckv, kr = randn(64, r), randn(64, dr)
        lat = append(ckv, kr, pos, slots)
        for i in range(m):
            b, p = int(seq[i]), int(pos[i])
            assert len(kept[b]) == p
            kept[b].append(torch.cat([lat[i].double(), _rope(kr[i], p).to(dt).double()]))

    prompts([17, 1, 30, 0], [17, 1, 30, 0])
    for step in range(6):
        if step == 3:                 # request 1 ends, request 3 comes
            kept[1] = []
            prompts([len(k) for k in kept[:3]] + [14], [0, 0, 0, 14])
        live = [len(k) > 0 for k in kept]
        lens = [len(k) + T if x else 0 for k, x in zip(kept, live)]
        n, (cu, seq, pos_, slots) = tables(lens, [T if x else 0 for x in live])
        parents = tu.parents_of("random", B, T, seed=step)
        mask = torch.empty(B * T, 1, dtype=i32, device=D_)
        pos = torch.empty(B * T, dtype=i32, device=D_)
        mla.tree_masks(dev(parents), n, mask, pos, state["err"])
        # the slot map numbers live tokens only; place them at their sequence's nodes
        at = torch.cat([torch.arange(T) + b * T for b in range(B) if live[b]])
        place = torch.full((B * T,), -1, dtype=torch.int64, device=D_)
        place[dev(at)] = slots[: len(at)]
        ckv, kr = randn(B * T, r), randn(B * T, dr)
        qn, qr = randn(B * T, H, dh), randn(B * T, H, dr)
        q = torch.empty(B * T, H, D, dtype=dt, device=D_)
        mla.absorb_query(cfg, dev(qn), dev(qr), pos, dev(w_uk), q, dev_err=state["err"])
        lat = append(ckv, kr, pos, place)
        o = torch.empty(B * T, H, dh, dtype=dt, device=D_)
        lse = torch.empty(B * T, H, device=D_)
        ws = torch.empty(mla.decode_tree_workspace_size(cfg, B, T), dtype=torch.uint8, device=D_)
        mla.decode_tree(cfg, q, pool, state["table"], n, T, mask, dev(w_uv), ws, o, lse, state["err"])
        seen = tu.seen_of(parents)
        paths, accepted = [], []
        for b in range(B):
            if not live[b]:
                assert (o[b * T:(b + 1) * T] == 0).all()
                accepted.append([])
                continue
            depth = seen[b].sum(-1) - 1
            new_rows = [torch.cat([lat[b * T + t].double(),
                                   _rope(kr[b * T + t], len(kept[b]) + int(depth[t])).to(dt).double()])
                        for t in range(T)]
            rows = torch.stack(kept[b] + new_rows)
            qx = torch.empty(T, H, D, dtype=torch.float64)
            for t in range(T):
                k = b * T + t
                qx[t, :, :r] = torch.einsum("hdr,hd->hr", w_uk.double(), qn[k].double())
                qx[t, :, r:] = _rope(qr[k], len(kept[b]) + int(depth[t]))
            got_q = q[b * T:(b + 1) * T].cpu()
            assert float((got_q.double() - qx).norm() / qx.norm()) < (2.0 ** -8 if dtype == "bf16" else 1e-5)
            want, wl, size, dot = tu.attend(got_q, rows, seen[b], w_uv, r, cfg.c().softmax_scale)
            tol, tol_l = tu.tolerances(dt, want, size, dot, D, len(rows))
            # the cache holds rows that may have rounded the other way: one step of the type each, in
            # the values (relative to size) and in the scores (relative to dot)
            step_ = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -22
            worst = 1e-2 if dtype == "bf16" else 2.0 ** -22   # share of values that do, or their step
            got = o[b * T:(b + 1) * T].cpu().double()
            assert ((got - want).abs() <= tol + step_ * size + 2 * worst * step_ * dot.amax() * size).all()
            leaf = int(torch.randint(0, T, (1,), generator=g))
            path = seen[b, leaf].nonzero().flatten().tolist()
            accepted.append(path)
            kept[b] += [new_rows[t] for t in path]
        steps = torch.full((B, T), -1, dtype=i32)
        for b, path in enumerate(accepted):
            steps[b, : len(path)] = torch.tensor(path, dtype=i32)
        counts = torch.tensor([len(p) for p in accepted], dtype=i32)
        mla.commit_tree(cfg, dev(steps), dev(counts), T, state["table"], pool, n, n, state["err"])
        assert n.tolist() == [len(k) for k in kept]
        assert int(state["err"]) == 0
        held = state["held"].tolist()
        used = sum((state["table"][b, :h].tolist() for b, h in enumerate(held)), [])
        rest = state["free"][: int(state["count"])].tolist()
        assert sorted(used + rest) == list(range(blocks))   # no block lost, none held twice


@pytest.mark.parametrize("dtype,H,dh,r,dr,bs", [("bf16", 16, 64, 512, 64, 64),
                                                 ("f32", 4, 32, 64, 32, 16)])
def test_a_whole_step_of_a_padded_batch_in_one_graph(mla, dtype, H, dh, r, dr, bs):
    """Tables to commit captured once and replayed over a batch whose requests grow, end and come:
    the same bits as call by call, in the outputs, the pool and the tables."""
    cfg = mla.Config(H, dh, r, dr, bs, dtype=dtype)
    dt, i32, D, B, T, width, blocks = cfg.torch_dtype, torch.int32, r + dr, 5, 4, 12, 64
    g = torch.Generator().manual_seed(5)
    randn = lambda *s: torch.randn(*s, generator=g).to(dt).to(D_)  # noqa: E731
    w_uk, w_uv, gamma = randn(H, dh, r) / r ** 0.5, randn(H, dh, r) / r ** 0.5, torch.ones(r, device=D_)
    pool, free = randn(blocks, bs, D), torch.randperm(blocks, generator=g).int().to(D_)

    def fresh():
        e = lambda *s, t=i32: torch.zeros(*s, dtype=t, device=D_)  # noqa: E731
        return dict(n=e(B), new=torch.full((B,), T, dtype=i32, device=D_), table=e(B, width) - 1,
                    held=e(B), free=free.clone(), count=e(1) + blocks, cu=e(B + 1), seq=e(B * T),
                    pos_=e(B * T), slots=e(B * T, t=torch.int64), parents=e(B, T), mask=e(B * T, 1),
                    pos=e(B * T), ckv=e(B * T, r, t=dt), kr=e(B * T, dr, t=dt),
                    qn=e(B * T, H, dh, t=dt), qr=e(B * T, H, dr, t=dt), q=e(B * T, H, D, t=dt),
                    o=e(B * T, H, dh, t=dt), path=e(B, T), many=e(B), out=e(B), pool=pool.clone(),
                    ws=e(mla.decode_tree_workspace_size(cfg, B, T), t=torch.uint8), err=e(1))

    def step(s):
        mla.build_tables(cfg, s["n"], s["new"], s["table"], s["held"], s["free"], s["count"], s["held"],
                         s["count"], s["cu"], s["seq"], s["pos_"], s["slots"], s["err"])
        mla.tree_masks(s["parents"], s["n"], s["mask"], s["pos"], s["err"])
        mla.absorb_query(cfg, s["qn"], s["qr"], s["pos"], w_uk, s["q"], dev_err=s["err"])
        mla.append_slots(cfg, s["ckv"], s["kr"], gamma, s["pos"], s["slots"], s["pool"], s["err"])
        mla.decode_tree(cfg, s["q"], s["pool"], s["table"], s["n"], T, s["mask"], w_uv, s["ws"],
                        s["o"], None, s["err"])
        mla.commit_tree(cfg, s["path"], s["many"], T, s["table"], s["pool"], s["n"], s["out"], s["err"])

    eager, graphed = fresh(), fresh()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(graphed)
    kept = [40, 0, 7, 0, 100]
    for k in range(6):
        if k == 2:
            kept[1], kept[4] = 13, 0
        if k == 4:
            kept[0], kept[3], kept[4] = 0, bs, 1
        parents = tu.parents_of("random", B, T, seed=k)
        seen = tu.seen_of(parents)
        paths = [seen[b, k % T].nonzero().flatten().tolist() if kept[b] else [] for b in range(B)]
        new = dict(n=torch.tensor([x + T if x else 0 for x in kept], dtype=i32), parents=parents,
                   path=torch.tensor([p + [-1] * (T - len(p)) for p in paths], dtype=i32),
                   many=torch.tensor([len(p) for p in paths], dtype=i32),
                   **{x: randn(*eager[x].shape) for x in ("ckv", "kr", "qn", "qr")})
        for s in (eager, graphed):
            for name, value in new.items():
                s[name].copy_(value)
        torch.cuda.synchronize()
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        for name in eager:
            if name != "ws":
                assert torch.equal(eager[name], graphed[name]), (k, name)
        assert int(eager["err"]) == 0
        kept = [x + len(p) for x, p in zip(kept, paths)]
        assert eager["out"].tolist() == kept
        empty = [b for b in range(B) if not kept[b]]
        assert (eager["slots"].view(B, T)[empty] == -1).all() and (eager["o"].view(B, T, -1)[empty] == 0).all()
        assert all((eager["o"].view(B, T, -1)[b] != 0).any() for b in range(B) if kept[b])


# ------------------------------------------------------------------- a wait that runs out

CHILD = r"""
import json, sys, time
sys.path.insert(0, ROOT)
import torch
import mla_latent_kv_44_b200 as mla
mla.LIB_PATH = mla.TEST_LIB_PATH
cfg = mla.Config(128, 128, 512, 64, 64)
d = "cuda"
pool = torch.randn(40, 64, 576, device=d).bfloat16()
table = torch.arange(40, dtype=torch.int32, device=d).view(1, 40)
T = 2
q = torch.randn(T, 128, 576, device=d).bfloat16()
w = torch.randn(128, 128, 512, device=d).bfloat16()
o = torch.empty(T, 128, 128, dtype=torch.bfloat16, device=d)
err = torch.zeros(1, dtype=torch.int32, device=d)
ws = torch.empty(mla.decode_tree_workspace_size(cfg, 1, T), dtype=torch.uint8, device=d)
lens = torch.tensor([2500], dtype=torch.int32, device=d)
bits, took = [], []
for _ in range(2):
    err.zero_()
    t0 = time.time()
    mla.decode_tree(cfg, q, pool, table, lens, T, None, w, ws, o, None, err)
    torch.cuda.synchronize()
    took.append(time.time() - t0)
    bits.append(int(err))
x = torch.ones(1000, device=d)
print(json.dumps(dict(bits=bits, took=took, alive=float((x + x).sum()))))
"""


def test_a_load_that_never_comes_ends_in_an_error(mla):
    """The test build leaves one K load of the first range out: the waits for it run out, the call
    reports it and returns, and the context goes on."""
    assert os.path.exists(mla.TEST_LIB_PATH), "build the libraries first"
    out = subprocess.run([sys.executable, "-c", CHILD.replace("ROOT", repr(ROOT))], capture_output=True,
                         text=True, timeout=120)
    assert out.returncode == 0, out.stderr[-2000:]
    got = json.loads(out.stdout.splitlines()[-1])
    assert got["bits"] == [mla.DEV_WAIT_TIMEOUT] * 2
    assert max(got["took"]) < 20 and got["alive"] == 2000.0
