"""Calls from host threads of a program: a thread's first call, and the same call from two threads at once."""
import threading

import pytest
import torch

from tests.test_tree_attention import Case

pytestmark = pytest.mark.gpu
D_ = "cuda"


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_44_b200 as m

    return m


def _absorb(mla, dtype, n, dh, r, dr, H=8):
    cfg = mla.Config(H, dh, r, dr, 64, dtype=dtype)
    t = [torch.randn(*s, device=D_).to(cfg.torch_dtype) for s in ((n, H, dh), (n, H, dr), (H, dh, r))]
    pos, out = torch.arange(n, dtype=torch.int32, device=D_), torch.zeros(n, H, r + dr, device=D_).to(t[0])
    return lambda s: mla.absorb_query(cfg, t[0], t[1], pos, t[2], out, stream=s)


def _output(mla, dtype, n, r, H=8):
    cfg = mla.Config(H, 64, r, 64, 64, dtype=dtype)
    lat, w = torch.randn(n, H, r, device=D_), torch.randn(H, 64, r, device=D_).to(cfg.torch_dtype)
    o = torch.zeros(n, H, 64, device=D_).to(cfg.torch_dtype)
    return lambda s: mla.output(cfg, lat, w, o, stream=s)


def _decode(mla, dr, dtype="f32", H=8):
    cfg = mla.Config(H, 64, 512, dr, 64, dtype=dtype)
    w = lambda *s: torch.randn(*s, device=D_).to(cfg.torch_dtype)  # noqa: E731
    q, pool = w(1, H, 512 + dr), w(2, 64, 512 + dr)
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device=D_), torch.ones(1, dtype=torch.int32, device=D_)
    ws = torch.zeros(mla.decode_workspace_size(cfg, 1, 1), dtype=torch.uint8, device=D_)
    lat, lse, err = torch.zeros(1, H, 512, device=D_), torch.zeros(1, H, device=D_), torch.zeros_like(lens)
    return lambda s: mla.decode(cfg, q, pool, table, lens, 1, ws, lat, lse, err, stream=s)


def _project(mla, n, d_model, dtype="bf16"):
    cfg = mla.Config(2, 64, 64, 64, 64, dtype=dtype)
    front, dt = mla.front_config(d_model), cfg.torch_dtype
    w = lambda *s: torch.randn(*s, device=D_).to(dt)  # noqa: E731
    x, w_q, w_qr, w_dkv, w_kr = (w(rows, d_model) for rows in (n, 128, 128, 64, 64))
    outs = [w(n, 2, 64), w(n, 2, 64), w(n, 64), w(n, 64)]
    ws = torch.zeros(max(256, mla.project_workspace_size(cfg, front, n)), dtype=torch.uint8, device=D_)
    return lambda s: mla.project(cfg, front, x, w_q, None, None, w_qr, w_dkv, w_kr, *outs, ws, stream=s)


def _prefill(mla, n, H=2):
    cfg = mla.Config(H, 128, 512, 64, 64)
    w = lambda *s: torch.randn(*s, device=D_).bfloat16()  # noqa: E731
    pos, cu = torch.arange(n, dtype=torch.int32, device=D_), torch.tensor([0, n], dtype=torch.int32, device=D_)
    t = w(n, H, 128), w(n, H, 64), pos, w(n, 576), w(H, 128, 512), w(H, 128, 512), cu
    o, ws = w(n, H, 128), torch.zeros(mla.prefill_workspace_size(cfg, n), dtype=torch.uint8, device=D_)
    return lambda s: mla.prefill(cfg, *t, n, o, ws, stream=s)


def _tree(mla, kernel, dtype="bf16", T=3, **kw):
    c = Case(mla, 16, T, [70], dtype=dtype, kernel=kernel, **kw)
    t = c.device(mla)
    return lambda s: c.call(mla, t, stream=s)


FIRST = {
    "decode_tree": lambda m: _tree(m, 2), "decode_tree, many tokens": lambda m: _tree(m, 2, T=40),
    "decode_tree, CUDA cores": lambda m: _tree(m, 1), "absorb_query": lambda m: _absorb(m, "bf16", 4, 128, 512, 64),
    "output": lambda m: _output(m, "bf16", 4, 512), "decode": lambda m: _decode(m, 64, "bf16", 128),
    "project": lambda m: _project(m, 4, 512), "prefill": lambda m: _prefill(m, 100)}


@pytest.mark.parametrize("name", FIRST)
def test_a_threads_first_call(mla, name):
    """The thread has done nothing with CUDA before: it has no context of its own yet."""
    call, stream = FIRST[name](mla), torch.cuda.Stream()
    torch.cuda.synchronize()
    caught = []

    def run():
        try:
            call(stream.cuda_stream)
        except mla.MlaError as e:
            caught.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not caught, caught


PAIRS = {  # function of the library, two calls of it through the same kernels
    "absorb_query bf16": lambda m: (_absorb(m, "bf16", 1, 128, 512, 64), _absorb(m, "bf16", 64, 256, 512, 64)),
    "absorb_query f32": lambda m: (_absorb(m, "f32", 9, 800, 64, 32), _absorb(m, "f32", 9, 1024, 64, 32)),
    "output bf16": lambda m: (_output(m, "bf16", 1, 512), _output(m, "bf16", 64, 512)),
    "output f32": lambda m: (_output(m, "f32", 9, 800), _output(m, "f32", 9, 1024)),
    "decode_stages f32": lambda m: (_decode(m, 0), _decode(m, 128)),
    "project bf16": lambda m: (_project(m, 1, 512), _project(m, 64, 512)),
    "project f32": lambda m: (_project(m, 2, 1024, "f32"), _project(m, 2, 8192, "f32"))}


@pytest.mark.parametrize("pair", PAIRS)
def test_two_threads_at_sizes_of_their_own(mla, pair):
    """Each with its stream and buffers: no launch may depend on the other thread's. The calls' arguments
    are taken down once and the library called with them, as a C program would."""
    name = "mla_" + pair.split()[0]
    fn, args = getattr(mla.lib, name), []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for call, s in zip(PAIRS[pair](mla), streams):
        call(s)
        mla.lib.__dict__[name] = lambda *a: args.append((a, call)) or mla.MLA_OK
        try:
            call(s)
        finally:
            mla.lib.__dict__[name] = fn
    torch.cuda.synchronize()
    failed = []

    def run(a):
        for _ in range(6000):
            st = fn(*a)
            if st:
                failed.append(st)

    threads = [threading.Thread(target=run, args=(a,)) for a, _ in args]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, (len(failed), failed[0])
