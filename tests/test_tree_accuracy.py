"""mla_decode_tree's bf16 outputs bounded by norm, per token and head: at 1000 to 40,000 rows the sum of all
terms' sizes, which an element's worst case is relative to, is many times the output itself, so that a bound
by it passes zeros. Here the roundings count as what they are, independent of each other.

The bound. With exact weights p_j and u_j = W_UV v_j the call returns sum_j p_j (1 + d_j) u_j, rounded to
bf16. d_j is the rounding of the weight to bf16 on the tensor cores, 2^-8 at most (0 on CUDA cores, whose
weights are fp32). Their signs are independent, so the sum's error has a squared norm of at most
2^-16 S^2, S^2 = sum_j p_j^2 |u_j|^2, on average; a rounding's own root mean square is 0.41 of its largest,
so that 2 * 2^-8 S is five times what is expected, and the largest there can be with up to four terms. The
output's rounding adds 2^-8 |o|. The rest is below 2^-13 S: the latent sum's two bf16 terms leave 2^-16; a
score's sum of 576 products is off by about sqrt(576) 2^-23 of the score (some units here), 3e-6 of a weight;
the sums over up to 40,000 rows and 512 dims by sqrt(n) 2^-23, 2.4e-5."""
import pytest
import torch

from tests import tree_util as tu
from tests.test_tree_attention import Case

GPU = pytest.mark.gpu


def attend(q, rows, seen, w_uv, r, scale, device="cpu"):
    """One sequence in 64 bits: o (T, H, d_v), S (T, H), and the weights p (T, H, L)."""
    q, rows, w_uv = (x.to(device).double() for x in (q, rows, w_uv))
    T, L = q.shape[0], rows.shape[0]
    vis = torch.ones((T, L), dtype=torch.bool, device=device)
    vis[:, L - T:] = seen.to(device)
    s = torch.einsum("thd,jd->thj", q, rows) * scale
    p = torch.softmax(torch.where(vis[:, None], s, -torch.inf), -1)
    o = torch.einsum("hvr,thr->thv", w_uv, torch.einsum("thj,jr->thr", p, rows[:, :r]))
    size = [(p[:, h] ** 2) @ (rows[:, :r] @ w_uv[h].T).pow(2).sum(1) for h in range(q.shape[1])]
    return o, torch.stack(size, 1).sqrt(), p


def bound(o, S, bf16_weights):
    return (2 * 2.0 ** -8 * S if bf16_weights else 0.0) + 2.0 ** -8 * o.norm(dim=-1) + 2.0 ** -13 * S


def off(got, want, S, bf16_weights):
    """The largest error over its bound."""
    return float(((got.double() - want).norm(dim=-1) / bound(want, S, bf16_weights)).max())


@pytest.mark.parametrize("L,H,T", [(1000, 6, 3), (4000, 4, 3), (40000, 3, 2)])
def test_the_bound_tells_mistakes_from_roundings(L, H, T):
    """On the CPU, mistakes planted in the 64-bit form; the bound by element passes some of them."""
    g = torch.Generator().manual_seed(L)
    q = torch.randn(T, H, 576, generator=g)
    q[..., :512] *= 0.5
    rows = torch.randn(L, 576, generator=g).bfloat16()
    w = (torch.randn(H, 128, 512, generator=g) / 512 ** 0.5).bfloat16()
    seen = tu.seen_of(tu.parents_of("chain", 1, T))[0]
    o, S, p = attend(q.bfloat16(), rows, seen, w, 512, 192 ** -0.5)
    lat = lambda x: torch.einsum("hvr,thr->thv", w.double(), x)  # noqa: E731
    v = rows[:, :512].double()
    top = p.amax(-1, keepdim=True)
    rounded = (p / top).bfloat16().double() * top
    good = lat(torch.einsum("thj,jr->thr", rounded, v)).bfloat16()
    assert off(good, o, S, True) <= 1
    assert off(o.bfloat16(), o, S, False) <= 1
    lost = p.clone()
    lost[..., L // 2:L // 2 + L // 64] = 0           # a piece of the rows left out of the merge
    lost /= lost.sum(-1, keepdim=True)
    twice = p.clone()
    twice[..., :L // 64] *= 2                        # ... or counted twice
    twice /= twice.sum(-1, keepdim=True)
    shifted = torch.einsum("thj,jr->thr", p, v.roll(1, 0))
    for wrong in (torch.zeros_like(o), o.roll(1, 1), o.roll(1, 0), lat(torch.einsum("thj,jr->thr", lost, v)),
                  lat(torch.einsum("thj,jr->thr", twice, v)), lat(shifted), o.roll(1, 2)):
        assert off(wrong, o, S, True) > 1.5
    if L == 40000:
        _, _, size, dot = tu.attend(q.bfloat16(), rows, seen, w, 512, 192 ** -0.5)
        tol, _ = tu.tolerances(torch.bfloat16, o, size, dot, 576, L)
        assert (o.abs() <= tol).all()                # zeros pass there


CASES = [  # up to 32 tokens the output kernel merges, above a kernel of its own
    dict(H=128, T=4, lens=[1000]), dict(H=128, T=1, lens=[4000, 64, 1]), dict(H=16, T=5, lens=[40000]),
    dict(H=128, T=2, lens=[40000]), dict(H=16, T=40, lens=[4000, 1000]), dict(H=64, T=17, lens=[1000, 4000, 900]),
    dict(H=3, T=7, lens=[4000] * 6, dv=33), dict(H=32, T=3, lens=[1000] * 40, bs=128),
    dict(H=128, T=9, lens=[4000, 0, 9, 2500])]


SMALL = [k for k in CASES if max(k["lens"]) <= 4000 and k["H"] * len(k["lens"]) <= 300]  # for CUDA cores


@GPU
@pytest.mark.parametrize("kernel,kw", [(2, k) for k in CASES] + [(1, k) for k in SMALL],
                         ids=lambda k: k if isinstance(k, int) else
                         f"H{k['H']}-T{k['T']}-B{len(k['lens'])}-L{k['lens'][0]}")
def test_outputs_by_norm(kernel, kw):
    import mla_latent_kv_44_b200 as mla

    c = Case(mla, kernel=kernel, seed=9, **kw)
    t = c.device(mla)
    c.call(mla, t)
    assert int(t["err"]) == 0
    for b, n in enumerate(c.lens):
        at = slice(b * c.T, (b + 1) * c.T)
        if n == 0:
            assert (t["o"][at] == 0).all()
            continue
        o, S, _ = attend(c.q[at], c.rows(b), c.seen[b], c.w_uv, c.r, c.scale, "cuda")
        e = off(t["o"][at], o, S, kernel == mla.DECODE_TENSOR)
        assert e <= 1, (b, n, e)
