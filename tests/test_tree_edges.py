"""Tree calls at sizes and inputs where they can go wrong apart from their values: limits that a launch
depends on, empty places of a padded batch, calls from two threads."""
import json
import os
import subprocess
import sys

import pytest
import torch

from tests import tree_util as tu

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
@pytest.mark.parametrize("batch", [3046, 3047, 3071, 3072])
def test_tables_where_shared_memory_passes_the_default_limit(batch):
    """In a process of its own: a larger call before would have raised the kernel's limit."""
    out = subprocess.run([sys.executable, "-c",
                          TABLES.replace("ROOT", repr(ROOT)).replace("BATCH", str(batch))],
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert json.loads(out.stdout.splitlines()[-1]) == [True] * 9
