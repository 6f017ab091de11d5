"""The hard selections on the LDS-poisoning debug build, whose kernels set their LDS objects to 0xFF bytes at entry:
a read of LDS that no thread of the launch wrote would show as NaN or a wrong count.  The cases are those of the
selections' own tests, run in one child process that loads the debug library."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
POISON = os.path.join(ROOT, "sparse_selection_primitive_amd", "liblapsum_ldspoison.so")

CHILD = r'''
import sys
sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
import torch
import sparse_selection_primitive_amd as L
import test_gpu_cache as c, test_gpu_dispatch as d, test_gpu_route as r
assert L.LIB_PATH.endswith("liblapsum_ldspoison.so"), L.LIB_PATH
L.load_library()
for score in ("softmax", "sigmoid"):
    for shape in ((33, 60, 6), (17, 256, 8), (9, 300, 32), (2, 1024, 5)):
        r.test_shapes(L, *shape, score)
    r.test_groups(L, 256, 8, 4, 8, score); r.test_groups(L, 60, 4, 2, 6, score); r.test_groups(L, 96, 3, 3, 5, score)
    print("ok route", score, flush=True)
for tokens, k, experts in ((24, 8, 256), (777, 5, 60), (5000, 8, 256)):
    d.test_plan(L, tokens, k, experts, 0.3)
d.test_rows(L, 17, 8, 32, 64, "bf16"); d.test_rows(L, 5, 3, 8, 2056, "fp32"); d.test_rows(L, 20, 32, 64, 129, "fp16")
print("ok dispatch", flush=True)
for news, group in ((1, 4), (5, 4), (20, 2)):
    for capacity in (1, 33, 256, 1000):
        c.test_lengths(L, capacity, news, group)
c.test_long(L, 128, "bf16"); c.test_widths(L, 96, "bf16"); c.test_widths(L, 256, "fp16")
c.test_what_a_token_does_not_see_does_not_reach_it(L, 6, 3, float("nan"))
print("ok attend", flush=True)
for capacity, lengths, keep in ((65, [65, 64], 64), (2500, [2477, 2100], 1111), (10000, [10000, 9999], 2500)):
    c.test_evict_lengths(L, capacity, lengths, keep, True)
c.test_evict_accounts(L, "few", 20000, 5000); c.test_evict_accounts(L, "equal", 3000, 1500)
c.test_evict_long_row(L)
print("all poison cases ok", flush=True)
'''


def test_hard_selections_with_poisoned_lds():
    if not os.path.exists(POISON):
        pytest.skip("liblapsum_ldspoison.so is not built (python __graft_entry__.py builds it)")
    env = dict(os.environ)
    env["LAPSUM_LIBRARY"] = POISON
    src = CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    res = subprocess.run([sys.executable, "-c", src], capture_output=True, text=True, timeout=300, env=env)
    print(res.stdout[-3000:])
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-4000:]
    assert "all poison cases ok" in res.stdout
