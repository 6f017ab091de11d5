"""As test_gpu_hard_poison, for the cases whose kernels use LDS of a size that the launch gives (the plan's counts, the
kept logits of whole caches), and for the cache operators' longer cases."""
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
import test_gpu_cache as c, test_gpu_cache_long as g, test_gpu_cache_nonfinite as f, test_gpu_dispatch as d
import test_gpu_route_far_choices as r
assert L.LIB_PATH.endswith("liblapsum_ldspoison.so"), L.LIB_PATH
L.load_library()
for tokens, k, experts in ((1, 1, 1), (128, 8, 64), (129, 8, 64), (777, 5, 60), (2048, 32, 1024)):
    d.test_plan(L, tokens, k, experts, 0.3)
d.test_plan_drops_what_names_no_expert(L)
print("ok plan", flush=True)
for capacity in (1, 31, 256, 700, 1500):
    c.test_many_short_caches(L, capacity, 3, 2, 96); c.test_many_short_caches(L, capacity, 1, 16, 128)
g.test_wide_whole_caches(L, 2, 2, "bf16")
for batch, capacity in ((2, 120), (2, 700), (130, 300)):
    for news, group in ((4, 2), (9, 4)):
        f.test_row_of_nan_gives_to_what_it_sees(L, batch, capacity, news, group)
for caches in ("few", "many"):
    for group in (4, 17, 70):
        f.test_value_that_the_newest_token_sees(L, caches, 120, group, 1)
g.test_many_new_tokens(L, 257, 3, 96, 300, [300], "bf16")
print("ok attend", flush=True)
g.test_long_rows_with_protected_entries(L, "few", 4, 512, True)
g.test_rows_past_the_preloaded_tiles(L, "", 600001, True)
print("ok evict", flush=True)
r.test_choice_by_the_bias(L, 150, 300, 20, "fp32"); r.test_choice_by_the_groups(L, 60, 4)
print("all poison cases ok", flush=True)
'''


def test_launch_sized_lds_poisoned():
    if not os.path.exists(POISON):
        pytest.skip("liblapsum_ldspoison.so is not built (python __graft_entry__.py builds it)")
    env = dict(os.environ)
    env["LAPSUM_LIBRARY"] = POISON
    src = CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    res = subprocess.run([sys.executable, "-c", src], capture_output=True, text=True, timeout=300, env=env)
    print(res.stdout[-3000:])
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-4000:]
    assert "all poison cases ok" in res.stdout
