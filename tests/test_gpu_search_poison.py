"""The LDS-poisoning debug build run over cases of the experts' products and the beam selection, one for every kernel and
layout: a read of LDS that no thread of the launch has written would show as NaN, or as a wrong count."""
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
import test_gpu_expert_product as e, test_gpu_beam_select as b
assert L.LIB_PATH.endswith("liblapsum_ldspoison.so"), L.LIB_PATH
L.load_library()
for stored in ("in_out", "out_in"):
    for dtype in ("bf16", "fp16", "fp32"):
        e.test_ragged(L, 264, 136, stored, dtype)
    e.test_sizes_of_no_whole_16_bytes(L, 65, 127, stored, "bf16")
    e.test_one_expert(L, 65, stored)
    e.test_many_rows(L, [300, 900, 0, 511], 512, 768, stored)
    e.test_tiles_of_every_kind(L, stored)
e.test_many_experts(L, 1024)
e.test_rows_of_no_expert_are_zero(L, 128, 256)
print("ok experts", flush=True)
for vocab in (1, 511, 8193):
    for dtype in ("fp32", "bf16"):
        b.test_vocabularies(L, vocab, dtype)
b.test_constant_rows(L, 5000, 0.0)
b.test_many_ties(L, "bf16")
b.test_masked_infinite_and_nan(L)
b.test_ended_beams(L, 512)
b.test_large_vocabulary_and_long_rows(L)
print("all poison cases ok", flush=True)
'''


def test_search_with_poisoned_lds():
    if not os.path.exists(POISON):
        pytest.skip("liblapsum_ldspoison.so is not built (python __graft_entry__.py builds it)")
    env = dict(os.environ)
    env["LAPSUM_LIBRARY"] = POISON
    src = CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    res = subprocess.run([sys.executable, "-c", src], capture_output=True, text=True, timeout=300, env=env)
    print(res.stdout[-3000:])
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-4000:]
    assert "all poison cases ok" in res.stdout
