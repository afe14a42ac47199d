"""Shared memory of the language-model launches: sizes around the 48 KB that a
kernel gets without asking."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _in_a_new_process(code):
    """A limit raised by an earlier call stays with the process, so each test brings its own."""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


ALTERNATIVES = """
import torch
import gradient_compression_sgd_gc_gb300 as gc
N, V, K = torch.cuda.get_device_properties(0).multi_processor_count + 1, {V}, {K}
x = torch.randn(N, V, generator=torch.Generator("cuda").manual_seed(V), device="cuda")
ids, lp = torch.zeros(N, dtype=torch.int32, device="cuda"), torch.empty(N, device="cuda")
ti, tl = torch.empty(N, K, dtype=torch.int32, device="cuda"), torch.empty(N, K, device="cuda")
gc.token_logprobs(x, ids, lp, top_ids=ti, top_logprobs=tl)
best = torch.topk(x, K, dim=1)
assert torch.equal(x.gather(1, ti.long()), best.values)
"""


@pytest.mark.parametrize("V,K", [(325_000, 64), (325_000, 62), (300_000, 100), (400_000, 128), (283_000, 125)])
def test_alternatives_of_long_fp32_rows(V, K):
    """More rows than SMs, so a CTA for each: its list of unit maxima and its candidates take just below 48 KB, to
    which the kernel's static memory comes."""
    _in_a_new_process(ALTERNATIVES.format(V=V, K=K))
