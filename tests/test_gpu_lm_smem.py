"""Shared memory of the language-model launches: sizes around the 48 KB that a
kernel gets without asking, and calls of two host threads that need different
sizes."""
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


TWO_THREADS = """
import threading
import torch
import gradient_compression_sgd_gc_gb300 as gc

def call(V, stream):
    T, D = 16, 8
    dout, out = torch.ones(T, D, device="cuda"), torch.empty(V, D, device="cuda")
    ids = torch.arange(T, device="cuda")
    ws = torch.empty(gc.embed_grad_workspace_bytes(T, V, D), dtype=torch.uint8, device="cuda")
    return out, gc.embed_grad(dout, ids, out, ws, stream=stream, prepare=True)

def call_top(V, K, stream):
    N = torch.cuda.get_device_properties(0).multi_processor_count + 1
    x = torch.randn(N, V, device="cuda")
    ids = torch.zeros(N, dtype=torch.int32, device="cuda")
    lp, tl = torch.empty(N, device="cuda"), torch.empty(N, K, device="cuda")
    ti = torch.empty(N, K, dtype=torch.int32, device="cuda")
    return ti, gc.token_logprobs(x, ids, lp, top_ids=ti, top_logprobs=tl, stream=stream, prepare=True)

streams = [torch.cuda.Stream() for _ in range(2)]
pair = [{calls}]
torch.cuda.synchronize()
errors = []

def many(prepared, stream):
    try:
        for k in range({times}):
            prepared()
            if k % 64 == 63:
                stream.synchronize()
    except Exception as e:
        errors.append(repr(e))

threads = [threading.Thread(target=many, args=(c, s)) for (_, c), s in zip(pair, streams)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not errors, errors
"""


def test_table_gradients_of_two_host_threads():
    """Tables of different sizes need different amounts of shared memory; neither call takes the other's away."""
    _in_a_new_process(TWO_THREADS.format(calls="call(131_072, streams[0]), call(1000, streams[1])", times=20_000))


def test_alternatives_of_two_host_threads():
    _in_a_new_process(TWO_THREADS.format(calls="call_top(400_000, 128, streams[0]), call_top(380_000, 64, streams[1])",
                                         times=400))
