"""GPU tests of calls made by several host threads at once: the first calls of
a process, and later ones, each on its own stream and workspace."""
import os
import subprocess
import sys

import pytest
import torch

from paged_kv_extend_gb300 import pkx

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST_CALLS = r"""
import threading, torch
from paged_kv_extend_gb300 import pkx
from paged_kv_extend_gb300 import workloads as W

N = 12
dev = torch.device("cuda:0")
wl = W.draw(W.small_spec(batch=2, prefix=[130, 5], extend=[20, 3], seed=3))
k, v = wl.pool(dev)
ke, ve = wl.extend_kv(dev)
q, qo, ptr, idx = (x.to(dev) for x in (wl.q, wl.qo_indptr, wl.kv_indptr, wl.kv_indices))
o = [torch.zeros_like(q) for _ in range(N)]
lse = [torch.zeros(q.shape[:2], device=dev) for _ in range(N)]
streams = [torch.cuda.Stream() for _ in range(N)]
ws = [torch.empty(pkx.extend_workspace_size(2, 23, 8, 2, 128, 128), dtype=torch.uint8, device=dev) for _ in range(N)]
codes = torch.randint(0, 256, (*k.shape[:2], 64), dtype=torch.uint8, device=dev)
scales = torch.full((*k.shape[:2], 8), 0x30, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
torch.cuda.synchronize()
gate, errors = threading.Barrier(N), []

def call(i):
    try:
        with torch.cuda.stream(streams[i]):
            gate.wait()
            if i % 2:
                pkx.extend_attention_fwd_streaming(q, ke, ve, o[i], k, v, qo, ptr, idx, 40, 4, wl.sm_scale,
                                                   lse=lse[i], workspace=ws[i])
            else:
                pkx.extend_attention_fwd_fp4(q, ke, ve, o[i], codes, scales, codes, scales, qo, ptr, idx,
                                             wl.sm_scale, lse=lse[i], workspace=ws[i])
    except Exception as e:
        errors.append(repr(e))

for _ in range(4):  # the first calls of the process, then later ones
    threads = [threading.Thread(target=call, args=(i,)) for i in range(N)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not errors, errors
    for i in range(2, N):
        assert torch.equal(o[i], o[i % 2]) and torch.equal(lse[i], lse[i % 2]), i
    assert o[0].any() and o[1].any() and all(pkx.workspace_status(w) == 0 for w in ws)
print("same results")
"""


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkx.load_library()


def test_first_calls_of_a_process_from_several_threads():
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same results" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("form", ["extend", "decode", "fp4"])
def test_first_cuda_call_of_a_thread(form):
    """A thread that has made no CUDA call yet."""
    import threading

    from test_gpu_fp4_extend import Case
    c = Case(128, 8, 2, [300, 5], [20, 3], 31, 0.3, 0.7)
    k, v = (x.cuda() for x in c.wl.pool())
    q = c.q[:2].contiguous()

    def run():
        o, lse = torch.zeros_like(q if form == "decode" else c.q), None
        try:
            if form == "extend":
                pkx.extend_attention_fwd(c.q, c.ke, c.ve, o, k, v, c.qo, c.ptr, c.idx, workspace=ws)
            elif form == "decode":
                pkx.decode_attention_fwd(q, o, k, v, c.ptr, c.idx, workspace=ws)
            else:
                pkx.extend_attention_fwd_fp4(c.q, c.ke, c.ve, o, *c.pool, c.qo, c.ptr, c.idx, workspace=ws)
        except Exception as e:
            outs.append(e)
        else:
            outs.append(o)

    ws = torch.empty(max(pkx.extend_workspace_size(2, 23, 8, 2, 128, 128),
                         pkx.decode_workspace_size(2, 8, 2, 128, 128)), dtype=torch.uint8, device="cuda:0")
    outs = []
    run()
    torch.cuda.synchronize()
    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert isinstance(outs[1], torch.Tensor), outs[1]
    assert outs[0].any() and torch.equal(outs[0], outs[1])


WRITES_AND_DECODES = r"""
import threading, torch
from paged_kv_extend_gb300 import pkx

N, SLOTS, HKV, D = 12, 700, 2, 128
dev = torch.device("cuda:0")
g = torch.Generator().manual_seed(4)
rows = torch.randn(300, HKV, D, generator=g).bfloat16().to(dev)
q = torch.randn(3, 8, D, generator=g).bfloat16().to(dev)
loc = torch.randperm(SLOTS, generator=g)[:300].to(dev)
idx, ptr = loc.to(torch.int32), torch.tensor([0, 120, 121, 300], dtype=torch.int32, device=dev)
pools = [[t for _ in range(2) for t in (
    torch.zeros(SLOTS, HKV, D // 2, dtype=torch.uint8, device=dev),
    torch.zeros(SLOTS, HKV, D // 16, dtype=torch.float8_e4m3fn, device=dev))] for _ in range(N)]
wide = [torch.zeros(2, SLOTS, HKV, D, dtype=torch.bfloat16, device=dev) for _ in range(N)]
o, streams = [torch.zeros_like(q) for _ in range(N)], [torch.cuda.Stream() for _ in range(N)]
back = [torch.zeros_like(rows) for _ in range(2 * N)]
space = [torch.empty(pkx.decode_fp4_workspace_size(3, 8, HKV, D, D), dtype=torch.uint8, device=dev) for _ in range(N)]
torch.cuda.synchronize()
gate, errors = threading.Barrier(N), []

def call(i):
    try:
        with torch.cuda.stream(streams[i]):
            gate.wait()
            pkx.set_kv_buffer_fp4(*pools[i], loc, rows, rows, 0.3, 0.5)
            pkx.get_kv_buffer_fp4(*pools[i], idx, 0.3, 0.5, back[2 * i], back[2 * i + 1])
            pkx.decode_attention_fwd_fp4(q, o[i], *pools[i], ptr, idx, workspace=space[i], k_scale=0.3, v_scale=0.5)
            pkx.set_kv_buffer(wide[i][0], wide[i][1], loc, rows, rows)
    except Exception as e:
        errors.append(repr(e))

for _ in range(4):
    threads = [threading.Thread(target=call, args=(i,)) for i in range(N)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not errors, errors
    for i in range(1, N):
        assert torch.equal(o[i], o[0]) and torch.equal(wide[i], wide[0]), i
        assert torch.equal(back[2 * i], back[0]) and torch.equal(back[2 * i + 1], back[1]), i
    assert o[0].any() and back[0].any() and torch.equal(wide[0][0][loc], rows)
    assert all(pkx.workspace_status(w) == 0 for w in space)
print("same results")
"""


def test_writes_and_decodes_from_several_threads():
    r = subprocess.run([sys.executable, "-c", WRITES_AND_DECODES], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "same results" in r.stdout, r.stdout + r.stderr
