"""The compiled binding around the C entries: what it holds and which device it has made current
while it calls them.  The entries are stand-ins that launch nothing."""
import ctypes
import os
import subprocess
import threading
import time

import pytest
import torch

import mamba_ssd_scan_03_b200 as ssd
from test_gpu_served import i32

pytestmark = pytest.mark.gpu

STAND_INS = r"""
#include <dlfcn.h>
#include <stddef.h>
#include <unistd.h>
static volatile int go, device = -1;
void set_go(int v) { go = v; }
int queried_on(void) { int d = device; device = -1; return d; }
static void note(void) {
  void* cuda = dlopen("libcuda.so.1", RTLD_NOW | RTLD_NOLOAD);
  int (*get)(int*) = (int (*)(int*))(cuda ? dlsym(cuda, "cuCtxGetDevice") : NULL);
  int d = -1;
  if (get && get(&d) == 0) device = d;
}
int ssd_conv_silu_step(void) {  /* SSD_OK when another thread says go within five seconds */
  for (int k = 0; k < 5000 && !go; ++k) usleep(1000);
  return go ? 0 : 4;
}
size_t ssd_selective_varlen_workspace_size(void) { note(); return 256; }
size_t ssd_group_norm_gate_bwd_workspace_size(void) { note(); return 256; }
int ssd_conv_silu_varlen(void) { return 0; }
int ssd_selective_scan_varlen(void) { return 0; }
int ssd_selective_step(void) { return 0; }
int ssd_group_norm_gate(void) { return 0; }
int ssd_group_norm_gate_bwd(void) { return 0; }
"""


@pytest.fixture
def stand_ins(tmp_path):
    src, lib = tmp_path / "stand_ins.c", str(tmp_path / "stand_ins.so")
    src.write_text(STAND_INS)
    subprocess.run([os.environ.get("CC", "gcc"), "-shared", "-fPIC", str(src), "-ldl", "-o", lib],
                   check=True)
    w = torch.ones(8, device="cuda")
    ssd.group_norm_gate(torch.ones(1, 8, device="cuda"), w)  # the binding is loaded
    fake = ctypes.CDLL(lib)
    ssd._served.bind(lib)
    yield fake
    ssd._served.bind(ssd.LIB_PATH)
    assert torch.all(ssd.group_norm_gate(torch.ones(1, 8, device="cuda"), w) > 0.99)


def test_other_threads_run_during_a_call(stand_ins):
    """A launch can wait for room in the driver's queue; other Python threads go on meanwhile, those
    among them that the GPU's work may be waiting for."""
    def later():
        time.sleep(0.1)
        stand_ins.set_go(1)

    cs, u = torch.zeros(2, 3, 8, device="cuda"), torch.zeros(2, 8, device="cuda")
    w = torch.zeros(8, 4, device="cuda")
    other = threading.Thread(target=later)
    other.start()
    try:
        assert ssd.conv_silu_step(cs, u, w).shape == (2, 8)
    finally:
        other.join()


def test_workspace_is_sized_on_the_tensors_device(stand_ins):
    """Plans follow the current device's SMs: the query comes from the tensors' device, whatever device
    is current (with one GPU they are the same)."""
    last = torch.cuda.device_count() - 1
    with torch.cuda.device(last):
        y, w = torch.ones(4, 8, device="cuda"), torch.ones(8, device="cuda")
        A, B, cu = torch.ones(8, 16, device="cuda"), torch.ones(4, 1, 16, device="cuda"), i32([0, 4])
    with torch.cuda.device(0):
        ssd.selective_scan_varlen(y, y, A, B, B, cu)
        assert stand_ins.queried_on() == last
    with torch.cuda.device(0):
        ssd.group_norm_gate_bwd(y, y, w)
        assert stand_ins.queried_on() == last
        assert torch.cuda.current_device() == 0


def test_threads_call_at_once():
    """Four threads, each on a stream of its own, at the same time:
    convolution, scan in chunks, norm and gradients give what one thread gets."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    u, w, raw, B = rand(700, 64), rand(64, 4), rand(700, 64), rand(700, 1, 16)
    A, z, nw, cu = -torch.exp(rand(64, 16)), rand(700, 64), rand(64), i32([0, 690, 700])
    state = rand(2, 64, 16)
    torch.cuda.synchronize()

    def block():
        st = state.clone()
        x = ssd.conv_silu_varlen(u, w, cu)
        y = ssd.selective_scan_varlen(x, raw, A, B, B, cu, z=z, softplus=True, state=st)
        y1 = ssd.selective_step(st, x[:2], raw[:2], A, B[:2], B[:2], softplus=True)
        n = ssd.group_norm_gate(y, nw, None, z, 4)
        g = ssd.group_norm_gate_bwd(n, y, nw, None, z, 4)
        return [x, y, st, y1, n, g["y"], g["z"], g["weight"]]

    got = [[] for _ in range(4)]

    def work(k):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got[k].append(block())
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    want = block()
    assert [len(r) for r in got] == [20] * 4
    for r in got:
        for one in r:
            assert all(torch.equal(a, b) for a, b in zip(one, want))
    assert ssd.device_status() == 0
