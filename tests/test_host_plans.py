"""Host-side decisions of the calls against a stand-in for the CUDA runtime's device queries and launches: workspaces of
devices with other SM counts, and the shared-memory limits that kernels are given.  No GPU."""
import os
import shutil
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Preloaded before the library: a device of FAKE_SMS SMs, launches that only write down what they were given.
FAKE = r"""
#include <stdio.h>
#include <stdlib.h>
#include <stddef.h>
typedef struct { unsigned x, y, z; } dim3_;
int cudaGetDevice(int* d) { *d = 0; return 0; }
int cudaDeviceGetAttribute(int* v, int attr, int dev) {
  *v = attr == 16 ? atoi(getenv("FAKE_SMS")) : attr == 97 ? 232448 : 0;  /* SMs, shared memory a block may ask for */
  return 0;
}
int cudaFuncSetAttribute(const void* f, int attr, int v) {
  printf("limit %p %d %d\n", f, attr, v);
  fflush(stdout);
  return 0;
}
int cudaLaunchKernel(const void* f, dim3_ grid, dim3_ block, void** args, size_t smem, void* stream) {
  printf("launch %p %zu\n", f, smem);
  fflush(stdout);
  return 0;
}
int cudaGetLastError(void) { return 0; }
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    """run(sms, code): what a process prints that runs `code` with the library on such a device."""
    from routed_expert_layer_moe_gb300 import build
    build.build()
    cc = shutil.which("gcc")
    if not cc:
        pytest.skip("gcc is missing")
    d = tmp_path_factory.mktemp("fake")
    src, so = d / "fake.c", d / "fake.so"
    src.write_text(FAKE)
    subprocess.check_call([cc, "-shared", "-fPIC", "-O1", "-o", str(so), str(src)])

    def call(sms, code):
        env = dict(os.environ, LD_PRELOAD=str(so), FAKE_SMS=str(sms), PYTHONPATH=ROOT)
        head = "import ctypes, routed_expert_layer_moe_gb300 as moe\nlib = moe.lib()\n"
        r = subprocess.run([sys.executable, "-c", head + textwrap.dedent(code)], env=env, capture_output=True, text=True,
                           timeout=300)
        assert r.returncode == 0, r.stderr
        return r.stdout.splitlines()

    return call


STATS = 4096  # counters at the start of a workspace


@pytest.mark.parametrize("wt,sms,splits,T,K,E,H,I", [
    # 12 chunks x 20 tile pairs = 240 units a split: on 142 SMs four splits are 6.76 waves, which fill 0.966 of seven
    # (three: 5.07 of six, two: 3.38 of four)
    ("mxfp4", 142, 4, 12, 6, 12, 5120, 10624), ("mxfp4", 152, 3, 12, 6, 12, 5120, 10624),
    ("mxfp4", 160, 2, 12, 6, 12, 5120, 10624),
    # the same rule in the GEMMs of the other types: units a split 17 x 7, 26 x 5, 34 x 11, 21 x 14
    ("bf16", 140, 7, 8, 5, 17, 1664, 12160), ("bf16", 146, 10, 28, 6, 26, 1280, 4224),
    ("e4m3", 140, 4, 18, 3, 34, 2816, 4224), ("e2m1", 146, 5, 23, 4, 21, 3456, 7936)])
def test_workspace_holds_the_split_of_any_device(run, wt, sms, splits, T, K, E, H, I):
    """The splits of the down product depend on the SM count; their partial sums [splits][T K][H] are fp32."""
    out = run(sms, "print('bytes', moe.moe_workspace_bytes(moe.Problem.make(T=%d, K=%d, E=%d, H=%d, I=%d, "
                   "layout='contig', wt='%s')))" % (T, K, E, H, I, wt))
    assert int(out[-1].split()[1]) >= STATS + splits * T * K * H * 4
