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
#include <string.h>
typedef struct { unsigned x, y, z; } dim3_;
typedef struct { dim3_ grid, block; size_t smem; } config_;  /* how cudaLaunchConfig_t begins */
int cudaGetDevice(int* d) { *d = 0; return 0; }
int cudaDeviceGetAttribute(int* v, int attr, int dev) {
  *v = attr == 16 ? atoi(getenv("FAKE_SMS")) : attr == 97 ? 232448 : 0;  /* SMs, shared memory a block may ask for */
  return 0;
}
int cudaOccupancyMaxActiveClusters(int* n, const void* f, const void* config) {
  *n = atoi(getenv("FAKE_SMS")) / 2;
  return 0;
}
int cudaFuncGetAttributes(char* a, const void* f) {  /* three sizes, the most threads, the registers */
  int regs = 255;
  memset(a, 0, 32);
  memcpy(a + 28, &regs, 4);
  return 0;
}
int cudaFuncSetAttribute(const void* f, int attr, int v) {
  printf("limit %p %d\n", f, v);
  fflush(stdout);
  return 0;
}
static int launch(const void* f, size_t smem) {
  printf("launch %p %zu\n", f, smem);
  fflush(stdout);
  return 0;
}
int __cudaGetKernel(void** k, const void* f) { *k = (void*)f; return 0; }
int __cudaLaunchKernel(void* k, dim3_ grid, dim3_ block, void** args, size_t smem, void* stream) { return launch(k, smem); }
int cudaLaunchKernelExC(const config_* c, const void* f, void** args) { return launch(f, c->smem); }
int cudaMemsetAsync(void* p, int v, size_t n, void* stream) { return 0; }
int cudaGetLastError(void) { return 0; }
static int encode(void) { return 0; }
int cudaGetDriverEntryPointByVersion(const char* name, void** f, unsigned version, unsigned long long flags, int* result) {
  *f = (void*)encode;
  *result = 0;
  return 0;
}
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
        r = subprocess.run([sys.executable, "-u", "-c", head + textwrap.dedent(code)], env=env, capture_output=True, text=True,
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


@pytest.mark.parametrize("wt,T,E,H,I,M_max", [
    ("e4m3", 640, 5, 1536, 6016, 0), ("e2m1", 768, 6, 1280, 6016, 0), ("e4m3", 640, 5, 1792, 1408, 640),
    ("e4m3", 64, 4, 1792, 1408, 64)])
def test_one_launch_ffn_splits_as_the_separate_down_product(run, wt, T, E, H, I, M_max):
    """128 rows a slot and H a multiple of 256: the separate down GEMM runs on SM pairs, not split, and the workspace has no
    room for a split.  moe_grouped_ffn runs it on single CTAs and must not split it either (5 slots + 640 / 64 = 15 chunks
    x 6 tile pairs are 90 units for 152 SMs).  With few rows a slot both are split: one more launch, the reduction."""
    out = run(152, """
        p = moe.Problem.make(T=%d, K=1, E=%d, H=%d, I=%d, M_max=%d, layout='%s', wt='%s')
        A, n, q = 4096, moe.moe_workspace_bytes(p), ctypes.byref(p)  # an address that is never followed
        print("down", lib.moe_grouped_down_gemm(q, A, A, A, A, A, A, A, A, A, n, None))
        print("ffn", lib.moe_grouped_ffn(q, A, A, A, A, A, A, A, A, A, A, A, A, A, n, None))
        """ % (T, E, H, I, M_max, "masked" if M_max else "contig", wt))
    kinds = [line.split()[0] for line in out if not line.startswith("limit")]
    launches = kinds.index("down")
    assert "down 0" in out and out[-1] == "ffn 0"
    assert launches == (1 if T * 1 / E >= 128 else 2)
    assert kinds[launches + 1:] == ["launch"] * launches + ["ffn"]


@pytest.mark.parametrize("backward", [False, True])
def test_norm_calls_never_lower_a_kernels_shared_memory_limit(run, backward):
    """One kernel serves many row lengths, and its limit is the process's: a call that lowered it to its own need would
    make a launch of another host thread fail that has set its own just before."""
    out = run(152, """
        A, F = 4096, ctypes.c_float
        for rep in range(2):
            for dtype, H in ((0, 8192), (0, 4352), (1, 8192), (1, 5632), (1, 4352), (0, 2048), (0, 1200), (0, 16384), (0, 9000)):
                a = (dtype, 5000, H, A, A, 0, None, A, A, F(1.0), F(1e-6))
                if %d:
                    n = moe.moe_block_norm_workspace_bytes(5000, H)
                    print("call", lib.moe_block_norm_backward(*a, A, A, A, A, None, A, A, A, n, None))
                else:
                    print("call", lib.moe_block_norm(*a, A, A, None))
        """ % backward)
    limit, launched = {}, set()
    for line in out:
        kind, *v = line.split()
        if kind == "limit":
            assert int(v[1]) >= limit.get(v[0], 0)
            limit[v[0]] = int(v[1])
        elif kind == "launch":
            assert int(v[1]) <= max(limit.get(v[0], 0), 48 * 1024)
            launched.add(int(v[1]))
        else:
            assert v == ["0"]
    assert len(launched) > 4  # calls of different needs


@pytest.mark.parametrize("wt", ["bf16", "e4m3", "mxfp4"])
def test_unaligned_workspace_of_a_split_product_is_refused(run, wt):
    """Partial sums of a split down product are written and read 16 bytes at a time."""
    out = run(152, """
        for I in (4096, 256):  # enough of K to split, and not
            p = moe.Problem.make(T=8, K=2, E=4, H=512, I=I, M_max=8, wt='%s')
            A, n, q = 4096, moe.moe_workspace_bytes(p), ctypes.byref(p)
            for ws in (A, A + 4):
                print("status", I, ws - A,
                      lib.moe_grouped_swiglu_gemm(q, A, A, A, A, A, A, A, A, A, ws, n, None),
                      lib.moe_grouped_down_gemm(q, A, A, A, A, A, A, A, A, ws, n, None),
                      lib.moe_grouped_ffn(q, A, A, A, A, A, A, A, A, A, A, A, A, ws, n, None),
                      lib.moe_ffn_combine(q, A, A, A, A, A, A, A, A, A, A, A, A, A, A, A, ws, n, None))
        """ % wt)
    got = {tuple(line.split()[1:3]): line.split()[3:] for line in out if line.startswith("status")}
    assert got == {("4096", "0"): ["0"] * 4, ("4096", "4"): ["0", "-2", "-2", "-2"],
                   ("256", "0"): ["0"] * 4, ("256", "4"): ["0"] * 4}
