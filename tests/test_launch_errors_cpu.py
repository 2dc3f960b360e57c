"""A launch that fails is reported by the call that made it and by no later one.
The C ABI's translation unit (csrc/api.cpp) is compiled here against a fake
runtime whose error word is sticky until it is read, and fake launchers whose
last step (the fold of the weight gradient, the sum of the loss) fails."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "row_wise_normalization_reduce_gb300")

FAKE = r"""
#include <cuda_runtime_api.h>
#include "nrm_internal.h"
static cudaError_t pending = cudaSuccess;
static bool fail = true;
static cudaError_t launch(bool bad) {
    if (bad) pending = cudaErrorLaunchOutOfResources;
    return bad ? cudaErrorLaunchOutOfResources : cudaSuccess;
}
extern "C" {
cudaError_t cudaGetLastError() { const cudaError_t e = pending; pending = cudaSuccess; return e; }
cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
int fake_pending() { return (int)pending; }
void fake_fail(int on) { fail = on != 0; }
}
namespace nrm {
unsigned *fault_word() { return nullptr; }
cudaError_t launch_dw_fold(const float *, float *, int64_t, int64_t, cudaStream_t) { return launch(fail); }
cudaError_t launch_loss_fold(const float *, float *, int64_t, cudaStream_t) { return launch(fail); }
cudaError_t launch_drop_bwd_f32(const DropRmsBwdArgs &, int, bool, int, cudaStream_t, Plan *, int64_t *parts) {
    *parts = 1;
    return launch(false);
}
cudaError_t launch_logit_rows_f32(const LogitArgs &, bool, bool, int, cudaStream_t, Plan *) { return launch(false); }
cudaError_t launch_logit_grad_f32(const LogitArgs &, cudaStream_t) { return launch(fail); }
}  // namespace nrm
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    cuda = next((p for p in (os.environ.get("CUDA_HOME", ""), "/usr/local/cuda")
                 if p and os.path.exists(os.path.join(p, "include", "cuda_runtime_api.h"))), None)
    if not gxx or not cuda:
        pytest.skip("g++ or the CUDA headers not found")
    d = tmp_path_factory.mktemp("fake")
    (d / "fake.cpp").write_text(FAKE)
    so = str(d / "libfake.so")
    # what the fake leaves out is never called; lazily bound, it stays unresolved
    cmd = [gxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-Wl,-z,lazy", "-I" + os.path.join(ROOT, "include"),
           "-I" + os.path.join(PKG, "csrc"), "-I" + os.path.join(cuda, "include"), os.path.join(PKG, "csrc", "api.cpp"),
           str(d / "fake.cpp"), "-o", so]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    from row_wise_normalization_reduce_gb300 import _binding
    fake = ctypes.CDLL(so, mode=os.RTLD_LAZY)

    class Rest:
        """Stands in for what the fake library does not define."""

    class Lib:
        def __getattr__(self, name):
            try:
                return getattr(fake, name)
            except AttributeError:
                return Rest()

    return _binding._declare(Lib())


OK, LAUNCH, A = 0, 9, 0x100000


def calls(lib):
    ws = lib.dropout_add_rms_bwd_workspace_size(4, 8, 0)

    def bwd(rows):
        return lib.dropout_add_rms_bwd(A, 2 * A, 3 * A, 4 * A, None, 5 * A, 6 * A, 7 * A, rows, 8, 0.1, 1, 0, None, 0, 8 * A, ws, None)

    def loss(rows):
        return lib.policy_loss(A, 2 * A, 3 * A, 4 * A, None, None, 0.2, 0.2, 0.0, 1.0, None, 5 * A, 6 * A, 7 * A, rows, 8, 0, 8 * A,
                               16, None)

    return {"dw of some rows": lambda: bwd(4), "dw of no rows": lambda: bwd(0), "loss of some rows": lambda: loss(4),
            "loss of no rows": lambda: loss(0),
            "gradient": lambda: lib.logprob_bwd(A, 2 * A, 3 * A, 4 * A, 5 * A, 4, 8, 1.0, 0, None)}


@pytest.mark.parametrize("name", ["dw of some rows", "dw of no rows", "loss of some rows", "loss of no rows", "gradient"])
def test_a_failed_launch_is_not_left_for_the_next_call(lib, name):
    call = calls(lib)[name]
    lib.fake_fail(1)
    assert call() == LAUNCH
    assert lib.fake_pending() == 0
    lib.fake_fail(0)
    assert call() == OK and lib.fake_pending() == 0
