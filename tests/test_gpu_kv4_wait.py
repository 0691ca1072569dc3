"""A wait for a copy into shared memory ends, whether or not the copy comes, and the lanes of a warp
can agree on it."""
import ctypes
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
MS = 1000000


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from top_selection_deepselect_gb300 import _build
    out = str(tmp_path_factory.mktemp("wait") / "libwait.so")
    subprocess.run([_build.nvcc()] + _build.NVCC_FLAGS +
                   ["-shared", "-I", _build.CSRC, "-I", _build.INCLUDE, "-o", out,
                    os.path.join(HERE, "kv4_wait_kernels.cu")], check=True)
    lib = ctypes.CDLL(out)
    lib.wait_of.argtypes = [ctypes.c_longlong] * 4 + [ctypes.c_void_p]
    return lib


@pytest.mark.parametrize("lane0,others,arrival,want", [
    (0, 0, 0, True), (0, 0, 5, True), (5, 0, 10, True), (0, 0, None, False),
    (60, 0, None, False), (0, 60, None, False),
    (60, 0, 40, None),         # the others may give up after 20 ms, lane 0 finds that it came
    (0, 60, 40, None),         # the other way round
    (60, 0, 10, True)])
def test_lanes_agree(lib, lane0, others, arrival, want):
    came = torch.full((32,), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    rc = lib.wait_of(lane0 * MS, others * MS, -1 if arrival is None else arrival * MS, 20 * MS,
                     came.data_ptr())
    assert rc == 0
    got = set(came.tolist())
    assert got in ([{0}, {1}] if want is None else [{int(want)}])
