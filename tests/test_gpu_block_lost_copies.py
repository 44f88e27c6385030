"""Rows of the norms whose copies into shared memory never land: every result that
such a row takes part in is NaN, not a number made from what the stage held before."""
import ctypes
import os
import subprocess

import pytest
import torch

from combine_ep_get_03_gb300 import build
from combine_ep_get_03_gb300 import ep

from test_gpu_block import Norms

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
P, I = ctypes.c_void_p, ctypes.c_int


@pytest.fixture(scope="module")
def lossy(tmp_path_factory):
    """The kernels compiled with a wait that tells all threads but one that it gave up."""
    lib = str(tmp_path_factory.mktemp("lossy") / "liblossy.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "norms_losing_copies.cu")
    cmd = [build.nvcc()] + build.ARCH + ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I", build.CSRC,
                                         "-I", os.path.join(build.ROOT, "include"), "-o", lib, src]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(lib)
    lib.lossy_forward.argtypes = [I] * 3 + [P] * 7 + [I, P]
    lib.lossy_backward.argtypes = [I] * 3 + [P] * 12 + [I, P]
    return lib


# one row a block; several rows in one block
@pytest.mark.parametrize("T,sms", [(40, 152), (2, 1)])
@pytest.mark.parametrize("H", [512, 2048, 5632, 7168])
@pytest.mark.parametrize("res", [torch.float32, torch.bfloat16])
def test_lost_rows_are_nan_in_every_result(lossy, T, sms, H, res):
    c = Norms(T, H, res, torch.float32, True, True, "none", scale=1.0)
    new, x, rstd = c.forward()
    stream = torch.cuda.current_stream().cuda_stream
    p = lambda t: t.data_ptr()  # noqa: E731
    got = [torch.zeros_like(new), torch.zeros_like(x), torch.zeros_like(rstd)]
    assert lossy.lossy_forward(T, H, res is torch.float32, p(c.post), p(c.pre), p(c.residual), p(c.y), p(got[0]),
                               p(got[1]), p(got[2]), sms, stream) == 0
    for t, name in zip(got, ("new residual", "x", "rstd")):
        assert t.isnan().all(), name
    dres, dy, dpost, dpre = torch.zeros_like(new), torch.zeros_like(c.y), torch.zeros(H, device=DEV), torch.zeros(H, device=DEV)
    ws = torch.zeros(ep.ep_block_norm_workspace_bytes(H), dtype=torch.uint8, device=DEV)
    assert lossy.lossy_backward(T, H, res is torch.float32, p(c.post), p(c.pre), p(new), p(c.y), p(rstd), p(c.dnew),
                                p(c.dx), p(dres), p(dy), p(dpost), p(dpre), p(ws), sms, stream) == 0
    for t, name in ((dres, "residual"), (dy, "y"), (dpost, "post")):
        assert t.isnan().all(), name
    # the one thread whose copies did come owns two words of eight channels at most, and
    # its sums of grad_x hn need nothing of the others
    assert (~dpre.isnan()).sum() <= 16
