"""What the 8-bit products leave behind where a bounded wait of theirs expires, in each of their
warps' roles: a status, no value but right ones, and a device that the next call finds as ever.

fp8_gemm.cu is built a second time with waits that say they expired (expired_products.cuh)."""
import os
import subprocess

import pytest
import torch

from expert_dispatch_gb300 import build, moe
from tests.test_gpu_fp8 import run_ffn

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def expiring(tmp_path_factory):
    """Path of the library with expiring waits in its 8-bit products."""
    build.build()
    to = tmp_path_factory.mktemp("expired")
    common = [build.nvcc(), *build.ARCH, "-Xcompiler", "-fPIC"]
    obj = str(to / "fp8_gemm.o")
    subprocess.run(common + ["-O3", "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC,
                             "-include", os.path.join(HERE, "expired_products.cuh"), "-c",
                             os.path.join(build.CSRC, "fp8_gemm.cu"), "-o", obj], check=True)
    objs = [obj if s == "fp8_gemm.cu" else os.path.join(build.BUILD, os.path.splitext(s)[0] + ".o")
            for s in build.SOURCES]
    path = str(to / "libmoe_expired.so")
    subprocess.run(common + ["-shared", "--cudart", "static", "-o", path] + objs, check=True)
    return path


# three units a block of gate/up and one or two of down, 16 blocks of 128 each; one of a block
@pytest.fixture(scope="module", params=[(2000, 2048, 2048), (90, 256, 320)], ids=["many", "one"])
def layer(request):
    T, d, I = request.param
    return run_ffn(T, d, I, 3, 2, 0)


# 0: copies, 1 and 2: products, 3: factors, 4 to 11: epilogue
@pytest.mark.parametrize("warp", [0, 1, 2, 3, 4, 7, 11])
def test_products_whose_wait_expired_end_and_say_so(expiring, monkeypatch, layer, warp):
    desc, x, off, tok, sw, W, ws, want = layer
    flags = ws[:16].view(torch.int32)

    def call(at):
        with monkeypatch.context() as m:
            m.setattr(moe, "LIB_PATH", expiring)
            m.setattr(moe, "_lib", None)
            flags.copy_(torch.tensor([0, at, 0, warp], dtype=torch.int32))
            y = torch.full_like(want, 7.0)
            moe.moe_expert_ffn_fp8(desc, x, off, tok, sw, *W, y, ws)
            torch.cuda.synchronize()
            return y, moe.moe_get_device_status(ws)

    y, status = call(-1)
    assert status == moe.MOE_OK and torch.equal(y, want)
    waits = int(flags[2])
    # copies wait only for stages that are taken a second time
    assert waits > 0 or (warp == 0 and desc.d <= 512)
    for at in sorted({0, 1, waits // 3, waits // 2, waits - 2, waits - 1} & set(range(waits))):
        y, status = call(at)
        # the epilogue waits for a block only where it has not come yet, so its waits' number varies
        came = int(flags[2]) > at
        assert came or warp >= 4 and at > 1
        assert status == (moe.MOE_ERR_TIMEOUT if came else moe.MOE_OK), at
        # the workspace holds this call's h from the call before, so rows that came out are right
        assert bool(((y == want) | (y == 7.0)).all()), at
        if at == waits - 1 and warp < 4 and desc.T == 2000:  # in the second product
            assert bool((y == 7.0).any())
        y, status = call(-1)
        assert status == moe.MOE_OK and torch.equal(y, want), at
