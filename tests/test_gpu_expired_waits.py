"""What the training operators return where a bounded wait in their kernels expires: NaN,
never values made of data that had not come.

The library is built a second time with waits that say they expired (expired_waits.cuh);
every result is compared with the same call's of the library itself.
"""
import concurrent.futures
import os
import subprocess

import pytest
import torch

from expert_dispatch_gb300 import build, moe

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def rnd(shape, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.fixture(scope="module")
def expiring(tmp_path_factory):
    """Path of the library with expiring waits."""
    build.build()
    to = tmp_path_factory.mktemp("expired")
    common = [build.nvcc(), *build.ARCH, "-Xcompiler", "-fPIC"]
    replaced = ["norm.cu", "ortho.cu", "ortho_chip.cu"]

    def obj(src):
        name = os.path.splitext(src)[0] + ".o"
        if src not in replaced:
            return os.path.join(build.BUILD, name)
        subprocess.run(common + ["-O3", "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC,
                                 "-include", os.path.join(HERE, "expired_waits.cuh"), "-c",
                                 os.path.join(build.CSRC, src), "-o", str(to / name)], check=True)
        return str(to / name)

    with concurrent.futures.ThreadPoolExecutor() as ex:
        objs = list(ex.map(obj, build.SOURCES))
    path = str(to / "libmoe_expired.so")
    subprocess.run(common + ["-shared", "--cudart", "static", "-o", path] + objs, check=True)
    return path


@pytest.fixture
def on_expiring(expiring, monkeypatch):
    """f() with the binding on that library."""
    def run(f):
        with monkeypatch.context() as m:
            m.setattr(moe, "LIB_PATH", expiring)
            m.setattr(moe, "_lib", None)
            out = f()
            torch.cuda.synchronize()
        return out
    return run


def nan_rows(got, want):
    """Rows of got that are NaN throughout; every other row is want's, bit for bit."""
    gone = got.isnan().view(len(got), -1)
    all_gone = gone.all(1)
    assert bool((gone.any(1) == all_gone).all())
    assert torch.equal(got[~all_gone], want[~all_gone])
    return all_gone


# block 0 takes many rows, one group of 8 warps or several of one to four, rings of one row
# and (layer norm, bf16) of two
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(6000, 64), (2601, 520), (1301, 2048), (1300, 4096)])
def test_norm_rows_of_an_expired_wait_are_nan(on_expiring, T, d, dtype, rms):
    x, dy, g = rnd((T, d), 1, dtype), rnd((T, d), 2, dtype), rnd((d,), 3)
    kind = moe.MOE_NORM_RMS if rms else moe.MOE_NORM_LAYER
    want = moe.norm(x, g, None, kind=kind, stats=True)
    back = moe.norm_backward(dy, x, g, want[1], want[2], kind=kind)
    got = on_expiring(lambda: moe.norm(x, g, None, kind=kind, stats=True))
    gone = nan_rows(got[0], want[0])
    assert bool(gone[0]) and int(gone.sum()) < T // 20  # block 0 has a 152nd at most
    assert torch.equal(nan_rows(got[2], want[2]), gone)
    if not rms:
        assert torch.equal(nan_rows(got[1], want[1]), gone)
    dx, dg, db = on_expiring(lambda: moe.norm_backward(dy, x, g, want[1], want[2], kind=kind))
    gone = nan_rows(dx, back[0])
    assert bool(gone[0]) and int(gone.sum()) < T // 20
    assert dg.isnan().all() and (rms or db.isnan().all())


# on chip in one CTA and in a cluster, 128 x 64 tiles whole and shared by a cluster, SM pairs
@pytest.mark.parametrize("n,rows,cols", [(2, 100, 90), (3, 70, 300), (1, 128, 2048), (1, 200, 330),
                                         (1, 256, 4096), (9, 600, 1100), (3, 1000, 2500)])
def test_ortho_results_of_an_expired_wait_are_nan(on_expiring, n, rows, cols):
    g = rnd((n, rows, cols), 1, torch.bfloat16)
    want = moe.orthogonalize(g)
    desc = moe.make_ortho_desc(g)
    ws = torch.zeros(moe.moe_ortho_workspace_size(desc), dtype=torch.uint8, device="cuda")
    flags = ws[:16].view(torch.int32)

    def call(expires):
        flags.copy_(torch.tensor([0, expires, 0, 0], dtype=torch.int32))
        out = torch.full_like(want, 7.0)
        on_expiring(lambda: moe.moe_orthogonalize(desc, g, out, ws))
        return out, moe.moe_get_device_status(ws)

    out, status = call(-1)
    assert status == moe.MOE_OK and torch.equal(out, want)
    waits = int(flags[2])  # of one warp: 15 products on chip or in launches, some twice
    assert waits >= 15
    for at in (0, 1, 2, waits // 2, waits - 5, waits - 1):
        out, status = call(at)
        assert status == moe.MOE_ERR_TIMEOUT
        assert bool((out.isnan() | (out == want)).all()), at
        # in the last product only its own share is lost, in whichever matrix that lies
        assert bool(out.isnan().any() if at == waits - 1 else out[0].isnan().all()), at
    # the next call on the workspace starts anew
    out, status = call(-1)
    assert status == moe.MOE_OK and torch.equal(out, want)
