"""Argument checks of the training operators that need no GPU: every refusal comes
back before anything is launched."""
import ctypes

import pytest
import torch

from expert_dispatch_gb300 import build as moe_build
from expert_dispatch_gb300 import moe, training

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10004)


@pytest.fixture(scope="module")
def L():
    moe_build.build()
    return moe.lib()


def _layer(**kw):
    base = dict(T=8, d=64, E=4, k=2, I=64, S=1, dtype=moe.MOE_BF16)
    base.update(kw)
    return ctypes.byref(moe.make_desc(**base))


def _norm(**kw):
    base = dict(T=8, d=96, kind=moe.MOE_NORM_LAYER, dtype=moe.MOE_BF16, wdtype=moe.MOE_F32,
                eps=1e-6)
    base.update(kw)
    return ctypes.byref(moe.NormDesc(*base.values()))


@pytest.mark.parametrize("call,n_ptr", [("moe_dispatch_rows", 4),
                                        ("moe_dispatch_rows_backward", 3)])
def test_row_calls_refuse(L, call, n_ptr):
    fn = getattr(L, call)
    ok = [FAKE] * n_ptr
    for i in range(n_ptr):
        for bad in (None, ODD):
            args = list(ok)
            args[i] = bad
            assert fn(_layer(), *args, None) == moe.MOE_ERR_INVALID_ARG, (i, bad)
    assert fn(None, *ok, None) == moe.MOE_ERR_INVALID_ARG
    assert fn(_layer(k=0), *ok, None) == moe.MOE_ERR_INVALID_ARG
    assert fn(_layer(d=72), *ok, None) == moe.MOE_ERR_UNSUPPORTED
    assert fn(_layer(T=0), *[None] * n_ptr, None) == moe.MOE_OK


def test_combine_backward_refuses(L):
    fn = L.moe_combine_backward
    # dy, y_perm, expert_offsets, slot_row, topk_w, dy_perm, dtopk_w
    ok = [FAKE] * 7
    for i in range(7):
        args = list(ok)
        args[i] = ODD
        assert fn(_layer(), *args, None) == moe.MOE_ERR_INVALID_ARG, i
    for i in (0, 1, 2, 3, 4, 5):  # with dtopk_w, y_perm and topk_w are needed too
        args = list(ok)
        args[i] = None
        assert fn(_layer(), *args, None) == moe.MOE_ERR_INVALID_ARG, i
    assert fn(_layer(E=0), *ok, None) == moe.MOE_ERR_INVALID_ARG
    assert fn(_layer(T=0), *[None] * 7, None) == moe.MOE_OK


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(d=0), moe.MOE_ERR_INVALID_ARG),
    (dict(kind=2), moe.MOE_ERR_INVALID_ARG),
    (dict(dtype=5), moe.MOE_ERR_INVALID_ARG),
    (dict(wdtype=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(eps=-1e-6), moe.MOE_ERR_INVALID_ARG),
    (dict(eps=float("nan")), moe.MOE_ERR_INVALID_ARG),
    (dict(eps=float("inf")), moe.MOE_ERR_INVALID_ARG),
    (dict(d=16385), moe.MOE_ERR_UNSUPPORTED),
    (dict(T=(1 << 30) + 1), moe.MOE_ERR_UNSUPPORTED),
])
def test_norm_descriptors_refused(L, bad, status):
    n = ctypes.c_size_t(0)
    assert L.moe_norm_workspace_size(_norm(**bad), ctypes.byref(n)) == status
    assert L.moe_norm_forward(_norm(**bad), *[FAKE] * 6, None) == status
    assert L.moe_norm_backward(_norm(**bad), *[FAKE] * 9, 1 << 30, None) == status


def test_norm_workspace(L):
    n = ctypes.c_size_t(0)
    assert L.moe_norm_workspace_size(_norm(), None) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_norm_workspace_size(_norm(T=0), ctypes.byref(n)) == moe.MOE_OK and n.value == 0
    sizes = []
    for T in (1, 100, 10 ** 6, 1 << 30):
        assert L.moe_norm_workspace_size(_norm(T=T), ctypes.byref(n)) == moe.MOE_OK
        assert n.value >= 2 * 96 * 4 and n.value % 256 == 0
        sizes.append(n.value)
    assert sizes == sorted(sizes) and sizes[2] == sizes[3]  # bounded however many rows


def test_norm_forward_refuses(L):
    fn = L.moe_norm_forward
    ok = [FAKE] * 6  # x, gamma, beta, y, mean, rstd
    for i in range(6):
        args = list(ok)
        args[i] = ODD
        assert fn(_norm(), *args, None) == moe.MOE_ERR_INVALID_ARG, i
    for i in (0, 3):
        args = list(ok)
        args[i] = None
        assert fn(_norm(), *args, None) == moe.MOE_ERR_INVALID_ARG, i
    rms = dict(kind=moe.MOE_NORM_RMS)
    assert fn(_norm(**rms), FAKE, FAKE, FAKE, FAKE, None, FAKE, None) == moe.MOE_ERR_INVALID_ARG
    assert fn(_norm(**rms), FAKE, FAKE, None, FAKE, FAKE, FAKE, None) == moe.MOE_ERR_INVALID_ARG
    assert fn(_norm(T=0), *[None] * 6, None) == moe.MOE_OK


def test_norm_backward_refuses(L):
    fn = L.moe_norm_backward
    big = 1 << 30
    ok = [FAKE] * 9  # dy, x, gamma, mean, rstd, dx, dgamma, dbeta, workspace
    for i in range(8):
        args = list(ok)
        args[i] = ODD
        assert fn(_norm(), *args, big, None) == moe.MOE_ERR_INVALID_ARG, i
    for i in (0, 1, 3, 4, 5):
        args = list(ok)
        args[i] = None
        assert fn(_norm(), *args, big, None) == moe.MOE_ERR_INVALID_ARG, i
    n = ctypes.c_size_t(0)
    assert L.moe_norm_workspace_size(_norm(), ctypes.byref(n)) == moe.MOE_OK
    assert fn(_norm(), *ok, n.value - 1, None) == moe.MOE_ERR_WORKSPACE
    assert fn(_norm(), *ok[:8], None, n.value, None) == moe.MOE_ERR_WORKSPACE
    assert fn(_norm(), *ok[:8], ODD, n.value, None) == moe.MOE_ERR_WORKSPACE
    rms = dict(kind=moe.MOE_NORM_RMS)
    assert fn(_norm(**rms), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, big,
              None) == moe.MOE_ERR_INVALID_ARG  # mean
    assert fn(_norm(**rms), FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, big,
              None) == moe.MOE_ERR_INVALID_ARG  # dbeta
    # no rows and nothing to sum: nothing is launched
    assert fn(_norm(T=0), *[None] * 9, 0, None) == moe.MOE_OK


def _ortho(**kw):
    base = dict(n_mats=2, rows=96, cols=40, dtype=moe.MOE_BF16, steps=5, eps=1e-7)
    base.update(kw)
    return ctypes.byref(moe.OrthoDesc(*base.values()))


@pytest.mark.parametrize("bad,status", [
    (dict(n_mats=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(rows=0), moe.MOE_ERR_INVALID_ARG),
    (dict(cols=-4), moe.MOE_ERR_INVALID_ARG),
    (dict(dtype=2), moe.MOE_ERR_INVALID_ARG),
    (dict(steps=0), moe.MOE_ERR_INVALID_ARG),
    (dict(steps=33), moe.MOE_ERR_INVALID_ARG),
    (dict(eps=-1.0), moe.MOE_ERR_INVALID_ARG),
    (dict(eps=float("nan")), moe.MOE_ERR_INVALID_ARG),
    (dict(rows=65537), moe.MOE_ERR_UNSUPPORTED),
    (dict(cols=65537), moe.MOE_ERR_UNSUPPORTED),
    (dict(n_mats=65536), moe.MOE_ERR_UNSUPPORTED),
    (dict(n_mats=20000, cols=65536), moe.MOE_ERR_UNSUPPORTED),
])
def test_ortho_descriptors_refused(L, bad, status):
    n = ctypes.c_size_t(0)
    assert L.moe_ortho_workspace_size(_ortho(**bad), ctypes.byref(n)) == status
    assert L.moe_orthogonalize(_ortho(**bad), FAKE, ctypes.c_void_p(0x20000), FAKE, 1 << 40,
                               None) == status


def test_ortho_refuses(L):
    n = ctypes.c_size_t(0)
    assert L.moe_ortho_workspace_size(_ortho(), None) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_ortho_workspace_size(_ortho(n_mats=0), ctypes.byref(n)) == moe.MOE_OK
    assert n.value == 0
    assert L.moe_ortho_workspace_size(_ortho(), ctypes.byref(n)) == moe.MOE_OK and n.value > 0
    sizes = []
    for m, cols in ((128, 2048), (129, 2048), (2048, 129), (1536, 4096)):
        assert L.moe_ortho_workspace_size(_ortho(rows=m, cols=cols), ctypes.byref(n)) == moe.MOE_OK
        sizes.append(n.value)
    # on chip the flags are enough; else two fp16 X and three m x m matrices, padded to 64
    assert sizes[0] == 256 and sizes[1] == sizes[2]
    assert sizes[1] > 2 * 2 * 2 * 192 * 2048
    assert sizes[3] > 2 * 2 * (2 * 1536 * 4096 + 3 * 1536 ** 2)
    assert L.moe_ortho_workspace_size(_ortho(), ctypes.byref(n)) == moe.MOE_OK
    out, fn = ctypes.c_void_p(0x20000), L.moe_orthogonalize
    for g, o in ((None, out), (FAKE, None), (ODD, out), (FAKE, ODD), (FAKE, FAKE)):
        assert fn(_ortho(), g, o, FAKE, n.value, None) == moe.MOE_ERR_INVALID_ARG
    assert fn(_ortho(), FAKE, out, FAKE, n.value - 1, None) == moe.MOE_ERR_WORKSPACE
    assert fn(_ortho(), FAKE, out, None, n.value, None) == moe.MOE_ERR_WORKSPACE
    assert fn(_ortho(), FAKE, out, ODD, n.value, None) == moe.MOE_ERR_WORKSPACE
    assert fn(_ortho(n_mats=0), None, None, None, 0, None) == moe.MOE_OK


def test_binding_checks_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.norm(x)
    with pytest.raises(ValueError, match="shape"):
        moe.norm(torch.zeros(4, 2, 64))
    with pytest.raises(TypeError):
        moe.norm(torch.zeros(4, 64, dtype=torch.float64))
    with pytest.raises(ValueError, match="CUDA"):
        moe.orthogonalize(x)
    with pytest.raises(TypeError):
        moe.orthogonalize(x.half())
    with pytest.raises(ValueError, match="shape"):
        moe.make_ortho_desc(x)
    d = moe.make_desc(4, 64, 4, 2, 64)
    with pytest.raises(ValueError, match="slot_row"):
        moe.moe_dispatch_rows_backward(d, torch.zeros(8, 64), torch.zeros(4, 3), x)
    with pytest.raises(ValueError, match="topk_w"):
        moe.moe_combine_backward(d, torch.zeros(4, 64), None, torch.zeros(5), torch.zeros(4, 2),
                                 torch.zeros(4, 3), torch.zeros(8, 64), None)


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 5])
def test_sizes_beyond_the_records_fields_are_refused(n):
    """Not taken modulo 2^32: five rows of 2^32 + 5 would be computed, and no error seen."""
    x = torch.empty((n, 1), dtype=torch.bfloat16, device="meta")
    for call in (moe.make_norm_desc, moe.norm, lambda t: moe.norm_backward(t, t, None, None, None)):
        with pytest.raises(ValueError, match="32 bits"):
            call(x)
    for shape in ((n, 1, 1), (1, n, 1), (1, 1, n)):
        with pytest.raises(ValueError, match="32 bits"):
            moe.make_ortho_desc(torch.empty(shape, dtype=torch.bfloat16, device="meta"))
    with pytest.raises(ValueError, match="32 bits"):
        moe.make_ortho_desc(x[:4, None], steps=n)
    assert moe.make_norm_desc(x[:8]).T == 8 and moe.make_ortho_desc(x[:4, None]).n_mats == 4


class _Here(torch.Tensor):
    """A CPU tensor that says it lies on the current GPU."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.get_device()))

    def get_device(self):
        return 0

    def data_ptr(self):
        return 0x10000


class _Elsewhere(_Here):
    """And one on another, whose address is not to be used."""

    def get_device(self):
        return 1

    def data_ptr(self):
        raise AssertionError("its address was about to be used")


def test_tensors_of_another_device_are_refused(L, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    i32, u8, f32, bf16 = torch.int32, torch.uint8, torch.float32, torch.bfloat16
    d = moe.make_desc(4, 64, 4, 2, 64, dtype=moe.MOE_F32)
    nd = moe.make_norm_desc(torch.zeros(4, 64))
    od = moe.make_ortho_desc(torch.zeros(1, 4, 64))
    x, rows, slot, off = ((4, 64), f32), ((8, 64), f32), ((4, 2), i32), ((5,), i32)
    w, s4, s64, ws = ((4, 2), f32), ((4,), f32), ((64,), f32), ((1 << 20,), u8)
    calls = [
        (lambda *a: moe.moe_dispatch_rows(d, *a), (x, off, slot, rows)),
        (lambda *a: moe.moe_dispatch_rows_backward(d, *a), (rows, slot, x)),
        (lambda *a: moe.moe_combine_backward(d, *a), (x, rows, off, slot, w, rows, w)),
        (lambda *a: moe.moe_norm_forward(nd, *a), (x, s64, s64, x, s4, s4)),
        (lambda *a: moe.moe_norm_backward(nd, *a), (x, x, s64, s4, s4, x, s64, s64, ws)),
        (lambda *a: moe.moe_orthogonalize(od, *a), (((1, 4, 64), f32), ((1, 4, 64), bf16), ws)),
        (lambda *a: moe.norm(*a), (x, s64, s64)),
        (lambda *a: moe.orthogonalize(*a), (x,)),
        (lambda *a: training.make_plan(d, *a), (((4, 2), i32), ws)),
        (lambda r, w, o, s, e: training.combine(r, w, training.Plan(d, o, None, s), e),
         (rows, w, off, slot, x))]
    for call, shapes in calls:
        for i in range(len(shapes)):
            if call is calls[-1][0] and i == 2:
                continue  # the forward combine takes no offsets
            args = [torch.zeros(sh, dtype=t).as_subclass(_Elsewhere if j == i else _Here)
                    for j, (sh, t) in enumerate(shapes)]
            with pytest.raises(ValueError, match="current device is cuda:0"):
                call(*args)
