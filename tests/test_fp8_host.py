"""Argument checks of the 8-bit, SwiGLU and gate calls that need no GPU: every refusal comes
back before anything is launched."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from expert_dispatch_gb300 import build as moe_build
from expert_dispatch_gb300 import moe, training
from tests.test_training_host import FAKE, ODD, _Elsewhere, _Here

BAD, UNSUP, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_OK


@pytest.fixture(scope="module")
def L():
    moe_build.build()
    return moe.lib()


def _layer(**kw):
    base = dict(T=8, d=64, E=4, k=2, I=64, S=1, dtype=moe.MOE_BF16)
    base.update(kw)
    return moe.make_desc(**base)


def _w(q=FAKE, scale=FAKE):
    return ctypes.byref(moe.Fp8WeightStruct(q, scale))


def each_bad(args, needed, optional=()):
    """args with one pointer missing or misaligned."""
    for i in needed + tuple(optional):
        for bad in (None, ODD):
            if bad is None and i in optional:
                continue
            yield [bad if j == i else a for j, a in enumerate(args)]


def test_quantize_fp8_refuses(L):
    fn = L.moe_quantize_fp8
    for n, r, k, dt in ((-1, 4, 4, 0), (1, 0, 4, 0), (1, 4, 0, 0), (1, 4, 4, 2)):
        assert fn(n, r, k, dt, FAKE, FAKE, FAKE, None) == BAD
    for args in each_bad([FAKE] * 3, (0, 1, 2)):
        assert fn(1, 4, 4, 0, *args, None) == BAD
    assert fn(1 << 20, 1 << 20, 128, 0, FAKE, FAKE, FAKE, None) == UNSUP
    assert fn((1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1, 0, FAKE, FAKE, FAKE, None) == UNSUP
    assert fn(0, 4, 4, 0, None, None, None, None) == OK


def test_expert_ffn_and_layer_refuse(L):
    d = _layer()
    n = moe.moe_workspace_size(d)
    by = ctypes.byref(d)
    ptrs = [FAKE] * 4  # x, offsets, token_indices, slot_w
    call = lambda p, w=(_w(), _w(), _w()), y=FAKE, ws=FAKE, b=n, desc=by: \
        L.moe_expert_ffn_fp8(desc, *p, *w, y, ws, b, None)  # noqa: E731
    for p in each_bad(ptrs, (0, 1, 2), (3,)):
        assert call(p) == BAD
    for i in range(3):
        for bad in (None, _w(None), _w(FAKE, None), _w(ODD), _w(FAKE, ODD)):
            assert call(ptrs, [bad if j == i else _w() for j in range(3)]) == BAD
    assert call(ptrs, y=None) == BAD and call(ptrs, y=ODD) == BAD
    assert call(ptrs, ws=None) == moe.MOE_ERR_WORKSPACE
    assert call(ptrs, b=n - 1) == moe.MOE_ERR_WORKSPACE
    assert call(ptrs, desc=ctypes.byref(_layer(dtype=moe.MOE_F32))) == UNSUP
    assert call(ptrs, desc=ctypes.byref(_layer(d=96))) == UNSUP
    assert call(ptrs, desc=None) == BAD
    assert call([None] * 4, [None] * 3, None, None, 0, ctypes.byref(_layer(T=0))) == OK

    def fwd(x=FAKE, wr=FAKE, lb=None, sb=None, w=None, res=None, y=FAKE, ids=None, tw=None,
            desc=by, b=n):
        w = w or [_w()] * 3
        return L.moe_layer_forward_fp8(desc, x, wr, lb, sb, *w, res, y, ids, tw, FAKE, b, None)

    for kw in (dict(x=None), dict(x=ODD), dict(wr=None), dict(wr=ODD), dict(y=None), dict(y=ODD),
               dict(res=ODD), dict(ids=ODD), dict(tw=ODD), dict(sb=FAKE),
               dict(w=[_w(), None, _w()])):
        assert fwd(**kw) == BAD, kw
    assert fwd(b=n - 1) == moe.MOE_ERR_WORKSPACE
    assert fwd(desc=ctypes.byref(_layer(dtype=moe.MOE_F32))) == UNSUP
    for fn in (L.moe_layer_forward_fp8_host,):
        assert fn(by, None, FAKE, None, None, _w(), _w(), _w(), None, FAKE, None, None, FAKE, n,
                  None) == BAD
    assert L.moe_layer_forward_fp8_host_pipelined(by, -1, FAKE, FAKE, None, None, _w(), _w(), _w(),
                                                  FAKE, FAKE, n, None) == BAD


def test_rows_and_swiglu_refuse(L):
    for fn in (L.moe_pack_rows, L.moe_unpack_rows):
        ptrs = [FAKE, ctypes.c_void_p(0x20000), ctypes.c_void_p(0x30000)]
        for r, n, dt in ((-1, 4, 0), (4, 0, 0), (4, 4, 3)):
            assert fn(r, n, dt, *ptrs, None) == BAD
        for args in each_bad(ptrs, (0, 1, 2)):
            assert fn(4, 4, 0, *args, None) == BAD
        assert fn(0, 4, 0, None, None, None, None) == OK
    p = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(10)]
    fwd, bwd = L.moe_swiglu_forward, L.moe_swiglu_backward
    for r, n, dt in ((-1, 4, 0), (4, 0, 0), (4, 4, 3)):
        assert fwd(r, n, dt, *p[:7], None) == BAD and bwd(r, n, dt, *p, None) == BAD
    for args in each_bad(p[:7], (0, 1, 2, 3, 4, 5, 6)):  # a part of the 8-bit outputs is refused
        assert fwd(4, 4, 0, *args, None) == BAD
    for args in ([p[0], p[1], p[0]], [p[0], p[1], p[1]]):  # h over an input
        assert fwd(4, 4, 0, *args, None, None, None, None, None) == BAD
    # dh, gate, up, gate8, gate_scale, up8, up_scale, dgate, dup, h
    plain = [p[0], p[1], p[2], None, None, None, None, p[7], p[8], p[9]]
    packed = [p[0], None, None, p[3], p[4], p[5], p[6], p[7], p[8], p[9]]
    for args in each_bad(plain, (0, 1, 2, 7, 8), (9,)):
        assert bwd(4, 4, 0, *args, None) == BAD
    for args in each_bad(packed, (0, 3, 4, 5, 6, 7, 8), (9,)):
        assert bwd(4, 4, 0, *args, None) == BAD
    assert bwd(4, 4, 0, *p, None) == BAD  # both forms at once
    for i, j in ((7, 8), (9, 7), (9, 8), (7, 0), (8, 1), (9, 2)):  # outputs over one another
        args = list(plain)
        args[i] = args[j]
        assert bwd(4, 4, 0, *args, None) == BAD
    assert bwd(0, 4, 0, *[None] * 10, None) == OK
    assert fwd(0, 4, 0, *[None] * 7, None) == OK


def test_products_are_not_launched_on_too_few_registers(tmp_path):
    """The warps of the products share the registers that the block was launched with, unevenly:
    72 for each thread of four warps, 216 of eight, of 384 times 168.  A kernel that another
    compiler gave fewer would wait for the missing ones without a limit, so it is refused
    before its launch.  The launcher runs on a runtime of its own (fake_launches.cuh)."""
    lib = str(tmp_path / "fake.so")
    subprocess.run([moe_build.nvcc(), *moe_build.ARCH, "-std=c++17", "-I", moe_build.INCLUDE, "-I",
                    moe_build.CSRC, "-Xcompiler", "-fPIC", "-include",
                    os.path.join(os.path.dirname(__file__), "fake_launches.cuh"), "-shared",
                    "--cudart", "static", "-o", lib,
                    os.path.join(moe_build.CSRC, "fp8_gemm.cu")], check=True)
    n = ctypes.c_int(-1)
    # registers come in steps of 8: 161 are 168
    for regs, fine in ((160, False), (128, False), (64, False), (217, False), (161, True),
                       (168, True)):
        run = ctypes.CDLL(shutil.copy(lib, str(tmp_path / ("%d.so" % regs)))).fake_products
        for _ in range(2):  # a refusal is not forgotten
            status = run(regs, ctypes.byref(n))
            assert (status, n.value) == ((0, 2) if fine else (9, 0)), regs


def test_outputs_that_overlap_an_input_or_another_output_are_refused(L):
    """By their ranges: 40 rows of 100, a buffer's first 16 bytes in the other's last."""
    def places(*sizes):
        return [0x1000000 * (i + 1) for i in range(len(sizes))]

    def pairs(call, sizes, outputs):
        """call with one output moved onto every other buffer: at its start, onto its end."""
        at = places(*sizes)
        for o in outputs:
            for j in range(len(sizes)):
                if j == o:
                    continue
                last = (sizes[j] - 1) // 16 * 16  # the last 16-byte address within it
                for to in {at[j], at[j] + last, at[j] - (sizes[o] - 1) // 16 * 16}:
                    args = [ctypes.c_void_p(to if i == o else a) for i, a in enumerate(at)]
                    assert call(args) == BAD, (o, j, hex(to))

    for es, dt in ((4, moe.MOE_F32), (2, moe.MOE_BF16)):
        full, codes, scales = 4000 * es, 4000, 40 * 4
        # x, q, scale
        pairs(lambda a: L.moe_pack_rows(40, 100, dt, *a, None), [full, codes, scales], (1, 2))
        # q, scale, x
        pairs(lambda a: L.moe_unpack_rows(40, 100, dt, *a, None), [codes, scales, full], (2,))
        # w, q, scale
        pairs(lambda a: L.moe_quantize_fp8(2, 20, 100, dt, *a, None), [full, codes, 8], (1, 2))
        # gate, up, h, gate8, gate_scale, up8, up_scale
        pairs(lambda a: L.moe_swiglu_forward(40, 100, dt, *a, None),
              [full] * 3 + [codes, scales] * 2, (2, 3, 4, 5, 6))
        pairs(lambda a: L.moe_swiglu_forward(40, 100, dt, *a, None, None, None, None, None),
              [full] * 3, (2,))
        # dh, gate, up, dgate, dup, h and dh, gate8, gate_scale, up8, up_scale, dgate, dup, h
        pairs(lambda a: L.moe_swiglu_backward(40, 100, dt, *a[:3], *[None] * 4, *a[3:], None),
              [full] * 6, (3, 4, 5))
        pairs(lambda a: L.moe_swiglu_backward(40, 100, dt, a[0], None, None, *a[1:], None),
              [full] + [codes, scales] * 2 + [full] * 3, (5, 6, 7))


def test_gate_refuses(L):
    n = ctypes.c_size_t(0)
    d = _layer()
    by = ctypes.byref(d)
    assert L.moe_gate_workspace_size(by, None) == BAD
    assert L.moe_gate_workspace_size(ctypes.byref(_layer(k=9)), ctypes.byref(n)) == BAD
    assert L.moe_gate_workspace_size(ctypes.byref(_layer(T=0)), ctypes.byref(n)) == OK
    assert n.value == 0
    assert L.moe_gate_workspace_size(by, ctypes.byref(n)) == OK and n.value % 256 == 0
    fwd, bwd = L.moe_gate_forward, L.moe_gate_backward
    ok = [FAKE] * 6  # logits, ids, w, counts, prob, loss
    for args in each_bad(ok, (0, 1), (2, 3, 4, 5)):
        assert fwd(by, 0, *args, FAKE, n.value, None) == BAD
    assert fwd(by, 2, *ok, FAKE, n.value, None) == BAD
    assert fwd(None, 0, *ok, FAKE, n.value, None) == BAD
    for ws, b in ((None, n.value), (ODD, n.value), (FAKE, 16)):
        assert fwd(by, 0, *ok, ws, b, None) == moe.MOE_ERR_WORKSPACE
    assert fwd(ctypes.byref(_layer(T=0)), 0, *[None] * 6, None, 0, None) == OK
    out = ctypes.c_void_p(0x90000)
    ok = [FAKE] * 5 + [out]  # logits, ids, counts, dw, dloss, dlogits
    for args in each_bad(ok, (0, 1, 5), (2, 3, 4)):
        assert bwd(by, 0, *args, None) == BAD
    assert bwd(by, 0, FAKE, FAKE, None, FAKE, FAKE, out, None) == BAD  # a loss without counts
    assert bwd(by, 0, out, FAKE, FAKE, FAKE, FAKE, out, None) == BAD   # over the logits
    assert bwd(by, 5, *ok, None) == BAD
    assert bwd(ctypes.byref(_layer(T=0)), 0, *[None] * 6, None) == OK


def test_binding_checks(monkeypatch):
    x, q = torch.zeros(4, 130), torch.zeros(4, 130, dtype=moe.FP8)
    s = torch.zeros(4, 2)
    r = moe.Rows8(q, s)
    assert r.shape == (4, 130)
    for bad in ((x, s), (q, s.double()), (q, s[:, :1]), (q[0], s)):
        with pytest.raises((TypeError, ValueError)):
            moe.Rows8(*bad)
    for bad in ((q, s), (q[None], s), (q[None], s[None].half())):
        with pytest.raises((TypeError, ValueError)):
            moe.Fp8Weight(*bad)
    assert moe.Fp8Weight(q[None], torch.zeros(1, 1, 2)).shape == (1, 4, 130)
    for call in (lambda: moe.pack_rows(x), lambda: moe.unpack_rows(r), lambda: moe.swiglu(x, x),
                 lambda: moe.swiglu_backward(x, x, x), lambda: moe.quantize_fp8(x[None])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        moe.pack_rows(x.half())
    with pytest.raises(ValueError, match="shape"):
        moe.pack_rows(x[0])
    with pytest.raises(ValueError, match="up"):
        moe.swiglu(x, x[:2])
    with pytest.raises(ValueError, match="32 bits"):
        moe.pack_rows(torch.empty((1 << 32, 1), dtype=torch.bfloat16, device="meta"))
    d = moe.make_desc(4, 64, 4, 2, 64)
    with pytest.raises(ValueError, match="logits"):
        moe.gate(d, x, torch.zeros(4, 2, dtype=torch.int32))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="Fp8Weight"):
        moe.moe_expert_ffn_fp8(d, _here((4, 64), torch.bfloat16), _here((5,), torch.int32),
                               _here((8,), torch.int32), None, x, x, x,
                               _here((8, 64), torch.bfloat16), None)


def test_training_swiglu_compares_shapes_before_it_flattens_rows(monkeypatch):
    """Tensors of other shapes are refused, also where their rows would fit in flattened order."""
    monkeypatch.setattr(moe, "swiglu", lambda *a, **kw: pytest.fail("it came to the call"))
    for a, b in (((2, 3, 8), (3, 2, 8)), ((6, 8), (1, 2, 3, 8)), ((1, 8), (8,)), ((2, 8), (1, 8)),
                 ((2, 8), (2, 4))):
        for packed in (True, False):
            with pytest.raises(ValueError, match="up has shape"), torch.no_grad():
                training.swiglu(torch.zeros(a), torch.zeros(b), packed)


def test_calls_with_the_callers_buffers_refuse(L, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    f32, bf16, f8 = torch.float32, torch.bfloat16, moe.FP8
    x, q, s = ((4, 130), bf16), ((4, 130), f8), ((4, 2), f32)
    R = moe.Rows8
    calls = [
        (moe.moe_pack_rows, (x, q, s)),
        (moe.moe_unpack_rows, (q, s, x)),
        (moe.moe_swiglu_forward, (x, x, x)),
        (lambda g, u, h, a, b, c, d: moe.moe_swiglu_forward(g, u, h, R(a, b), R(c, d)),
         (x, x, x, q, s, q, s)),
        (moe.moe_swiglu_backward, (x, x, x, x, x, x)),
        (lambda dh, a, b, c, d, e, f, h: moe.moe_swiglu_backward(dh, R(a, b), R(c, d), e, f, h),
         (x, q, s, q, s, x, x, x))]
    for call, shapes in calls:
        for i, (shape, dtype) in enumerate(shapes):
            def args(sh, t, cls=_Here):
                return [_here(sh, t, cls) if j == i else _here(*a) for j, a in enumerate(shapes)]

            with pytest.raises(ValueError, match="current device is cuda:0"):
                call(*args(shape, dtype, _Elsewhere))
            for bad in ((shape[0] + 1, shape[1]), (shape[0], shape[1] - 1), shape[:1]):
                with pytest.raises(ValueError, match="shape"):
                    call(*args(bad, dtype))
            with pytest.raises(TypeError):
                call(*args(shape, torch.float16))
            with pytest.raises(ValueError, match="contiguous"):
                a = args(shape, dtype)
                a[i] = torch.zeros(shape[::-1], dtype=dtype).t().as_subclass(_Here)
                call(*a)
    t, r = _here(*x), R(_here(*q), _here(*s))
    with pytest.raises(ValueError, match="both or neither"):
        moe.moe_swiglu_forward(t, t, t, r)
    for g, u in ((r, t), (t, r)):
        with pytest.raises(TypeError):
            moe.moe_swiglu_backward(t, g, u, t, t)


def _here(shape, dtype, cls=_Here):
    return torch.zeros(shape, dtype=dtype).as_subclass(cls)


def test_tensors_of_another_device_are_refused(L, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    i32, u8, f32, bf16, f8 = torch.int32, torch.uint8, torch.float32, torch.bfloat16, moe.FP8
    d = moe.make_desc(4, 64, 4, 2, 64)
    ws = ((1 << 20,), u8)
    w3, s3 = ((4, 64, 64), f8), ((4, 1, 1), f32)
    x, rows = ((4, 64), bf16), ((8, 64), bf16)
    r8, rs = ((4, 64), f8), ((4, 1), f32)
    lg, ids, tw = ((4, 4), f32), ((4, 2), i32), ((4, 2), f32)

    def ffn(x, off, tok, sw, a, b, c, e, f, g, y, w):
        W = moe.Fp8Weight
        moe.moe_expert_ffn_fp8(d, x, off, tok, sw, W(a, b), W(c, e), W(f, g), y, w)

    def fwd(x, wr, a, b, c, e, f, g, res, y, i, t, w):
        W = moe.Fp8Weight
        moe.moe_layer_forward_fp8(d, x, wr, None, None, W(a, b), W(c, e), W(f, g), res, y, i, t, w)

    calls = [
        (ffn, (x, ((5,), i32), ((8,), i32), ((8,), f32), w3, s3, w3, s3, w3, s3, rows, ws)),
        (fwd, (x, x, w3, s3, w3, s3, w3, s3, ((4, 64), f32), ((4, 64), f32), ids, tw, ws)),
        (moe.moe_quantize_fp8, (((1, 4, 64), f32), ((1, 4, 64), f8), ((1, 1, 1), f32))),
        (lambda t: moe.pack_rows(t), (x,)),
        (lambda q, s: moe.unpack_rows(moe.Rows8(q, s)), (r8, rs)),
        (lambda a, b: moe.swiglu(a, b), (x, x)),
        (lambda a, b, c: moe.swiglu_backward(a, b, c), (x, x, x)),
        (lambda h, a, b, c, e: moe.swiglu_backward(h, moe.Rows8(a, b), moe.Rows8(c, e)),
         (x, r8, rs, r8, rs)),
        (lambda *a: moe.moe_gate_forward(d, *a), (lg, ids, tw, ((5,), i32), ((4,), f32),
                                                  ((1,), f32), ws)),
        (lambda *a: moe.moe_gate_backward(d, *a), (lg, ids, ((5,), i32), tw, ((1,), f32), lg))]
    for call, shapes in calls:
        for i in range(len(shapes)):
            args = [_here(sh, t, _Elsewhere if j == i else _Here)
                    for j, (sh, t) in enumerate(shapes)]
            with pytest.raises(ValueError, match="current device is cuda:0"):
                call(*args)
