"""What the experts' calls refuse, without a GPU: the C entry points' checks
with fake pointers (every call carries an argument they reject, or no rows), and
the binding's with host tensors."""
import pytest
import torch

import combine_topk_route_amd as m
from combine_topk_route_amd import _lib

OK, INVALID, ALIGN, CAP = (_lib.MOE_OK, _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_ALIGNMENT,
                           _lib.MOE_ERR_CAPACITY)
P = 0x10000   # a fake, 16-byte aligned address; never dereferenced
P8 = 0x10008  # not 16-byte aligned

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host-only checks with fake pointers; run without a GPU")

GATED = dict(x=P, off=P, w=P, rows=4, E=2, H=16, I=8, act=1, h=P, gu=None, stream=None)
GATED_B = dict(dh=P, gu=P, x=P, off=P, w=P, rows=4, E=2, H=16, I=8, act=1, dgu=P, dx=P, dw=P, f32=0,
               stream=None)
MATMUL = dict(x=P, off=P, w=P, bias=None, res=None, rows=4, E=2, K=16, N=8, act=0, y=P, pre=None,
              stream=None)
MATMUL_B = dict(dy=P, pre=None, x=P, off=P, w=P, rows=4, E=2, K=16, N=8, act=0, dpre=None, dx=P,
                dw=P, f32=0, dbias=None, stream=None)
COMBINE_B = dict(dout=P, y=P, row=P, w=P, T=4, H=16, k=2, cap=8, dy=P, dw=P, stream=None)

SIZES = [(dict(rows=-1), INVALID), (dict(rows=2**31), INVALID), (dict(E=0), INVALID),
         (dict(E=1025), INVALID), (dict(act=4), INVALID), (dict(act=-1), INVALID),
         (dict(x=P8), ALIGN), (dict(w=P8), ALIGN), (dict(off=0x10002), ALIGN),
         (dict(off=None), INVALID)]
BAD = [("moe_expert_gated", GATED, c, st) for c, st in SIZES + [
    (dict(H=0), INVALID), (dict(H=12), ALIGN), (dict(I=4), INVALID), (dict(I=20), ALIGN),
    (dict(H=2**20 + 8), INVALID), (dict(act=0), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(h=None), INVALID), (dict(h=P8), ALIGN), (dict(gu=P8), ALIGN)]]
BAD += [("moe_expert_gated_backward", GATED_B, c, st) for c, st in SIZES + [
    (dict(H=12), ALIGN), (dict(I=4), INVALID), (dict(act=0), INVALID), (dict(dh=None), INVALID),
    (dict(gu=None), INVALID), (dict(dgu=None), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(f32=2), INVALID), (dict(dx=P8), ALIGN), (dict(dw=P8), ALIGN),
    (dict(dh=P8), ALIGN), (dict(gu=P8), ALIGN), (dict(dgu=P8), ALIGN)]]
BAD += [("moe_expert_matmul", MATMUL, c, st) for c, st in SIZES + [
    (dict(K=12), ALIGN), (dict(K=0), INVALID), (dict(N=2**20 + 8), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(y=P8), ALIGN), (dict(pre=P8), ALIGN),
    (dict(bias=P8), ALIGN), (dict(res=P8), ALIGN)]]
BAD += [("moe_expert_matmul_backward", MATMUL_B, c, st) for c, st in SIZES + [
    (dict(K=12), ALIGN), (dict(N=4), INVALID), (dict(dy=None), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(act=1), INVALID), (dict(act=1, pre=P), INVALID),
    (dict(act=1, dpre=P), INVALID), (dict(f32=-1), INVALID), (dict(dbias=0x10002), ALIGN),
    (dict(dy=P8), ALIGN), (dict(dx=P8), ALIGN), (dict(dw=P8), ALIGN),
    (dict(act=1, pre=P8, dpre=P), ALIGN), (dict(act=1, pre=P, dpre=P8), ALIGN)]]
BAD += [("moe_combine_backward", COMBINE_B, c, st) for c, st in [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(k=33), INVALID), (dict(T=2**30, k=2), INVALID),
    (dict(H=0), INVALID), (dict(H=12), ALIGN), (dict(H=2**20 + 8), INVALID), (dict(cap=7), CAP),
    (dict(dout=None), INVALID), (dict(y=None), INVALID), (dict(row=None), INVALID),
    (dict(w=None), INVALID), (dict(dy=None), INVALID), (dict(dw=None), INVALID),
    (dict(dout=P8), ALIGN), (dict(y=P8), ALIGN), (dict(dy=P8), ALIGN), (dict(row=0x10002), ALIGN),
    (dict(w=0x10002), ALIGN), (dict(dw=0x10002), ALIGN)]]


@pytest.mark.parametrize("name,good,change,status", BAD,
                         ids=[f"{n[4:]}-{'-'.join(f'{k}={v}' for k, v in c.items())}" for n, _, c, _ in BAD])
def test_c_entry_points_refuse(name, good, change, status):
    assert getattr(_lib.load(), name)(*{**good, **change}.values()) == status


def test_no_rows_enqueue_nothing():
    lib = _lib.load()
    for name, good, none in [
            ("moe_expert_gated", GATED, dict(rows=0, x=None, h=None)),
            ("moe_expert_matmul", MATMUL, dict(rows=0, x=None, y=None)),
            ("moe_expert_gated_backward", GATED_B, dict(rows=0, dh=None, gu=None, x=None, dgu=None,
                                                        dx=None, dw=None)),
            ("moe_expert_matmul_backward", MATMUL_B, dict(rows=0, dy=None, x=None, dx=None, dw=None)),
            ("moe_combine_backward", COMBINE_B, dict(T=0, dout=None, y=None, dy=None, dw=None))]:
        assert getattr(lib, name)(*{**good, **none}.values()) == OK, name


def test_binding_refuses_host_tensors():
    bf = torch.bfloat16
    x, off, w = torch.zeros((4, 16), dtype=bf), torch.zeros(3, dtype=torch.int32), \
        torch.zeros((2, 16, 16), dtype=bf)
    for call in (lambda: m.moe_expert_gated(x, off, w), lambda: m.moe_expert_matmul(x, off, w),
                 lambda: m.moe_expert_gated_backward(x, x, x, off, w),
                 lambda: m.moe_expert_matmul_backward(x, x, off, w),
                 lambda: m.moe_combine_backward(x, x, torch.zeros((2, 2), dtype=torch.int32),
                                                torch.zeros((2, 2)))):
        with pytest.raises(ValueError, match="device"):
            call()
    with pytest.raises(TypeError, match="torch.Tensor"):
        m.moe_expert_gated([[0.0] * 16], off, w)


def test_activation_names():
    from combine_topk_route_amd import experts
    assert {a: experts._act(a) for a in _lib.ACTS} == _lib.ACTS
    for bad in ("swish", None, ["silu"]):
        with pytest.raises(ValueError, match="act must be one of"):
            experts._act(bad)
    import os
    import re
    header = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                               "moe_route.h")).read()
    declared = {n.lower(): int(v) for n, v in re.findall(r"MOE_ACT_(\w+) = (\d)", header)}
    assert declared == _lib.ACTS


def test_gradient_dtype_is_checked():
    from combine_topk_route_amd import experts
    assert experts._dw_dtype(None, torch.float32) is torch.float32
    assert experts._dw_dtype(torch.zeros(1, dtype=torch.bfloat16), torch.float32) is torch.bfloat16
    with pytest.raises(TypeError, match="dw must be"):
        experts._dw_dtype(None, torch.float16)
