"""What the C entry points of the experts' products, the checkpoints and the
gate refuse, before any HIP call and so without a GPU.  Pointers used here are
never dereferenced: every call fails validation (or is a no-op) first.
"""

import pytest

import block_scaled_precision_gemm_amd as bsmm

OK, NULL, SHAPE, SCALE, LAYOUT, ALIGN, DTYPE, UNSUP, ARG = 0, 1, 2, 3, 4, 5, 6, 7, 9
F32, BF16, I32, E4M3 = bsmm.F32, bsmm.BF16, bsmm.I32, bsmm.E4M3
P = 0x10000          # a fake, 16-byte-aligned "device pointer" (never touched)


def said(status):
    if status != OK:
        assert bsmm.load().bsmm_last_error().decode()
    return status


def mm(*, x=P, ldx=64, w=P, w_se=2048, w_sn=64, w_sk=1, dt=BF16, order=P, offsets=P, per=2, rs=P,
       out=P, ldo=32, odt=BF16, E=4, R=8, S=16, N=32, K=64):
    return said(bsmm.load().bsmm_expert_mm(x, ldx, w, w_se, w_sn, w_sk, dt, order, offsets, per,
                                           rs, out, ldo, odt, E, R, S, N, K, None, 0, None))


@pytest.mark.parametrize("kw,status", [
    (dict(dt=I32), DTYPE), (dict(dt=E4M3), DTYPE), (dict(odt=I32), DTYPE),
    (dict(E=-1), SHAPE), (dict(R=-1), SHAPE), (dict(S=-1), SHAPE), (dict(N=-1), SHAPE),
    (dict(K=-1), SHAPE), (dict(R=2**31), UNSUP), (dict(N=2**31), UNSUP), (dict(K=2**31), UNSUP),
    (dict(E=1025), UNSUP), (dict(E=0), SHAPE), (dict(per=0), ARG), (dict(per=-2), ARG),
    (dict(S=17), SHAPE), (dict(offsets=None), NULL), (dict(out=None), NULL), (dict(x=None), NULL),
    (dict(w=None), NULL), (dict(order=P + 2), ALIGN), (dict(offsets=P + 1), ALIGN),
    (dict(rs=P + 2), ALIGN), (dict(ldo=31), SHAPE), (dict(out=P + 1), ALIGN),
    (dict(odt=F32, out=P + 2), ALIGN), (dict(ldx=63), SHAPE), (dict(w_se=-1), LAYOUT),
    (dict(w_sn=63), LAYOUT), (dict(w_sn=64, w_sk=2), LAYOUT), (dict(w_sn=1, w_sk=31), LAYOUT),
    (dict(w_sn=0), LAYOUT), (dict(w_sn=-64), LAYOUT), (dict(x=P + 1), ALIGN), (dict(w=P + 1), ALIGN),
    (dict(dt=F32, x=P + 2), ALIGN), (dict(dt=F32, w=P + 2), ALIGN),
    (dict(R=2**30, S=2**30, N=2**20, ldo=2**20), UNSUP), (dict(R=2**30, S=2**31 - 1024), UNSUP),
])
def test_mm_rejects(kw, status):
    assert mm(**kw) == status


def test_mm_noops():
    assert mm(S=0, offsets=None, out=None) == OK
    assert mm(N=0, w=None, out=None, ldo=0) == OK


def wgrad(*, dy=P, ldy=32, dt=BF16, yper=1, x=P, ldx=64, xper=2, sc=None, s_r=2, order=P, offsets=P,
          dw=P, w_se=2048, ldw=64, odt=F32, E=4, Ry=16, Rx=8, S=16, N=32, K=64):
    return said(bsmm.load().bsmm_expert_wgrad(dy, ldy, dt, yper, x, ldx, xper, sc, s_r, order,
                                              offsets, dw, w_se, ldw, odt, E, Ry, Rx, S, N, K,
                                              None, 0, None))


@pytest.mark.parametrize("kw,status", [
    (dict(dt=I32), DTYPE), (dict(odt=E4M3), DTYPE), (dict(E=-1), SHAPE), (dict(Ry=-1), SHAPE),
    (dict(Rx=-1), SHAPE), (dict(S=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=-1), SHAPE),
    (dict(Rx=2**31), UNSUP), (dict(K=2**31), UNSUP), (dict(E=1025), UNSUP), (dict(yper=0), ARG),
    (dict(S=2**31 - 1024, Rx=2**30, yper=2**30), UNSUP),
    (dict(xper=0), ARG), (dict(S=17, Rx=9), SHAPE), (dict(S=17, Ry=17), SHAPE),
    (dict(sc=P, K=48), UNSUP), (dict(offsets=None), NULL), (dict(dw=None), NULL),
    (dict(dy=None), NULL), (dict(x=None), NULL), (dict(order=P + 1), ALIGN),
    (dict(offsets=P + 2), ALIGN), (dict(ldw=63), SHAPE), (dict(w_se=2047), LAYOUT),
    (dict(dw=P + 2), ALIGN), (dict(odt=BF16, dw=P + 1), ALIGN), (dict(ldy=31), SHAPE),
    (dict(ldx=63), SHAPE), (dict(sc=P, s_r=1), SCALE), (dict(dy=P + 1), ALIGN),
    (dict(x=P + 1), ALIGN), (dict(dt=F32, x=P + 2), ALIGN),
    (dict(E=1024, N=2**18, K=2**18, ldy=2**18, ldx=2**18, ldw=2**18, w_se=2**36), UNSUP),
])
def test_wgrad_rejects(kw, status):
    assert wgrad(**kw) == status


def test_wgrad_noops():
    assert wgrad(E=0, dw=None, offsets=None) == OK
    assert wgrad(N=0, dw=None, offsets=None) == OK
    assert wgrad(K=0, dw=None, offsets=None) == OK


def quant(*, x=P, ldx=64, dt=BF16, q=P, ldq=64, s=P, s_r=2, v=P, ldv=64, R=8, K=64):
    return said(bsmm.load().bsmm_quant_int8_mx(x, ldx, dt, q, ldq, s, s_r, v, ldv, R, K, None))


@pytest.mark.parametrize("kw,status", [
    (dict(dt=I32), DTYPE), (dict(R=-1), SHAPE), (dict(K=-32), SHAPE), (dict(R=2**31), UNSUP),
    (dict(K=2**30), UNSUP), (dict(K=48), UNSUP), (dict(R=2**24, K=2**10), UNSUP),
    (dict(x=None), NULL), (dict(q=None), NULL), (dict(s=None), NULL), (dict(ldx=56), SHAPE),
    (dict(ldq=56), SHAPE), (dict(ldv=56), SHAPE), (dict(s_r=1), SCALE), (dict(x=P + 8), ALIGN),
    (dict(ldx=68), ALIGN), (dict(q=P + 4), ALIGN), (dict(ldq=68), ALIGN), (dict(v=P + 8), ALIGN),
    (dict(ldv=68), ALIGN),
])
def test_quantiser_rejects(kw, status):
    assert quant(**kw) == status


def gate(*, h=P, ldh=128, dt=BF16, a=P, lda=64, q=P, ldq=128, s=P, s_r=4, R=8, F=64):
    return said(bsmm.load().bsmm_swiglu(h, ldh, dt, a, lda, q, ldq, s, s_r, R, F, None))


@pytest.mark.parametrize("kw,status", [
    (dict(dt=E4M3), DTYPE), (dict(R=-1), SHAPE), (dict(F=-64), SHAPE), (dict(F=40), UNSUP),
    (dict(F=2**30), UNSUP), (dict(q=None), NULL), (dict(s=None), NULL), (dict(h=None), NULL),
    (dict(a=None), NULL), (dict(ldh=120), SHAPE), (dict(lda=56), SHAPE), (dict(ldq=120), SHAPE),
    (dict(s_r=3), SCALE), (dict(h=P + 4), ALIGN), (dict(ldh=132), ALIGN), (dict(a=P + 8), ALIGN),
    (dict(lda=68), ALIGN), (dict(q=P + 2), ALIGN), (dict(ldq=132), ALIGN),
])
def test_gate_rejects(kw, status):
    assert gate(**kw) == status


def back(*, da=P, ldda=64, dt=BF16, q=P, ldq=128, s=P, s_r=4, rs=P, dh=P, lddh=128, act=P, ldact=64,
         drow=P, R=8, F=64):
    return said(bsmm.load().bsmm_swiglu_backward(da, ldda, dt, q, ldq, s, s_r, rs, dh, lddh, act,
                                                 ldact, drow, R, F, None))


@pytest.mark.parametrize("kw,status", [
    (dict(dt=I32), DTYPE), (dict(R=-1), SHAPE), (dict(F=33), UNSUP), (dict(rs=None), ARG),
    (dict(rs=P + 2), ALIGN), (dict(drow=P + 1), ALIGN), (dict(da=None), NULL), (dict(q=None), NULL),
    (dict(s=None), NULL), (dict(dh=None), NULL), (dict(ldda=56), SHAPE), (dict(ldq=120), SHAPE),
    (dict(s_r=3), SCALE), (dict(lddh=120), SHAPE), (dict(ldact=56), SHAPE), (dict(da=P + 4), ALIGN),
    (dict(dh=P + 4), ALIGN), (dict(act=P + 4), ALIGN), (dict(ldact=68), ALIGN), (dict(q=P + 1), ALIGN),
])
def test_gate_gradient_rejects(kw, status):
    assert back(**kw) == status


def test_noops():
    assert quant(R=0, x=None, q=None, s=None, v=None) == OK
    assert quant(K=0, x=None, q=None, s=None, v=None) == OK
    assert gate(R=0, h=None, a=None) == OK
    assert gate(F=0, h=None, a=None) == OK
    assert back(R=0, da=None, q=None, s=None, dh=None) == OK


def test_workspaces():
    """Where tiles are few, for a bf16 checkpoint, and nothing else."""
    mm_need = bsmm.load().bsmm_expert_mm_workspace_bytes
    assert mm_need(BF16, 0, 8, 4096, 4096, 4096) == 0
    need = mm_need(BF16, 0, 1, 300, 130, 4096)
    assert need > 0 and need % (300 * 130 * 4) == 0
    assert mm_need(F32, 1, 1, 300, 130, 4096) > 0
    for bad in ((I32, 0, 1, 300, 130, 4096), (BF16, 0, 0, 300, 130, 4096), (BF16, 0, 1, 0, 9, 9),
                (BF16, 0, 1, 9, -1, 9), (BF16, 0, 1, 2**31, 9, 9), (BF16, 0, 1025, 9, 9, 9)):
        assert mm_need(*bad) == 0
    w_need = bsmm.load().bsmm_expert_wgrad_workspace_bytes
    assert w_need(BF16, 0, 8, 4096, 4096, 4096, 4096) == 0
    assert w_need(BF16, 1, 8, 4096, 4096, 4096, 4096) == 4096 * 4096 * 2
    assert w_need(F32, 1, 8, 4096, 4096, 4096, 4096) == 0
    need = w_need(F32, 0, 1, 9000, 9000, 64, 72)
    assert need > 0 and need % (64 * 72 * 4) == 0
    assert w_need(BF16, 1, 1, 9000, 9000, 64, 96) > 9000 * 96 * 2
    for bad in ((I32, 1, 1, 9, 9, 9, 32), (BF16, 1, 0, 9, 9, 9, 32), (BF16, 1, 1, 2**31, 9, 9, 32),
                (BF16, 1, 1, 9, -1, 9, 32)):
        assert w_need(*bad) == 0
    # the largest sizes: no overflow on the way (see the sanitized run of these tests)
    mm_need(BF16, 1, 1024, 2**31 - 1, 2**31 - 1, 2**31 - 1)
    w_need(BF16, 1, 1024, 2**31 - 1, 2**31 - 1, 2**31 - 1, 2**31 - 1)
