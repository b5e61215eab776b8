"""What the C entry points of the 4-bit weight operations and the router
refuse, before any HIP call and so without a GPU.  Pointers used here are
never dereferenced: every call fails validation (or is a no-op) first.
"""

import pytest

import block_scaled_precision_gemm_amd as bsmm

OK, NULL, SHAPE, SCALE, LAYOUT, ALIGN, DTYPE, UNSUP, ARG = 0, 1, 2, 3, 4, 5, 6, 7, 9
F32, BF16, I32 = bsmm.F32, bsmm.BF16, bsmm.I32
P = 0x10000          # a fake, 16-byte-aligned "device pointer" (never touched)


def test_status_names():
    assert {n: bsmm.STATUS[n] for n in (NULL, SHAPE, SCALE, LAYOUT, ALIGN, DTYPE, UNSUP, ARG)} == \
        {NULL: "BSMM_ERR_NULL", SHAPE: "BSMM_ERR_SHAPE", SCALE: "BSMM_ERR_SCALE_SHAPE",
         LAYOUT: "BSMM_ERR_LAYOUT", ALIGN: "BSMM_ERR_ALIGN", DTYPE: "BSMM_ERR_DTYPE",
         UNSUP: "BSMM_ERR_UNSUPPORTED", ARG: "BSMM_ERR_ARG"}


def said(status):
    if status != OK:
        assert bsmm.load().bsmm_last_error().decode()
    return status


def quant(*, w=P, ldw=256, wdt=BF16, q=P, ldq=128, s=P, s_r=4, sdt=F32, z=P, z_r=4, v=P, ldv=256,
          group=64, R=8, K=256):
    return said(bsmm.load().bsmm_quant_w4(w, ldw, wdt, q, ldq, s, s_r, sdt, z, z_r, v, ldv, group,
                                          R, K, None))


@pytest.mark.parametrize("kw,status", [
    (dict(wdt=I32), DTYPE), (dict(sdt=I32), DTYPE), (dict(R=-1), SHAPE), (dict(K=-64), SHAPE),
    (dict(R=2**31), UNSUP), (dict(group=16), ARG), (dict(group=256), ARG), (dict(group=0), ARG),
    (dict(K=96), UNSUP), (dict(K=32, group=64), UNSUP),
    (dict(R=2**24, K=4096), UNSUP),
    (dict(w=None), NULL), (dict(q=None), NULL), (dict(s=None), NULL),
    (dict(ldw=248), SHAPE), (dict(ldq=112), SHAPE), (dict(ldv=248), SHAPE),
    (dict(s_r=3), SCALE), (dict(z_r=3), SCALE),
    (dict(w=P + 8), ALIGN), (dict(ldw=260), ALIGN), (dict(q=P + 4), ALIGN), (dict(ldq=136), ALIGN),
    (dict(v=P + 2), ALIGN), (dict(ldv=260), ALIGN), (dict(s=P + 2), ALIGN),
    (dict(s=P + 1, sdt=BF16), ALIGN),
])
def test_quantiser_rejects(kw, status):
    assert quant(**kw) == status


def test_quantiser_noops():
    assert quant(R=0, w=None, q=None, s=None) == OK
    assert quant(K=0, w=None) == OK


def mm(*, x=P, ldx=256, xdt=BF16, w=P, ldw=128, s=P, s_n=4, sdt=F32, z=P, z_n=4, group=64, out=P,
       ldo=64, odt=BF16, M=8, N=64, K=256, ws=None, wsb=0):
    return said(bsmm.load().bsmm_w4_mm(x, ldx, xdt, w, ldw, s, s_n, sdt, z, z_n, group, out, ldo,
                                       odt, M, N, K, ws, wsb, None))


def experts(*, x=P, ldx=256, xdt=BF16, w=P, w_se=8192, ldw=128, s=P, s_se=256, s_n=4, sdt=F32,
            z=P, z_se=256, z_n=4, group=64, order=P, offsets=P, per=2, rs=P, out=P, ldo=64,
            odt=BF16, E=4, R=8, S=16, N=64, K=256):
    return said(bsmm.load().bsmm_w4_expert_mm(
        x, ldx, xdt, w, w_se, ldw, s, s_se, s_n, sdt, z, z_se, z_n, group, order, offsets, per, rs,
        out, ldo, odt, E, R, S, N, K, None, 0, None))


BOTH = [
    (dict(xdt=I32), DTYPE), (dict(sdt=I32), DTYPE), (dict(odt=I32), DTYPE),
    (dict(N=-1), SHAPE), (dict(K=-64), SHAPE), (dict(N=2**31), UNSUP), (dict(K=2**31), UNSUP),
    (dict(group=48), ARG), (dict(K=224), UNSUP), (dict(x=None), NULL), (dict(w=None), NULL),
    (dict(s=None), NULL), (dict(out=None), NULL), (dict(ldx=248), SHAPE), (dict(ldw=112), SHAPE),
    (dict(ldo=63), SHAPE), (dict(s_n=3), SCALE), (dict(s_n=-4), SCALE), (dict(z_n=3), SCALE),
    (dict(x=P + 8), ALIGN), (dict(ldx=260), ALIGN), (dict(w=P + 8), ALIGN), (dict(ldw=136), ALIGN),
    (dict(out=P + 2), ALIGN), (dict(s=P + 2), ALIGN), (dict(s=P + 1, sdt=BF16), ALIGN),
]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(M=-1), SHAPE), (dict(M=2**31), UNSUP), (dict(M=2**30, N=2**20, ldo=2**20), UNSUP)])
def test_mm_rejects(kw, status):
    assert mm(**kw) == status


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(E=-1), SHAPE), (dict(R=-1), SHAPE), (dict(S=-1), SHAPE), (dict(E=1025), UNSUP),
    (dict(E=0), SHAPE), (dict(R=2**31, S=1), UNSUP), (dict(S=17), SHAPE), (dict(per=0), ARG),
    (dict(order=None), NULL), (dict(offsets=None), NULL), (dict(order=P + 2), ALIGN),
    (dict(offsets=P + 1), ALIGN), (dict(rs=P + 2), ALIGN), (dict(w_se=-16), LAYOUT),
    (dict(w_se=8200), ALIGN), (dict(s_se=-1), SCALE), (dict(z_se=-1), SCALE)])
def test_experts_reject(kw, status):
    assert experts(**kw) == status


def test_product_noops():
    assert mm(M=0, x=None, out=None) == OK
    assert mm(N=0, w=None, out=None) == OK
    assert experts(S=0, order=None, offsets=None) == OK
    assert experts(N=0, out=None, ldo=0) == OK


def test_product_workspace():
    """Planes for an fp32 x where tiles are worth it, and only there."""
    need = bsmm.load().bsmm_w4_workspace_bytes
    assert need(F32, 1, 2048, 2048, 4096, 4096, 128) == 3 * 2048 * 4096 * 2
    assert need(F32, 8, 4096, 4096, 4096, 4096, 128) == 3 * 4096 * 4096 * 2
    assert need(F32, 1, 13, 13, 4099, 7168, 32) == 0
    assert need(BF16, 1, 2048, 2048, 4096, 4096, 128) == 0
    # planes beyond 32-bit offsets: run without
    assert need(F32, 1, 2**20, 2**20, 4096, 4096, 128) == 0
    for bad in ((F32, 0, 9, 9, 9, 64, 32), (F32, 1, -1, 9, 9, 64, 32),
                (F32, 1, 2**31, 2**31, 4096, 4096, 32), (F32, 1025, 9, 9, 9, 64, 32)):
        assert need(*bad) == 0


def route(*, x=P, ldl=64, dt=F32, mask=None, k=4, index=P, weight=P, counts=P, offsets=P, order=P,
          live=P, prob=P, loss=P, T=100, E=64, ws=P, wsb=1 << 30):
    return said(bsmm.load().bsmm_route_topk(x, ldl, dt, mask, k, 1, 0.01, index, weight, counts,
                                            offsets, order, live, prob, loss, T, E, ws, wsb, None))


@pytest.mark.parametrize("kw,status", [
    (dict(dt=I32), DTYPE), (dict(T=-1), SHAPE), (dict(E=-1), SHAPE), (dict(E=0), UNSUP),
    (dict(E=1025, ldl=1025), UNSUP), (dict(k=0), ARG), (dict(k=33), ARG), (dict(E=3, k=4), ARG),
    (dict(T=2**23 + 1), UNSUP), (dict(x=None), NULL), (dict(ldl=63), SHAPE), (dict(x=P + 2), ALIGN),
    (dict(x=P + 1, dt=BF16), ALIGN), (dict(counts=None), NULL), (dict(offsets=None), NULL),
    (dict(index=None), NULL), (dict(weight=None), NULL), (dict(order=None), NULL),
    (dict(live=None), NULL), (dict(prob=None), NULL), (dict(loss=None), NULL),
    (dict(index=P + 2), ALIGN), (dict(prob=P + 2), ALIGN), (dict(order=P + 1), ALIGN),
    (dict(ws=None), ARG), (dict(wsb=16), ARG), (dict(ws=P + 8), ALIGN),
])
def test_router_rejects(kw, status):
    assert route(**kw) == status


def back(*, x=P, ldl=64, dt=F32, index=P, weight=P, counts=P, live=P, k=4, dw=P, dl=P, dx=P,
         ldd=64, T=100, E=64):
    return said(bsmm.load().bsmm_route_topk_backward(x, ldl, dt, None, index, weight, counts, live,
                                                     k, 1, 0.01, dw, dl, dx, ldd, T, E, None))


@pytest.mark.parametrize("kw,status", [
    (dict(dt=I32), DTYPE), (dict(T=-1), SHAPE), (dict(E=1025, ldl=1025, ldd=1025), UNSUP),
    (dict(k=0), ARG), (dict(k=65), ARG), (dict(x=None), NULL), (dict(dx=None), NULL),
    (dict(ldl=63), SHAPE), (dict(ldd=63), SHAPE), (dict(x=P + 2), ALIGN), (dict(dx=P + 2), ALIGN),
    (dict(index=None), NULL), (dict(weight=None), NULL), (dict(counts=None), NULL),
    (dict(live=None), NULL), (dict(index=P + 2), ALIGN), (dict(dw=P + 2), ALIGN),
    (dict(dl=P + 2), ALIGN),
])
def test_router_backward_rejects(kw, status):
    assert back(**kw) == status


def test_router_backward_noop():
    assert back(T=0, x=None, dx=None, index=None) == OK


def test_router_workspace():
    need = bsmm.load().bsmm_route_workspace_bytes
    assert need(64, 64) == 0 and need(65, 64) > 0 and need(2**23, 1024) > 0
    assert need(0, 64) == need(-1, 64) == need(100, 0) == need(100, 1025) == 0
    assert need(2**23 + 1, 64) == 0
