"""Host-only checks of the nvfp4_fp8_* and nvfp4_moe_* entry points: sizes, and bad arguments refused before any launch."""
import pytest
import torch

import nvfp4_block_scaled_amd as nv

FAKE, ODD, HALF = 0x10000, 0x10001, 0x10008            # never dereferenced; HALF: 8-byte aligned only


def checked(name, **good):
    """A call of a C entry point with some arguments changed."""
    def call(**kw):
        assert set(kw) <= set(good)
        return getattr(nv.lib(), name)(*{**good, **kw}.values())
    return call


def test_quantize():
    f = checked("nvfp4_fp8_quantize", x=FAKE, dtype=1, rows=3, K=256, ldx=512, gated=0, codes=FAKE, scales=FAKE, stream=None)
    assert f(rows=0) == nv.OK and f(rows=0, x=None) == nv.OK
    assert f(dtype=3) == nv.ERR_DTYPE and f(dtype=-1) == nv.ERR_DTYPE and f(gated=2) == nv.ERR_VALUE
    assert f(rows=-1) == nv.ERR_SHAPE and f(K=0) == nv.ERR_SHAPE and f(K=250) == nv.ERR_SHAPE and f(ldx=255) == nv.ERR_SHAPE
    assert f(gated=1, ldx=511) == nv.ERR_SHAPE and f(rows=1 << 40) == nv.ERR_SHAPE and f(K=1 << 40, ldx=1 << 40) == nv.ERR_SHAPE
    for name in ("x", "codes", "scales"):
        assert f(**{name: None}) == nv.ERR_NULL and f(**{name: ODD}) == nv.ERR_ALIGN
    assert f(codes=HALF) == nv.ERR_ALIGN and f(dtype=0, x=0x10002) == nv.ERR_ALIGN


def test_quantize_weight():
    f = checked("nvfp4_fp8_quantize_weight", w=FAKE, dtype=1, experts=2, N=5, K=256, ldw=256, stride=1280, codes=FAKE, scales=FAKE,
                stream=None)
    assert f(experts=0) == nv.OK and f(dtype=3) == nv.ERR_DTYPE
    for bad in (dict(experts=-1), dict(N=0), dict(K=0), dict(K=24), dict(ldw=255), dict(stride=-1), dict(N=1 << 28, K=1 << 28, ldw=1 << 28)):
        assert f(**bad) == nv.ERR_SHAPE, bad
    for name in ("w", "codes", "scales"):
        assert f(**{name: None}) == nv.ERR_NULL and f(**{name: ODD}) == nv.ERR_ALIGN


def test_product():
    f = checked("nvfp4_fp8_gemm", a=FAKE, sa=FAKE, w=FAKE, sw=FAKE, M=3, N=5, K=256, out=FAKE, dtype=1, ldo=5, ws=None, n=0, stream=None)
    assert f(M=0) == nv.OK and f(M=0, a=None, out=None) == nv.OK
    for bad in (0, 3, -1):
        assert f(dtype=bad) == nv.ERR_DTYPE
    for bad in (dict(M=-1), dict(M=1 << 31), dict(N=0), dict(K=0), dict(K=100), dict(ldo=4), dict(N=1 << 40, ldo=1 << 40), dict(K=1 << 40)):
        assert f(**bad) == nv.ERR_SHAPE, bad
    for name in ("a", "sa", "w", "sw", "out"):
        assert f(**{name: None}) == nv.ERR_NULL and f(**{name: ODD}) == nv.ERR_ALIGN
    assert f(a=HALF) == nv.ERR_ALIGN and f(w=HALF) == nv.ERR_ALIGN and f(sa=0x10002) == nv.ERR_ALIGN


def test_product_workspace():
    need = nv.lib().nvfp4_fp8_gemm_workspace_bytes
    for M, N, K in ((-1, 5, 256), (0, 5, 256), (3, 0, 256), (3, 5, 100), (1 << 40, 5, 256)):
        assert need(M, N, K) == 0
    f = checked("nvfp4_fp8_gemm", a=FAKE, sa=FAKE, w=FAKE, sw=FAKE, M=200, N=5120, K=17408, out=FAKE, dtype=1, ldo=5120, ws=None, n=0,
                stream=None)
    n = need(200, 5120, 17408)
    if n:
        assert f() == nv.ERR_WORKSPACE and f(ws=FAKE, n=n - 1) == nv.ERR_WORKSPACE and f(ws=HALF, n=n) == nv.ERR_ALIGN


def test_product_by_expert():
    f = checked("nvfp4_fp8_gemm_grouped", a=FAKE, sa=FAKE, a_rows=9, rows=FAKE, w=FAKE, sw=FAKE, experts=4, offsets=FAKE, M=12, N=5, K=256,
                out=FAKE, dtype=2, ldo=5, stream=None)
    assert f(M=0) == nv.OK and f(a_rows=0) == nv.OK and f(dtype=0) == nv.ERR_DTYPE
    for bad in (dict(M=-1), dict(N=0), dict(K=8), dict(ldo=4), dict(experts=0), dict(experts=1025), dict(a_rows=-1), dict(rows=None)):
        assert f(**bad) == nv.ERR_SHAPE, bad                    # without rows, a needs as many as out
    for name in ("a", "sa", "w", "sw", "out", "offsets"):
        assert f(**{name: None}) == nv.ERR_NULL and f(**{name: ODD}) == nv.ERR_ALIGN
    assert f(rows=ODD) == nv.ERR_ALIGN


def test_sort():
    f = checked("nvfp4_moe_sort", ids=FAKE, id_bytes=4, tokens=3000, top=4, experts=64, offsets=FAKE, tokens_out=FAKE, places=FAKE, ws=FAKE,
                n=1 << 20, stream=None)
    need = nv.lib().nvfp4_moe_sort_workspace_bytes
    n = need(3000, 4, 64)
    assert n > 0 and need(3, 4, 64) == 0 and need(3, 4, 0) == 0 and need(-1, 4, 64) == 0
    assert f(id_bytes=2) == nv.ERR_DTYPE
    for bad in (dict(tokens=-1), dict(top=0), dict(experts=0), dict(experts=1025), dict(tokens=1 << 30), dict(tokens=1 << 62, top=1 << 62)):
        assert f(**bad) == nv.ERR_SHAPE, bad
    for name in ("ids", "offsets", "tokens_out", "places"):
        assert f(**{name: None}) == nv.ERR_NULL and f(**{name: ODD}) == nv.ERR_ALIGN
    assert f(id_bytes=8, ids=0x10004) == nv.ERR_ALIGN
    assert f(ws=None) == nv.ERR_WORKSPACE and f(n=n - 1) == nv.ERR_WORKSPACE and f(ws=HALF) == nv.ERR_ALIGN


def test_rows_to_places_and_back():
    gather = checked("nvfp4_moe_gather", x=FAKE, dtype=0, ldx=40, places=FAKE, tokens=3, top=2, width=40, out=FAKE, ldo=40, stream=None)
    combine = checked("nvfp4_moe_combine", y=FAKE, dtype=0, ldy=40, places=FAKE, weights=FAKE, tokens=3, top=2, width=40, out=FAKE, ldo=40,
                      stream=None)
    back = checked("nvfp4_moe_combine_backward", grad=FAKE, ldg=40, y=FAKE, ldy=40, dtype=0, places=FAKE, weights=FAKE, tokens=3, top=2,
                   width=40, grad_y=FAKE, ldo=40, grad_weights=FAKE, stream=None)
    for f, tensors, strides in ((gather, ("x", "places", "out"), ("ldx", "ldo")), (combine, ("y", "places", "out"), ("ldy", "ldo")),
                                (back, ("grad", "y", "places", "weights", "grad_y", "grad_weights"), ("ldg", "ldy", "ldo"))):
        assert f(tokens=0) == nv.OK and f(dtype=3) == nv.ERR_DTYPE
        for bad in (dict(tokens=-1), dict(top=0), dict(width=0), dict(width=1 << 40), dict(tokens=1 << 30, top=2), *({s: 39} for s in strides)):
            assert f(**bad) == nv.ERR_SHAPE, bad
        for name in tensors:
            assert f(**{name: None}) == nv.ERR_NULL and f(**{name: ODD}) == nv.ERR_ALIGN
    assert combine(weights=ODD) == nv.ERR_ALIGN


def test_binding_refuses_host_tensors():
    x, i = torch.zeros((4, 128)), torch.zeros((4, 2), dtype=torch.int32)
    c = torch.zeros((4, 128), dtype=torch.uint8)
    s = torch.zeros((4, 1))
    for call in (lambda: nv.nvfp4_fp8_quantize(x), lambda: nv.nvfp4_fp8_quantize_weight(x), lambda: nv.nvfp4_fp8_gemm(c, s, c, s),
                 lambda: nv.nvfp4_fp8_gemm_grouped(c, s, c[None], s[None], i), lambda: nv.nvfp4_moe_sort(i, 4),
                 lambda: nv.nvfp4_moe_gather(x, i), lambda: nv.nvfp4_moe_combine(x, i), lambda: nv.nvfp4_moe_gather_backward(x, i),
                 lambda: nv.nvfp4_moe_combine_backward(x, x, i, x), lambda: nv.nvfp4_fp8_quantize(None)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.gpu
def test_binding_refusals():
    z = lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype, device="cuda")      # noqa: E731
    x, c, s = z(4, 128), z(4, 128, dtype=torch.float8_e4m3fn), z(4, 1)
    w, sw = z(200, 128, dtype=torch.uint8), z(2, 1)
    i = z(4, 2, dtype=torch.int32)
    nv.nvfp4_fp8_gemm(c, s, w, sw)
    out = z(4, 200, dtype=torch.bfloat16)
    value = [lambda: nv.nvfp4_fp8_quantize(z(4, 120)), lambda: nv.nvfp4_fp8_quantize(z(4, 33), gated=True), lambda: nv.nvfp4_fp8_quantize(z(128)),
             lambda: nv.nvfp4_fp8_quantize(z(4, 0)), lambda: nv.nvfp4_fp8_quantize(x, codes=z(4, 256, dtype=torch.uint8)[:, :128]),
             lambda: nv.nvfp4_fp8_quantize(x, scales=z(4, 2)), lambda: nv.nvfp4_fp8_quantize_weight(z(0, 128)),
             lambda: nv.nvfp4_fp8_gemm(c, z(4, 2), w, sw), lambda: nv.nvfp4_fp8_gemm(c, s, w, z(3, 1)), lambda: nv.nvfp4_fp8_gemm(c, s, w[:, :112], sw),
             lambda: nv.nvfp4_fp8_gemm(c[:, ::2], s, w, sw), lambda: nv.nvfp4_fp8_gemm(c, s, w, sw, out=out[:, ::2]),
             lambda: nv.nvfp4_fp8_gemm(c, s, w, sw, out=out[:1].expand(4, 200)), lambda: nv.nvfp4_fp8_gemm(c, s, w, sw, out=out[:3]),
             lambda: nv.nvfp4_fp8_gemm_grouped(c, s, w[None], sw[None], z(3, dtype=torch.int32)),
             lambda: nv.nvfp4_fp8_gemm_grouped(c, s, w, sw, z(2, dtype=torch.int32)),
             lambda: nv.nvfp4_moe_sort(i, 0), lambda: nv.nvfp4_moe_sort(i, 1025), lambda: nv.nvfp4_moe_sort(i[0], 4),
             lambda: nv.nvfp4_moe_gather(z(3, 8), i), lambda: nv.nvfp4_moe_gather(z(4, 8), i, out=z(7, 8)),
             lambda: nv.nvfp4_moe_gather(z(8, 8)[:4], i, out=z(8, 9)), lambda: nv.nvfp4_moe_combine(z(8, 8), i, z(4, 3)),
             lambda: nv.nvfp4_moe_combine_backward(z(4, 9), z(8, 8), i, z(4, 2))]
    shared = z(12, 8)
    value += [lambda: nv.nvfp4_moe_gather(shared[:4], i, out=shared[3:11]), lambda: nv.nvfp4_moe_combine(shared[:8], i, out=shared[:4])]
    kind = [lambda: nv.nvfp4_fp8_quantize(x.double()), lambda: nv.nvfp4_fp8_gemm(x, s, w, sw), lambda: nv.nvfp4_fp8_gemm(c, s.double(), w, sw),
            lambda: nv.nvfp4_fp8_gemm(c, s, w, sw, out_dtype="f32"), lambda: nv.nvfp4_fp8_gemm(c, s, w, sw, out=z(4, 200)),
            lambda: nv.nvfp4_fp8_gemm_grouped(c, s, w[None], sw[None], z(2, dtype=torch.int64)), lambda: nv.nvfp4_moe_sort(i.short(), 4),
            lambda: nv.nvfp4_moe_gather(z(4, 8), i.long()), lambda: nv.nvfp4_moe_combine(z(8, 8), i, z(4, 2).half()),
            lambda: nv.nvfp4_moe_combine_backward(z(4, 8).half(), z(8, 8), i, z(4, 2))]
    for error, calls in ((ValueError, value), (TypeError, kind)):
        for n, call in enumerate(calls):
            with pytest.raises(error):
                call()
                print(error, n)
    torch.cuda.synchronize()
