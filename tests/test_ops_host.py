"""Host-side checks of the mixture-of-experts operators: the library exports
what det_ops.h declares, the C entry points refuse bad arguments before they
touch a GPU, and the binding refuses bad tensors. No GPU needed."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "det_ops.h")
P = 0x100000      # a fake, aligned device address; never dereferenced here
Q = 0x40000000
R = 0x80000000
S = 0xC0000000
W = 0x100000000
OK, INVALID, ALIGN, NO_DEVICE = 0, 1, 3, 4


@pytest.fixture(scope="module")
def dg():
    from invariant_deterministic_gemm_gb300 import _build
    _build.build()
    import invariant_deterministic_gemm_gb300 as m
    m.lib()
    return m


_CTYPES = {"int64_t": ctypes.c_int64, "int": ctypes.c_int, "float": ctypes.c_float, "det_gemm_stream": ctypes.c_void_p}


def declared():
    """Each function of the header: its result's and its arguments' ctypes."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    out = {}
    for m in re.finditer(r"\b(det_gemm_status|int64_t)\s+(det_[a-z0-9_]+)\s*\(([^;]*)\);", text):
        args = [a.strip() for a in m.group(3).split(",")]
        out[m.group(2)] = (ctypes.c_int64 if m.group(1) == "int64_t" else ctypes.c_int,
                           [ctypes.c_void_p if "*" in a else _CTYPES[a.rsplit(" ", 1)[0]] for a in args])
    return out


@pytest.fixture(scope="module")
def fn(dg):
    """The library's C functions, by name."""
    def get(name):
        f = getattr(ctypes.CDLL(dg.LIB_PATH), name)
        f.restype, f.argtypes = declared()[name]
        return f
    return get


def test_every_declared_function_is_exported(dg):
    names = declared()
    assert len(names) == 17
    for n in names:
        assert hasattr(dg.lib(), n), n


def test_public_names_are_exported(dg):
    for n in declared():
        if n != "det_embedding_grad_workspace":
            assert callable(getattr(dg, n)), n
            assert n in dg.__all__, n


def route(fn, logits=P, fp32=1, bias=None, w=Q, ids=R, T=4, E=8, ldl=8, k=2, score=0, G=1, tg=1, gb=2, rn=1):
    return fn("det_moe_route")(logits, fp32, bias, w, ids, T, E, ldl, k, score, G, tg, gb, rn, 1.0, None)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(E=0), dict(E=513, ldl=513), dict(k=0), dict(k=9), dict(score=2), dict(G=0),
                                 dict(G=3), dict(G=4, tg=5), dict(G=8, tg=1, k=2), dict(gb=3), dict(ldl=7),
                                 dict(logits=None), dict(w=None), dict(ids=None), dict(ids=Q), dict(w=P), dict(k=33, E=64, ldl=64)])
def test_route_refuses(fn, bad):
    assert route(fn, **bad) == INVALID


def test_route_misaligned(fn):
    assert route(fn, logits=P + 2) == ALIGN
    assert route(fn, logits=P + 1, fp32=0) == ALIGN
    assert route(fn, bias=S + 2) == ALIGN


def test_route_bwd_refuses(fn):
    def call(dw=P, l=Q, ids=R, dl=S, T=4, E=8, ldl=8, ldd=8, k=2, score=0):
        return fn("det_moe_route_bwd")(dw, l, 1, ids, dl, T, E, ldl, ldd, k, score, 1, 1.0, None)
    for bad in (dict(T=-1), dict(k=9), dict(score=-1), dict(ldd=7), dict(dl=None), dict(dl=Q), dict(dw=None)):
        assert call(**bad) == INVALID, bad
    assert call(T=0, dl=None) == OK


def test_dispatch_refuses(fn):
    def call(ids=P, off=Q, rows=R, slots=S, T=4, E=8, k=2):
        return fn("det_moe_dispatch")(ids, off, rows, slots, T, E, k, None)
    for bad in (dict(T=-1), dict(E=0), dict(E=513), dict(k=0), dict(k=33), dict(off=None), dict(rows=None), dict(slots=R),
                dict(T=1 << 30, k=8)):
        assert call(**bad) == INVALID, bad


def test_rows_refuse(fn):
    def gather(x=P, rows=Q, xs=R, T=4, n=8, H=64, k=2, ldx=64, ldxs=64):
        return fn("det_moe_gather")(x, rows, xs, T, n, H, k, ldx, ldxs, None)
    for bad in (dict(T=-1), dict(k=0), dict(ldx=63), dict(ldxs=56), dict(x=None), dict(rows=None), dict(xs=P)):
        assert gather(**bad) == INVALID, bad
    assert gather(x=P + 8) == ALIGN and gather(ldx=68) == ALIGN and gather(n=0) == OK and gather(H=0) == OK

    def combine(ys=P, slots=Q, w=R, y=S, T=4, n=8, H=64, k=2, ldys=64, ldy=64):
        return fn("det_moe_combine")(ys, slots, w, y, T, n, H, k, ldys, ldy, None)
    for bad in (dict(k=33), dict(ldy=63), dict(y=P), dict(slots=None), dict(y=R), dict(H=-1)):
        assert combine(**bad) == INVALID, bad
    assert combine(T=0) == OK

    def bwd(dy=P, ys=Q, rows=R, slots=S, w=W, dys=2 * W, dw=3 * W, T=4, H=64, k=2, ld=64):
        return fn("det_moe_combine_bwd")(dy, ys, rows, slots, w, dys, dw, T, H, k, ld, ld, ld, None)
    for bad in (dict(k=0), dict(w=None), dict(dw=None), dict(dys=P), dict(ld=56)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(ld=68) == ALIGN


def test_quantisers_refuse(fn):
    def rows(x=P, r=None, q=Q, s=R, T=4, M=4, K=256, k=1, ldx=256, ldq=256, lds=4):
        return fn("det_fp8_quantize_rows")(x, r, q, s, T, M, K, k, ldx, ldq, lds, None)
    for bad in (dict(M=5), dict(k=0), dict(ldq=255), dict(lds=3), dict(q=None), dict(s=None), dict(q=P), dict(T=-1, M=-1)):
        assert rows(**bad) == INVALID, bad
    assert rows(ldq=264) == ALIGN and rows(q=Q + 8) == ALIGN and rows(T=0, M=0) == OK

    def cols(x=P, off=None, q=Q, s=R, M=200, K=64, G=0, nb=2, ldx=64, ldq=256, lds=64):
        return fn("det_fp8_quantize_cols")(x, off, q, s, M, K, G, nb, ldx, ldq, lds, None)
    for bad in (dict(nb=1), dict(off=S, G=2, nb=3, ldq=384), dict(ldq=128), dict(G=513), dict(lds=63), dict(x=None)):
        assert cols(**bad) == INVALID, bad
    assert cols(M=0) == OK

    def tiles(w=P, q=Q, s=R, qt=None, st=None, G=1, N=64, K=64, ld=64, g=4096):
        return fn("det_fp8_quantize_tiles")(w, q, s, qt, st, G, N, K, ld, g, ld, g, ld, g, None)
    for bad in (dict(s=None), dict(qt=S), dict(ld=63), dict(G=-1), dict(G=2, g=100), dict(w=Q)):
        assert tiles(**bad) == INVALID, bad
    assert tiles(G=0) == OK and tiles(q=None, s=None) == OK


def gemm(fn, a=P, sa=Q, w=R, sb=S, c=W, f32=0, M=4, N=32, K=256, lda=256, sr=1, sk=4, ldw=256, sbr=2, ldc=32):
    return fn("det_fp8_gemm")(a, sa, w, sb, c, f32, M, N, K, lda, sr, sk, ldw, sbr, ldc, None)


@pytest.mark.parametrize("bad", [dict(M=-1), dict(N=-1), dict(K=-1), dict(a=None), dict(sa=None), dict(w=None), dict(sb=None),
                                 dict(c=None), dict(lda=240), dict(ldw=128), dict(ldc=24), dict(sbr=1), dict(sr=-1), dict(c=P),
                                 dict(c=R)])
def test_product_refuses(fn, bad):
    assert gemm(fn, **bad) == INVALID


def test_product_misaligned_and_empty(fn):
    assert gemm(fn, a=P + 8) == ALIGN and gemm(fn, lda=264) == ALIGN and gemm(fn, ldc=36) == ALIGN
    assert gemm(fn, M=0, c=None) == OK and gemm(fn, N=0, c=None) == OK


def test_grouped_and_weight_gradient_refuse(fn):
    def grouped(off=2 * W, G=2, gw=32 * 256, M=4, c=W, gsb=2):
        return fn("det_fp8_gemm_grouped")(P, Q, R, S, off, c, 0, G, M, 32, 256, 256, 1, 4, 256, gw, 2, gsb, 32, None)
    for bad in (dict(off=None), dict(G=513), dict(G=-1), dict(gw=100), dict(gsb=1), dict(c=R)):
        assert grouped(**bad) == INVALID, bad
    assert grouped(gw=32 * 256 + 8) == ALIGN

    def wgrad(y=P, sy=Q, x=R, sx=S, off=None, G=1, M=200, nb=2, d=W, ldy=256, gd=0, ldd=64):
        return fn("det_fp8_gemm_wgrad")(y, sy, x, sx, off, d, 0, G, M, 32, 64, nb, ldy, 32, 256, 64, ldd, gd, None)
    for bad in (dict(G=2), dict(nb=1), dict(y=None), dict(d=None), dict(ldd=56), dict(ldy=128), dict(d=P),
                dict(off=2 * W, G=2, nb=4, ldy=512, gd=10)):
        assert wgrad(**bad) == INVALID, bad
    assert wgrad(G=0, off=2 * W, nb=2, d=None) == OK


def test_embedding_refuses(fn):
    def look(t=P, i64=1, w=Q, o=R, T=4, V=10, H=64, ldt=64, ldo=64):
        return fn("det_embedding")(t, i64, w, o, T, V, H, 1.0, ldt, ldo, None)
    for bad in (dict(T=-1), dict(t=None), dict(w=None), dict(o=Q), dict(ldt=63)):
        assert look(**bad) == INVALID, bad
    assert look(t=P + 4) == ALIGN and look(T=0) == OK

    size = fn("det_embedding_grad_workspace")(4, 10, 64)
    assert size > 0

    def grad(dy=P, t=Q, d=R, T=4, V=10, H=64, pad=-1, acc=0, ldd=64, ws=S, n=size):
        return fn("det_embedding_grad")(dy, t, 1, d, 0, T, V, H, 1.0, pad, acc, 64, ldd, ws, n, None)
    for bad in (dict(T=-1), dict(pad=10), dict(pad=-2), dict(d=None), dict(d=P), dict(ws=None), dict(n=size - 1), dict(ldd=63),
                dict(ws=R)):
        assert grad(**bad) == INVALID, bad
    assert grad(ws=S + 16) == ALIGN and grad(V=0) == OK and grad(T=0, acc=1) == OK


def test_valid_arguments_without_a_gpu_report_unsupported_device(fn):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert route(fn) == NO_DEVICE and gemm(fn) == NO_DEVICE
    assert fn("det_ops_check")(None) == NO_DEVICE


def test_binding_refuses_tensors_before_any_call(dg):
    x = torch.zeros(4, 8)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    q = torch.zeros(4, 16).to(torch.float8_e4m3fn)
    for call in (lambda: dg.det_moe_route(x, 2), lambda: dg.det_moe_dispatch(ids, 8),
                 lambda: dg.det_moe_gather(x.bfloat16(), ids[:, 0].contiguous(), 1),
                 lambda: dg.det_fp8_quantize_rows(x.bfloat16()),
                 lambda: dg.det_embedding(torch.zeros(3, dtype=torch.int64), x.bfloat16())):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    for call in (lambda: dg.det_moe_route(x.double(), 2), lambda: dg.det_fp8_quantize_rows(x),
                 lambda: dg.det_embedding(x[0], x), lambda: dg.det_fp8_gemm(x, x, q, x),
                 lambda: dg.det_moe_dispatch(ids.long(), 8)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="2-D"):
        dg.det_moe_dispatch(ids[:, 0], 8)
