"""Host-side checks of the attention operators: exports, refusals of the C
entry points before they touch a GPU, and of the binding. No GPU needed."""
import ctypes
import os
import re

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "det_attn.h")
A = [0x100000 + 0x40000000 * i for i in range(16)]     # fake, aligned device addresses; never dereferenced here
OK, INVALID, ALIGN, NO_DEVICE = 0, 1, 3, 4
_CTYPES = {"int64_t": ctypes.c_int64, "int": ctypes.c_int, "float": ctypes.c_float, "det_gemm_stream": ctypes.c_void_p}


@pytest.fixture(scope="module")
def dg():
    from invariant_deterministic_gemm_gb300 import _build
    _build.build()
    import invariant_deterministic_gemm_gb300 as m
    m.lib()
    return m


def declared():
    """Each function of the header: its result's ctype, and its arguments' names and ctypes."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    out = {}
    for m in re.finditer(r"\b(det_gemm_status|int64_t)\s+(det_[a-z0-9_]+)\s*\(([^;]*)\);", text):
        args = [a.strip() for a in m.group(3).split(",")]
        out[m.group(2)] = (ctypes.c_int64 if m.group(1) == "int64_t" else ctypes.c_int,
                           [(a.replace("*", " ").split()[-1], ctypes.c_void_p if "*" in a else _CTYPES[a.rsplit(" ", 1)[0]]) for a in args])
    return out


@pytest.fixture(scope="module")
def call(dg):
    """call(name, **arguments): the rest from DEFAULTS."""
    d = declared()

    def go(name, **kw):
        f = getattr(ctypes.CDLL(dg.LIB_PATH), name)
        f.restype, f.argtypes = d[name][0], [t for _, t in d[name][1]]
        base = dict(DEFAULTS[name])
        assert not set(kw) - set(base), set(kw) - set(base)
        base.update(kw)
        return f(*[base[n] for n, _ in d[name][1]])
    return go


DEFAULTS = {
    "det_rope": dict(x=A[0], cosine=A[1], sine=A[2], positions=A[3], y=A[4], T=4, H=2, D=64, rot=32, P=100, interleaved=0, inverse=0,
                     xt=128, xh=64, ldt=16, yt=128, yh=64, stream=None),
    "det_kv_append": dict(q=A[0], k=A[1], v=A[2], cosine=A[3], sine=A[4], positions=A[5], slots=A[6], q_out=A[7], k_cache=A[8], v_cache=A[9],
                          T=4, H=4, KV=2, D=64, rot=64, P=100, pages=3, page_size=8, interleaved=0, qt=256, qh=64, kt=128, kh=64, vt=128, vh=64,
                          ldt=32, ot=256, oh=64, kcp=1024, kcs=128, kch=64, vcp=1024, vcs=128, vch=64, stream=None),
    "det_attn_decode_workspace": dict(B=3, H=4, KV=2, D=64, max_tokens=80),
    "det_attn_decode": dict(q=A[0], k_cache=A[1], v_cache=A[2], table=A[3], lengths=A[4], out=A[5], B=3, H=4, KV=2, D=64, pages=20, page_size=16,
                            max_pages=5, scale=0.1, window=0, sinks=0, qt=256, qh=64, kcp=2048, kcs=128, kch=64, vcp=2048, vcs=128, vch=64, ldt=5,
                            ot=256, oh=64, workspace=A[6], workspace_bytes=1 << 30, stream=None),
    "det_attn": dict(q=A[0], k=A[1], v=A[2], q_bounds=A[3], k_bounds=None, out=A[4], lse=A[5], N=2, T=10, S=10, H=4, KV=2, D=64, scale=0.1,
                     window=0, sinks=0, qt=256, qh=64, kt=128, kh=64, vt=128, vh=64, ot=256, oh=64, stream=None),
    "det_attn_bwd_workspace": dict(N=2, T=10, S=10, H=4, KV=2, D=64, window=0, sinks=0),
    "det_attn_bwd": dict(dout=A[0], q=A[1], k=A[2], v=A[3], out=A[4], lse=A[5], q_bounds=A[6], k_bounds=None, dq=A[7], dk=A[8], dv=A[9], N=2, T=10,
                         S=10, H=4, KV=2, D=64, scale=0.1, window=0, sinks=0, dot=256, doh=64, qt=256, qh=64, kt=128, kh=64, vt=128, vh=64,
                         ot=256, oh=64, dqt=256, dqh=64, dkt=128, dkh=64, dvt=128, dvh=64, workspace=A[10], workspace_bytes=1 << 30, stream=None),
}
NAN, INF = float("nan"), float("inf")
HEADS = [dict(D=0), dict(D=4), dict(D=12), dict(D=136), dict(KV=3), dict(KV=0), dict(H=0), dict(H=2048, KV=1024)]
MASK = [dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(window=-1), dict(sinks=-1)]
BAD = {
    "det_rope": [dict(T=-1), dict(H=-1), dict(H=2000), dict(D=4), dict(D=136), dict(rot=0), dict(rot=3), dict(rot=66), dict(P=-1), dict(x=None), dict(y=None),
                 dict(cosine=None), dict(positions=None), dict(xt=64), dict(yh=32), dict(ldt=8), dict(y=A[0] + 128), dict(y=A[0], yt=256),
                 dict(y=A[3]), dict(xt=1 << 40)],
    "det_kv_append": [dict(T=-1), dict(KV=0), dict(D=12), dict(page_size=0), dict(pages=1 << 30), dict(slots=None), dict(k=None), dict(k_cache=None),
                      dict(v_cache=A[8]), dict(k_cache=A[1]), dict(kcs=64), dict(vcp=512), dict(q_out=None), dict(q_out=A[0]), dict(rot=65), dict(kch=0)],
    "det_attn_decode": HEADS + MASK + [dict(B=-1), dict(H=65, KV=1), dict(page_size=4), dict(page_size=12), dict(page_size=0), dict(max_pages=-1),
                                       dict(max_pages=1 << 28), dict(pages=1 << 28), dict(ldt=4), dict(table=None), dict(lengths=None),
                                       dict(workspace=None), dict(workspace_bytes=0), dict(out=A[0]), dict(out=None), dict(kcp=1024), dict(workspace=A[5])],
    "det_attn": HEADS + MASK + [dict(N=-1), dict(T=-1), dict(S=9), dict(q_bounds=None), dict(q_bounds=None, k_bounds=A[6]), dict(T=(1 << 31) - 5000, S=(1 << 31) - 5000),
                                dict(q=None), dict(v=None), dict(out=None), dict(lse=None), dict(out=A[2]), dict(lse=A[1]), dict(kt=64), dict(oh=32)],
    "det_attn_bwd": HEADS + MASK + [dict(S=11), dict(dout=None), dict(lse=None), dict(dq=A[1]), dict(dk=A[9]), dict(workspace=None), dict(workspace=A[7]),
                                    dict(workspace_bytes=16), dict(dvt=64), dict(dv=None), dict(out=None)],
}


@pytest.mark.parametrize("name,bad", [(n, b) for n in BAD for b in BAD[n]], ids=lambda x: x if isinstance(x, str) else "-".join(x))
def test_refuses(call, name, bad):
    assert call(name, **bad) == INVALID


@pytest.mark.parametrize("name,bad", [("det_rope", dict(x=A[0] + 8)), ("det_rope", dict(xt=132)), ("det_rope", dict(cosine=A[1] + 2)), ("det_kv_append", dict(kcs=132, kcp=2048)),
                                      ("det_kv_append", dict(slots=A[6] + 1)), ("det_attn_decode", dict(qh=68, qt=512)), ("det_attn_decode", dict(workspace=A[6] + 16)),
                                      ("det_attn_decode", dict(vcs=132, vcp=4096)), ("det_attn", dict(v=A[2] + 2)), ("det_attn", dict(kt=136 + 4)),
                                      ("det_attn_bwd", dict(dq=A[7] + 8)), ("det_attn_bwd", dict(workspace=A[10] + 64))])
def test_misaligned(call, name, bad):
    assert call(name, **bad) == ALIGN


def test_empty_and_valid(call):
    assert call("det_rope", T=0) == OK and call("det_rope", H=0) == OK and call("det_kv_append", T=0) == OK
    assert call("det_attn_decode", B=0) == OK and call("det_attn", T=0, S=0) == OK and call("det_attn_bwd", T=0, S=0) == OK
    if not torch.cuda.is_available():
        for name in BAD:
            assert call(name) == NO_DEVICE, name
        assert call("det_rope", y=A[0]) == NO_DEVICE                    # in place
        assert call("det_kv_append", q=None, q_out=None) == NO_DEVICE
        assert call("det_attn", q_bounds=None, N=1, S=50) == NO_DEVICE
        assert call("det_attn", k_bounds=A[6], S=50) == NO_DEVICE


def test_workspaces(call):
    assert call("det_attn_decode_workspace") > 0 and call("det_attn_decode_workspace", B=-1) == 0
    assert call("det_attn_bwd_workspace") >= 4 * 10 * 4 and call("det_attn_bwd_workspace", H=3) == 0
    assert call("det_attn_bwd_workspace", window=100, sinks=4) > call("det_attn_bwd_workspace", window=100) and call("det_attn_bwd_workspace", sinks=-1) == 0


def test_exports(dg):
    names = declared()
    assert len(names) == 7
    for n in names:
        assert hasattr(dg.lib(), n), n
        if not n.endswith("_workspace"):
            assert callable(getattr(dg, n)) and n in dg.__all__, n


def test_binding_refuses_tensors_before_any_call(dg):
    x, i = torch.zeros(4, 2, 64).bfloat16(), torch.zeros(4, dtype=torch.int32)
    c = torch.zeros(10, 16)
    for f in (lambda: dg.det_rope(x, c, c, i), lambda: dg.det_attn(x, x, x), lambda: dg.det_attn_bwd(x, x, x, x, x, c),
              lambda: dg.det_kv_append(None, x, x, c, c, i, i, x[None], x[None]), lambda: dg.det_attn_decode(x, x[None], x[None], i[None], i)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()
    for f in (lambda: dg.det_rope(x.float(), c, c, i), lambda: dg.det_attn(x.half(), x, x), lambda: dg.det_attn(None, x, x)):
        with pytest.raises(TypeError):
            f()


@pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.device_count() < 2, reason="a fake tensor of cuda:1 needs none or two GPUs")
def test_tensors_of_different_devices_are_refused(dg):
    with FakeTensorMode():
        def t(dtype, *shape, device="cuda:0"):
            return torch.empty(shape, dtype=dtype, device=device)
        f32, i32, bf16, far = torch.float32, torch.int32, torch.bfloat16, dict(device="cuda:1")
        x, c, i = t(bf16, 4, 2, 64), t(f32, 10, 16), t(i32, 4)
        y, kc = t(bf16, 4, 2, 64, **far), t(bf16, 3, 8, 2, 64)
        for n, f in enumerate([lambda: dg.det_rope(x, c, c, t(i32, 4, **far)), lambda: dg.det_rope(x, c, c, i, out=y),
                               lambda: dg.det_kv_append(x, x, x, c, c, i, i, kc, t(bf16, 3, 8, 2, 64, **far)),
                               lambda: dg.det_attn_decode(x, kc, kc, t(i32, 4, 2, **far), i), lambda: dg.det_attn(x, x, y),
                               lambda: dg.det_attn(x, x, x, t(i32, 3, **far)), lambda: dg.det_attn_bwd(y, x, x, x, x, t(f32, 2, 4))]):
            with pytest.raises(ValueError, match="different devices: cuda:[01] and cuda:[01]"):
                f()
                pytest.fail("call %d was not refused" % n)


# Keys and values in one buffer: [pages, 2, size, KV, D], [pages, size, 2, KV, D], [pages, size, KV, 2, D].
BETWEEN = [(2048, dict(kcp=2048, vcp=2048)), (256, dict(kcp=2048, vcp=2048, kcs=256, vcs=256)),
           (128, dict(kcp=2048, vcp=2048, kcs=256, vcs=256, kch=128, vch=128))]


@pytest.mark.parametrize("at,strides", BETWEEN)
@pytest.mark.parametrize("first", ["k_cache", "v_cache"])
def test_caches_that_lie_between_one_another(call, at, strides, first):
    second = "v_cache" if first == "k_cache" else "k_cache"
    if not torch.cuda.is_available():
        assert call("det_kv_append", **{first: A[8], second: A[8] + at}, **strides) == NO_DEVICE
    for off in (0, at // 2, at + 16, 2 * at + 64):
        assert call("det_kv_append", **{first: A[8], second: A[8] + off}, **strides) in (INVALID, ALIGN), off


def test_rows_times_heads_below_two_to_the_31(call):
    assert call("det_attn_decode", B=1 << 21, H=1024, KV=1024) == INVALID
    assert call("det_attn_decode_workspace", B=1 << 21, H=1024, KV=1024) == 0
