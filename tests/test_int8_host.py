"""Refusals of the 8-bit integer operators: host checks before any launch, no GPU needed."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

import routed_moe_swiglu_b200 as rm

F = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first


def at(n):
    return ctypes.c_void_p((1 << 20) + n)


def test_int8_plans():
    def plan(**kw):
        return rm.moe_plan_create(**dict(dict(hidden=2048, ffn=1024, num_experts=128, top_k=8, capacity=256,
                                              precision="int8"), **kw))

    p, b = plan(), plan(precision="bf16")
    assert p.precision == "int8"
    wb = rm.moe_weight_buffer_bytes(p)  # a byte per weight and a scale per channel
    assert 3 * 128 * 2048 * 1024 + 128 * 4096 * 4 <= wb < 0.52 * rm.moe_weight_buffer_bytes(b)
    assert rm.moe_weight_buffer_bytes(plan(squared_relu=True)) < wb
    assert plan(hidden=2056, ffn=1032).hidden == 2056
    for kw, code in ((dict(hidden=2052), 2), (dict(ffn=1025), 2), (dict(keep_h_fp32=True), 1), (dict(hidden=16392), 2)):
        with pytest.raises(rm.MoeError) as e:
            plan(**kw)
        assert e.value.code == code, kw


def test_quantize_rejects_bad_arguments():
    def call(x=F, rows=4, cols=64, ld=64, q=F, s=F):
        return rm.load_library().int8_quantize_rows(x, rows, cols, ld, q, s, None, None)

    for kw in (dict(x=None), dict(q=None), dict(s=None), dict(rows=-1), dict(cols=0), dict(ld=56)):
        assert call(**kw) == 1, kw
    assert call(cols=60) == 2
    for kw in (dict(ld=68), dict(x=at(8)), dict(q=at(4)), dict(s=at(2))):
        assert call(**kw) == 3, kw
    assert call(rows=0) == 0


def test_products_reject_bad_arguments():
    lib = rm.load_library()
    nb = rm.int8_linear_workspace_bytes(4, 64)

    def matmul(x=F, xs=F, rows=4, K=64, ld=64, w=F, ws=F, N=32, out=F, ldo=32, bf16=0):
        return lib.int8_matmul(x, xs, rows, K, ld, w, ws, N, out, ldo, bf16, None, None, None)

    def linear(x=F, rows=4, K=64, ld=64, w=F, ws=F, N=32, out=F, ldo=32, bf16=0, buf=F, n=nb):
        return lib.int8_linear(x, rows, K, ld, w, ws, N, out, ldo, bf16, None, buf, n, None, None)

    for call in (matmul, linear):
        for kw in (dict(x=None), dict(w=None), dict(ws=None), dict(out=None), dict(rows=-1), dict(K=0), dict(N=0),
                   dict(ld=48), dict(ldo=31)):
            assert call(**kw) == 1, (call, kw)
        big = dict(K=rm.MOE_INT8_MAX_K + 16, ld=rm.MOE_INT8_MAX_K + 16)
        for kw in (dict(K=40, ld=48), big, dict(rows=(1 << 24) + 1), dict(N=(1 << 20) + 1, ldo=(1 << 20) + 1)):
            assert call(**kw, **({"n": 1 << 60} if call is linear else {})) == 2, (call, kw)
        for kw in (dict(x=at(8)), dict(w=at(8)), dict(ws=at(2)), dict(out=at(2)), dict(out=at(1), bf16=1), dict(ld=68)):
            assert call(**kw) == 3, (call, kw)
        assert call(rows=0, **({"n": 1 << 20} if call is linear else {})) == 0
    assert matmul(xs=None) == 1 and matmul(ld=72) == 3
    assert linear(buf=None) == 1 and linear(n=nb - 1) == 4 and linear(buf=at(64)) == 3
    assert rm.int8_linear_workspace_bytes(-1, 64) == 0 and rm.int8_linear_workspace_bytes(3, 0) == 0
    assert rm.int8_linear_workspace_bytes(100, 256) >= 100 * 260


def test_no_rows():
    """An empty tensor's pointer is null: with no rows the rows' pointers are not asked for."""
    lib = rm.load_library()
    assert lib.int8_quantize_rows(None, 0, 64, 64, None, None, None, None) == 0
    assert lib.int8_matmul(None, None, 0, 64, 64, F, F, 32, None, 32, 0, None, None, None) == 0
    assert lib.int8_linear(None, 0, 64, 64, F, F, 32, None, 32, 1, None, F, 256, None, None) == 0
    # what does not belong to the rows is
    assert lib.int8_matmul(None, None, 0, 64, 64, None, F, 32, None, 32, 0, None, None, None) == 1
    assert lib.int8_linear(None, 0, 64, 64, F, F, 32, None, 32, 1, None, None, 256, None, None) == 1
    assert lib.int8_quantize_rows(None, 0, 60, 64, None, None, None, None) == 2


def test_the_binding_refuses_other_types_and_shapes():
    i8, bf = torch.int8, torch.bfloat16
    x, q, s = torch.zeros(4, 64, dtype=bf), torch.zeros(4, 64, dtype=i8), torch.zeros(4)
    w, ws, out = torch.zeros(32, 64, dtype=i8), torch.zeros(32), torch.zeros(4, 32)
    buf = torch.zeros(1024, dtype=torch.uint8)
    for bad in (lambda: rm.int8_quantize_rows(x.float(), q, s), lambda: rm.int8_quantize_rows(x, q[:3], s),
                lambda: rm.int8_quantize_rows(x, q.to(torch.uint8), s), lambda: rm.int8_quantize_rows(x, q, s[:3]),
                lambda: rm.int8_quantize_rows(x.T, q, s), lambda: rm.int8_quantize_rows(x, q, s),  # host tensors
                lambda: rm.int8_matmul(q, s, w[:, :32], ws, out), lambda: rm.int8_matmul(q, s, w, ws[:31], out),
                lambda: rm.int8_matmul(q, s[:3], w, ws, out), lambda: rm.int8_matmul(q, s, w, ws, out.half()),
                lambda: rm.int8_matmul(q, s, w, ws, out[:, :31]), lambda: rm.int8_matmul(x, s, w, ws, out),
                lambda: rm.int8_matmul(q, s, w.T.contiguous().T, ws, out),
                lambda: rm.int8_linear(q, w, ws, out, buf), lambda: rm.int8_linear(x, w.float(), ws, out, buf)):
        with pytest.raises(ValueError):
            bad()


def test_the_compiled_binding_leaves_host_tensors_alone():
    rm.load_library()
    if rm._short is None:
        pytest.skip("the compiled binding is not built, or this torch has no exchange table")
    x, q, s = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    for args in ((None, x, q, s, None), (None, None, None, None, None), (None, "x", 1, object(), None), (None, x, q, s),
                 (), ("stream", x, q, s, None)):
        assert rm._short.int8_quantize_rows(*args) is None
    assert rm._short.moe_combine_backward(None, 0, s, s, s, s, s, s, s) is None
    assert rm._short.start(*[None] * 11) is False and rm._short.start() is False


def test_a_table_that_the_compiled_binding_does_not_know():
    """A capsule of another name or no capsule at all: the binding says that it cannot serve and raises
    nothing, and the library loads without it."""
    rm.load_library()
    if rm._short is None:
        pytest.skip("the compiled binding is not built, or this torch has no exchange table")
    new = ctypes.pythonapi.PyCapsule_New
    new.restype, new.argtypes = ctypes.py_object, [ctypes.c_void_p, ctypes.c_char_p, ctypes.c_void_p]
    room = (ctypes.c_uint64 * 16)()
    other = new(ctypes.addressof(room), b"some_other_table", None)
    types = (torch.Tensor, torch.nn.Parameter)
    for api in (other, 7, None, "dlpack_exchange_api"):
        assert rm._short.start(api, *types, *[1 << 20] * 8) is False
    api = torch.Tensor.__dlpack_c_exchange_api__
    for entries in ([1 << 20] * 7 + [0], [1 << 20] * 7 + [None], [1 << 20] * 7 + [-1], [1 << 20] * 7):
        assert rm._short.start(api, *types, *entries) is False
    x, q, s = (torch.zeros(4, 64, dtype=t) for t in (torch.bfloat16, torch.int8, torch.float32))
    assert rm._short.int8_quantize_rows(None, x, q, s, None) is None  # as before


def test_the_library_loads_beside_a_strange_table(monkeypatch):
    """load_library() with a torch whose exchange attribute is something else falls back to ctypes."""
    lib = rm.load_library()
    for api in (object(), 7, "dlpack_exchange_api"):
        monkeypatch.setattr(torch.Tensor, "__dlpack_c_exchange_api__", api, raising=False)
        monkeypatch.setattr(rm, "_short", None)
        rm._load_short(lib)
        assert rm._short is None


@pytest.mark.parametrize("compiler", ["/nowhere/c++", "false"])
def test_the_library_builds_without_the_binding(tmp_path, monkeypatch, capsys, compiler):
    """A missing or failing C++ compiler leaves the binding out, an older one too, and says so."""
    from routed_moe_swiglu_b200 import build

    old = tmp_path / "_binding.so"
    old.write_bytes(b"of other sources")
    monkeypatch.setattr(build, "BINDING", str(old))
    monkeypatch.setenv("CXX", compiler)
    build._build_binding(True, False)
    assert list(tmp_path.iterdir()) == [] and "the compiled binding is not built" in capsys.readouterr().err


def test_the_binding_is_built_for_one_interpreter():
    """The file's name carries this interpreter's tag, so that another Python version does not load it."""
    from importlib.machinery import EXTENSION_SUFFIXES

    from routed_moe_swiglu_b200 import build

    name = os.path.basename(build.BINDING)
    assert name == "_binding" + EXTENSION_SUFFIXES[0] != "_binding.so"
    assert not os.path.exists(os.path.join(build.PKG, "_binding.so"))
    rm.load_library()
    if rm._short is not None:
        assert rm._short.__file__ == build.BINDING


def test_an_older_binding_without_a_tag_goes(tmp_path, monkeypatch):
    from routed_moe_swiglu_b200 import build

    (tmp_path / "_binding.so").write_bytes(b"of some interpreter")
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / os.path.basename(build.BINDING)))
    monkeypatch.setenv("CXX", "false")
    build._build_binding(False, False)
    assert list(tmp_path.iterdir()) == []


def test_the_compiled_binding_serves_where_it_can():
    """With torch's exchange table, Python.h and a C++ compiler at hand the short way must be there: the
    tests that go through it skip where it is not."""
    import shutil
    import sysconfig

    if getattr(torch.Tensor, "__dlpack_c_exchange_api__", None) is None:
        pytest.skip("this torch has no exchange table")
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")) or \
            shutil.which(os.environ.get("CXX", "g++")) is None:
        pytest.skip("nothing to build it with")
    rm.load_library()
    assert rm._short is not None
