"""Checks of include/wtconv_block.h and its binding that need no GPU: every
declared entry point is exported with the declared argument kinds, and each
call refuses bad arguments with a status before it touches the device."""
import ctypes
import os
import re

import pytest
import torch

from conftest import ROOT

from memory_bound_cnn_wtconv2d_gb300 import blockops, build, wtconv

FAKE = 0x10000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def L():
    build.build()
    return blockops.lib()


def prototypes():
    src = open(os.path.join(ROOT, "include", "wtconv_block.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    out = {}
    for m in re.finditer(r"\b(wtconv_\w+)\s*\(([^;{]*?)\)\s*;", src):
        out[m.group(1)] = [a.strip() for a in m.group(2).split(",") if a.strip() not in ("", "void")]
    return out


def test_every_declared_entry_point_is_bound(L):
    protos = prototypes()
    assert sorted(protos) == sorted(blockops.EXPORTS)
    for name, params in protos.items():
        argtypes = getattr(L, name).argtypes
        assert len(argtypes) == len(params), name
        for decl, t in zip(params, argtypes):
            if "*" in decl:
                assert t in (ctypes.c_void_p, ctypes.POINTER(blockops.GnDesc), ctypes.POINTER(blockops.NsDesc)), decl
            else:
                kind = {"size_t": ctypes.c_size_t, "long long": ctypes.c_longlong, "float": ctypes.c_float,
                        "int": ctypes.c_int}[re.match(r"size_t|long long|float|int", decl).group(0)]
                assert t is kind, (name, decl)


def test_descriptors_match_the_header():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "wtconv_block.h")).read(), flags=re.S)
    for struct, name in ((blockops.GnDesc, "wtconv_gn_desc_t"), (blockops.NsDesc, "wtconv_ns_desc_t")):
        body = re.search(r"typedef struct \{([^}]*)\} " + name, src).group(1)
        fields = [f.strip() for line in body.split(";") if line.strip()
                  for f in re.sub(r"^\s*(long long|int|float)\s", "", line.strip()).split(",")]
        assert fields == [f for f, _ in struct._fields_]


def gn(N=2, S=9, C=16, G=4, dtype=0, act=1, eps=1e-5, xs=None, xr=None):
    S_, C_ = max(S, 0), max(C, 0)
    xs, xr = S_ * C_ if xs is None else xs, C_ if xr is None else xr
    return blockops.GnDesc(N, S, C, G, dtype, act, eps, xs, xr, S_ * C_, C_)


def call_gn_fwd(L, d, x=FAKE, y=FAKE, mean=FAKE, ws=FAKE, n=1 << 30):
    p = lambda v: ctypes.c_void_p(v) if v else None  # noqa: E731
    return L.wtconv_gn_act_fwd(ctypes.byref(d), p(x), None, None, p(y), p(mean), p(FAKE), p(ws), n, None)


@pytest.mark.parametrize("over,status", [
    (dict(N=-1), 1), (dict(S=-1), 1), (dict(C=0), 1), (dict(G=0), 1), (dict(G=3), 1), (dict(dtype=3), 1),
    (dict(act=3), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(xr=-1), 1), (dict(C=16384), 2),
    (dict(N=70000), 2), (dict(S=1 << 31), 2), (dict(xs=1 << 61), 2)])
def test_group_norm_descriptors_refused(L, over, status):
    d = gn(**over)
    assert call_gn_fwd(L, d) == status
    assert L.wtconv_last_error().decode()
    assert L.wtconv_gn_workspace_size(ctypes.byref(d), blockops.OP_GN_FWD) == 0


def test_group_norm_pointers_refused(L):
    d = gn(N=64, S=100000)
    assert call_gn_fwd(L, d, x=0) == wtconv.WTCONV_ERR_INVALID_ARG
    assert call_gn_fwd(L, d, mean=0) == wtconv.WTCONV_ERR_INVALID_ARG
    assert call_gn_fwd(L, d, y=FAKE + 2) == wtconv.WTCONV_ERR_MISALIGNED
    need = L.wtconv_gn_workspace_size(ctypes.byref(d), blockops.OP_GN_BWD)
    assert need > 0 and need % 256 == 0
    p = ctypes.c_void_p(FAKE)
    assert L.wtconv_gn_act_bwd(ctypes.byref(d), p, p, p, p, None, None, p, p, p, p, need - 1, None) == \
        wtconv.WTCONV_ERR_WORKSPACE
    assert L.wtconv_gn_act_bwd(ctypes.byref(d), p, p, p, p, None, None, p, p, p, ctypes.c_void_p(FAKE + 16), need,
                               None) == wtconv.WTCONV_ERR_MISALIGNED
    assert L.wtconv_gn_act_fwd(None, p, None, None, p, p, p, p, need, None) == wtconv.WTCONV_ERR_INVALID_ARG


def ns(count=2, m=200, n=300, dtype=0, steps=5, a=3.4, b=-4.7, c=2.0, eps=1e-7):
    return blockops.NsDesc(count, m, n, dtype, steps, a, b, c, eps)


def call_orth(L, d, ld=300, ptrs=(FAKE, FAKE), out=(FAKE, FAKE), ws=FAKE, n=None):
    arr = lambda v: (ctypes.c_void_p * len(v))(*v)  # noqa: E731
    n = L.wtconv_ns_workspace_size(ctypes.byref(d)) if n is None else n
    return L.wtconv_orthogonalize(ctypes.byref(d), arr(ptrs), ld, arr(out), 300, ctypes.c_void_p(ws) if ws else None, n, None)


@pytest.mark.parametrize("over,status", [
    (dict(count=-1), 1), (dict(m=-1), 1), (dict(n=-1), 1), (dict(dtype=5), 1), (dict(steps=-1), 1), (dict(steps=65), 1),
    (dict(a=17.0), 1), (dict(b=float("nan")), 1), (dict(c=float("inf")), 1), (dict(eps=-1.0), 1), (dict(count=65), 2),
    (dict(m=40000), 2)])
def test_matrix_descriptors_refused(L, over, status):
    d = ns(**over)
    assert call_orth(L, d, n=1 << 40) == status
    assert L.wtconv_ns_workspace_size(ctypes.byref(d)) == 0


def test_matrix_pointers_refused(L):
    d = ns()
    assert call_orth(L, d, ld=299) == wtconv.WTCONV_ERR_INVALID_ARG
    assert call_orth(L, d, ptrs=(FAKE, 0)) == wtconv.WTCONV_ERR_INVALID_ARG
    assert call_orth(L, d, out=(FAKE, FAKE + 2)) == wtconv.WTCONV_ERR_MISALIGNED
    assert call_orth(L, d, ws=0) == wtconv.WTCONV_ERR_WORKSPACE
    assert call_orth(L, d, n=16) == wtconv.WTCONV_ERR_WORKSPACE
    assert call_orth(L, d, ws=FAKE + 8) == wtconv.WTCONV_ERR_MISALIGNED
    arr = (ctypes.c_void_p * 2)(FAKE, FAKE)
    need = L.wtconv_ns_workspace_size(ctypes.byref(d))
    p = ctypes.c_void_p(FAKE)
    step = lambda mu, rate: L.wtconv_muon_step(ctypes.byref(d), arr, 300, arr, 300, arr, 300, mu, 1, 1.0, rate, p, need, None)  # noqa: E731
    assert step(float("nan"), 0.1) == wtconv.WTCONV_ERR_INVALID_ARG
    assert step(0.9, float("inf")) == wtconv.WTCONV_ERR_INVALID_ARG
    assert L.wtconv_muon_step(ctypes.byref(d), None, 300, arr, 300, arr, 300, 0.9, 1, 1.0, 0.1, p, need, None) == \
        wtconv.WTCONV_ERR_INVALID_ARG


def test_empty_calls_need_nothing(L):
    assert L.wtconv_gn_act_fwd(ctypes.byref(gn(N=0)), None, None, None, None, None, None, None, 0, None) == 0
    d = ns(m=0)
    assert L.wtconv_ns_workspace_size(ctypes.byref(d)) == 0
    assert L.wtconv_orthogonalize(ctypes.byref(d), None, 12, None, 12, None, 0, None) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError):
        blockops.wtconv_gn_act_fwd(x, 2)
    with pytest.raises(ValueError):
        blockops.wtconv_orthogonalize(torch.zeros(3, 4))


def test_modules_refuse_bad_shapes():
    from memory_bound_cnn_wtconv2d_gb300.block import WTConvBlock, block_optimizers
    from memory_bound_cnn_wtconv2d_gb300.muon import Muon, shape_scale
    from memory_bound_cnn_wtconv2d_gb300.norm import GroupNormAct
    for args in ((3, 16), (0, 16), (4, 0)):
        with pytest.raises(ValueError):
            GroupNormAct(*args)
    with pytest.raises(ValueError):
        GroupNormAct(4, 16, activation="relu")
    assert shape_scale(400, 100) == 2.0 and shape_scale(100, 400) == 1.0
    assert shape_scale(100, 400, "rms") == pytest.approx(4.0)
    with pytest.raises(ValueError):
        shape_scale(1, 1, "other")
    block = WTConvBlock(16, levels=1, num_groups=4)
    muon, adam = block_optimizers(block)
    assert isinstance(muon, Muon)
    taken = [p for o in (muon, adam) for g in o.param_groups for p in g["params"]]
    assert sorted(map(id, taken)) == sorted(map(id, block.parameters()))


def test_matrices_side_by_side_or_overlapping():
    def stack(ts):
        s = blockops._Stack.__new__(blockops._Stack)
        s.tensors = ts
        s.m, s.n = ts[0].shape
        s.ld = ts[0].stride(0)
        s.pointers = [t.data_ptr() for t in ts]
        return s
    big = torch.zeros(6, 20)
    stack([big[:, :10], big[:, 10:]]).separate("w")
    stack([big[:3], big[3:]]).separate("w")
    for ts in ([big[:, :10], big[:, 9:19]], [big[:3], big[2:5]], [big, big], [big[:, :10], big[1:, :10][:5]]):
        with pytest.raises(ValueError):
            stack(ts).separate("w")
