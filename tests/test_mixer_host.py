"""Checks of include/wtconv_mixer.h and its binding that need no GPU: every
declared entry point is exported with the declared argument kinds, and each
call refuses bad arguments with a status before it touches the device."""
import ctypes
import os
import re

import pytest
import torch

from conftest import ROOT

from memory_bound_cnn_wtconv2d_gb300 import build, mixerops, wtconv

FAKE = 0x10000  # never dereferenced: every call below fails validation first
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    build.build()
    return mixerops.lib()


def header():
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "wtconv_mixer.h")).read(), flags=re.S)


def test_every_declared_entry_point_is_bound(L):
    protos = {m.group(1): [a.strip() for a in m.group(2).split(",") if a.strip() not in ("", "void")]
              for m in re.finditer(r"\b(wtconv_\w+)\s*\(([^;{]*?)\)\s*;", header())}
    assert sorted(protos) == sorted(mixerops.EXPORTS)
    descs = {"wtconv_rms_desc_t": mixerops.RmsDesc, "wtconv_gated_desc_t": mixerops.GatedDesc, "wtconv_tensor_t": mixerops.Tensor}
    kinds = {"size_t": ctypes.c_size_t, "float": ctypes.c_float, "int": ctypes.c_int}
    for name, params in protos.items():
        argtypes = getattr(L, name).argtypes
        assert len(argtypes) == len(params), name
        for decl, t in zip(params, argtypes):
            if "*" in decl:
                d = next((v for k, v in descs.items() if k in decl), None)
                assert t is (ctypes.POINTER(d) if d else ctypes.c_void_p), (name, decl)
            else:
                assert t is kinds[decl.split()[0]], (name, decl)


def test_descriptors_match_the_header():
    for struct, name in ((mixerops.RmsDesc, "wtconv_rms_desc_t"), (mixerops.GatedDesc, "wtconv_gated_desc_t"),
                         (mixerops.Tensor, "wtconv_tensor_t")):
        body = re.search(r"typedef struct \{([^}]*)\} " + name, header()).group(1)
        fields = [f.strip() for line in body.split(";") if line.strip()
                  for f in re.sub(r"^\s*(long long|int|float|void\*)\s", "", line.strip()).split(",")]
        assert fields == [f for f, _ in struct._fields_]


P = ctypes.c_void_p


def rms(M=4, C=64, dtype=0, eps=1e-6, xs=64, rs=64, ds=64):
    return mixerops.RmsDesc(M, C, dtype, eps, xs, rs, ds)


@pytest.mark.parametrize("over,status", [
    (dict(M=-1), INVALID), (dict(C=0), INVALID), (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(xs=63), INVALID), (dict(xs=-1), INVALID), (dict(rs=5), INVALID),
    (dict(C=16385, xs=16385, rs=16385), UNSUPPORTED), (dict(M=1 << 31), UNSUPPORTED), (dict(xs=1 << 40), UNSUPPORTED)])
def test_norm_descriptors_refused(L, over, status):
    d = rms(**over)
    p = P(FAKE)
    assert L.wtconv_rms_norm_fwd(ctypes.byref(d), p, p, None, p, p, p, None) == status
    assert L.wtconv_last_error().decode()
    assert L.wtconv_rms_norm_q8(ctypes.byref(d), p, p, None, p, p, p, None) == status


def test_norm_pointers_refused(L):
    d, p = rms(), P(FAKE)
    ref = ctypes.byref(d)
    assert L.wtconv_rms_norm_fwd(None, p, p, None, p, p, p, None) == INVALID
    assert L.wtconv_rms_norm_fwd(ref, None, p, None, p, p, p, None) == INVALID
    assert L.wtconv_rms_norm_fwd(ref, p, p, None, None, p, p, None) == INVALID
    assert L.wtconv_rms_norm_fwd(ref, p, p, None, p, p, None, None) == INVALID
    assert L.wtconv_rms_norm_fwd(ref, P(FAKE + 2), p, None, p, p, p, None) == MISALIGNED
    assert L.wtconv_quantize_rows(ref, p, None, p, None) == INVALID
    need = L.wtconv_rms_workspace_size(ref)
    assert need > 0 and need % 256 == 0 and L.wtconv_rms_workspace_size(ctypes.byref(rms(C=0))) == 0
    bwd = lambda dw, ws, n, rstd=p: L.wtconv_rms_norm_bwd(ref, p, p, None, rstd, None, p, dw, ws, n, None)  # noqa: E731
    assert bwd(p, p, need - 1) == WORKSPACE and bwd(p, None, need) == WORKSPACE
    assert bwd(p, P(FAKE + 16), need) == MISALIGNED and bwd(p, p, need, None) == INVALID
    assert L.wtconv_rms_norm_bwd(ctypes.byref(rms(ds=3)), p, p, None, p, None, p, p, p, need, None) == INVALID


def gated(M=300, C=64, H=48, dtype=2, act=1, xs=64, gs=64, us=64, ds=48):
    return mixerops.GatedDesc(M, C, H, dtype, act, xs, gs, us, ds)


@pytest.mark.parametrize("over,status", [
    (dict(M=-1), INVALID), (dict(C=0), INVALID), (dict(H=0), INVALID), (dict(dtype=3), INVALID), (dict(act=3), INVALID),
    (dict(act=-1), INVALID), (dict(xs=63), INVALID), (dict(gs=1), INVALID), (dict(us=-64), INVALID),
    (dict(M=1 << 31), UNSUPPORTED), (dict(H=65537), UNSUPPORTED), (dict(C=65537, xs=65537, gs=65537, us=65537), UNSUPPORTED),
    (dict(xs=1 << 40), UNSUPPORTED)])
def test_gated_descriptors_refused(L, over, status):
    d, p = gated(**over), P(FAKE)
    ref = ctypes.byref(d)
    assert L.wtconv_gated_fwd(ref, p, p, p, p, p, 1 << 50, None) == status
    assert L.wtconv_gated_bwd(ref, p, p, p, p, p, p, p, p, 1 << 50, None) == status
    assert L.wtconv_gated_workspace_size(ref, mixerops.OP_GATED_FWD) == 0
    assert L.wtconv_last_error().decode()


def test_gated_pointers_refused(L):
    d, p = gated(), P(FAKE)
    ref = ctypes.byref(d)
    big = 1 << 50
    assert L.wtconv_gated_fwd(None, p, p, p, p, p, big, None) == INVALID
    assert L.wtconv_gated_fwd(ref, None, p, p, p, p, big, None) == INVALID
    assert L.wtconv_gated_fwd(ref, p, P(FAKE + 1), p, p, p, big, None) == MISALIGNED
    assert L.wtconv_gated_fwd(ref, p, p, p, None, p, big, None) == INVALID
    need = L.wtconv_gated_workspace_size(ref, mixerops.OP_GATED_BWD)
    assert need > 0 and need % 256 == 0 and L.wtconv_gated_workspace_size(ref, 3) == 0
    bwd = lambda dx, dg, du, ws, n: L.wtconv_gated_bwd(ref, p, p, p, p, dx, dg, du, ws, n, None)  # noqa: E731
    assert bwd(p, p, p, p, need - 1) == WORKSPACE and bwd(p, p, p, None, need) == WORKSPACE
    assert bwd(p, p, p, P(FAKE + 16), need) == MISALIGNED and bwd(p, p, None, p, need) == INVALID
    assert L.wtconv_gated_bwd(ctypes.byref(gated(ds=3)), p, p, p, p, p, p, p, p, big, None) == INVALID
    q8 = lambda d, x=p, s=p: L.wtconv_gated_q8(ctypes.byref(d), x, s, p, p, p, p, p, p, big, None)  # noqa: E731
    assert q8(gated(C=72, xs=80, gs=80, us=80)) == UNSUPPORTED and q8(gated(xs=72)) == UNSUPPORTED
    assert q8(gated(), P(FAKE + 8)) == MISALIGNED and q8(gated(), p, None) == INVALID


def test_lists_refused(L):
    entry = lambda data=FAKE, n=10, t=0: (mixerops.Tensor * 1)(mixerops.Tensor(data, n, t))  # noqa: E731
    need = L.wtconv_clip_workspace_size(1)
    p = P(FAKE)
    assert need > 0 and need % 256 == 0 and L.wtconv_clip_workspace_size(-1) == 0
    norm = lambda e, n=1, ws=p, b=need, out=p: L.wtconv_grad_norm(e, n, out, ws, b, None)  # noqa: E731
    assert norm(entry(), -1) == INVALID and norm(None) == INVALID and norm(entry(t=3)) == INVALID
    assert norm(entry(n=-1)) == INVALID and norm(entry(data=0)) == INVALID and norm(entry(data=FAKE + 2)) == MISALIGNED
    assert norm(entry(n=1 << 44)) == UNSUPPORTED and norm(entry(), out=None) == INVALID
    assert norm(entry(), ws=None) == WORKSPACE and norm(entry(), b=need - 1) == WORKSPACE
    for limit, eps in ((-1.0, 0.0), (float("nan"), 0.0), (1.0, -1.0), (1.0, float("inf"))):
        assert L.wtconv_clip_grads(entry(), 1, limit, eps, p, p, need, None) == INVALID


def test_lists_that_overlap_refused(L):
    p, need = P(FAKE), L.wtconv_clip_workspace_size(3)

    def status(*spans):  # (start, bytes, type); norm = NULL is refused after the overlap
        e = (mixerops.Tensor * len(spans))(*[mixerops.Tensor(a, n // (2 if t else 4), t) for a, n, t in spans])
        s = L.wtconv_clip_grads(e, len(spans), 1.0, 0.0, None, p, need, None)
        return s == INVALID and "overlap" in L.wtconv_last_error().decode()

    assert status((4096, 64, 0), (8192, 64, 0), (4156, 8, 1)) and status((4096, 64, 0), (4096, 64, 0))
    assert status((8192, 4, 0), (4096, 4098, 2)) and not status((4096, 64, 0), (4160, 64, 1), (4032, 64, 2))
    assert not status((4096, 64, 0), (4096, 0, 0), (4100, 0, 1))


def test_the_binding_knows_dense_tensors():
    t = torch.zeros(4, 6, 5)
    for d in (t, t.permute(2, 0, 1), t[1], t[:, :, :], t.view(-1)[7:19], torch.zeros(3, 1, 2).transpose(0, 1), torch.zeros(())):
        assert mixerops._dense(d)
    for d in (t[:, ::2], t[:, :5], t[:, :, :1], t[:1].expand(4, 6, 5), t.view(-1)[::2]):
        assert not mixerops._dense(d)


def test_the_binding_refuses_before_the_device(monkeypatch):
    monkeypatch.setattr(mixerops._c, "_on_cuda", lambda t: True)
    x = torch.zeros(6, 64)
    assert mixerops._row_stride(x, "x") == 64 and mixerops._row_stride(x[::2], "x") == 128
    assert mixerops._row_stride(x[:, 3:9], "x") == 64 and mixerops._row_stride(x[0], "x") == 64
    assert mixerops._row_stride(x.view(2, 3, 64)[:, :1], "x") == 192
    for bad in (x.t(), x[:1].expand(6, 64), x.view(2, 3, 64)[:, :2], x[:, :0], x.view(6, 8, 8)[:, :, :1].transpose(1, 2)):
        with pytest.raises(ValueError):
            mixerops._row_stride(bad, "x")
    with pytest.raises(ValueError):
        mixerops._list([x, x[:, ::2]])
