"""Softmax attention without a GPU: what the calls refuse, on the host, before anything is launched."""
import ctypes
import warnings

import pytest
import torch

import gated_delta_rule_86_b200 as kda
from gated_delta_rule_86_b200 import _lib
from gated_delta_rule_86_b200.attention import _native

E, U, OK = _lib.KDA_ERR_INVALID_ARG, _lib.KDA_ERR_UNSUPPORTED, _lib.KDA_OK
F = 1 << 20            # aligned, never dereferenced: every call below is rejected first
ODD = F + 8
B16, F32 = _lib.KDA_BF16, _lib.KDA_F32


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_86_b200 import build
    build.build_library()
    build.build_binding()
    return _lib.load()


def fwd(lib, q=F, k=F, v=F, qs=0, ks=0, vs=0, cu=None, cuk=None, n=0, B=1, Tq=8, Tk=8, Hq=4, Hkv=2, d=64, scale=0.1,
        dt=B16, out=F, rest=None, lse=None):
    return lib.kda_attn_fwd(q, k, v, qs, ks, vs, cu, cuk, n, B, Tq, Tk, Hq, Hkv, d, 1, scale, dt, out, rest, lse, None)


def bwd(lib, Tq=8, Tk=8, out=F, rest=None, lse=F, g=F, dq=F, dk=F, dv=F, ws=F, size=1 << 20, **kw):
    a = dict(Hq=4, Hkv=2, d=64, scale=0.1, dt=B16) | kw
    return lib.kda_attn_bwd(F, F, F, 0, 0, 0, None, None, 0, 1, Tq, Tk, a["Hq"], a["Hkv"], a["d"], 1, a["scale"], a["dt"],
                            out, rest, lse, g, dq, dk, dv, ws, size, None)


def append(lib, q=F, k=F, v=F, qs=0, ks=0, vs=0, freq=F, rot=64, cu=None, n=0, B=1, T=1, Hq=4, Hkv=2, d=64, dt=B16,
           lens=F, table=F, row=0, width=4, kc=F, vc=F, kp=0, vp=0, pages=8, size=16, qo=F, ko=None):
    return lib.kda_kv_append(q, k, v, qs, ks, vs, freq, rot, 0, cu, n, B, T, Hq, Hkv, d, dt, lens, table, row, width, kc,
                             vc, kp, vp, pages, size, qo, ko, None)


def decode(lib, q=F, qs=0, kc=F, vc=F, kp=0, vp=0, pages=8, size=16, table=F, row=0, width=400, lens=F, B=1, Hq=4, Hkv=2,
           d=64, scale=0.1, dt=B16, out=F, lse=None, ws=F, ws_bytes=1 << 30):
    return lib.kda_attn_decode_step(q, qs, kc, vc, kp, vp, pages, size, table, row, width, lens, B, Hq, Hkv, d, scale, dt,
                                    out, lse, ws, ws_bytes, None)


BAD_HEADS = [(dict(Hq=3), E), (dict(Hkv=0), E), (dict(d=0), E), (dict(dt=9), E), (dict(d=96), U), (dict(d=256), U)]


@pytest.mark.parametrize("kw,want", BAD_HEADS + [
    (dict(q=None), E), (dict(k=None), E), (dict(out=None), E), (dict(v=ODD), E), (dict(B=0), E), (dict(Tq=-1), E),
    (dict(scale=0.0), E), (dict(scale=-1.0), E), (dict(scale=float("nan")), E), (dict(scale=float("inf")), E),
    (dict(qs=100), E), (dict(qs=260), E), (dict(ks=129), E), (dict(cuk=F), E), (dict(cu=F, n=0), E),
    (dict(cu=F, n=2, B=2), E), (dict(cu=F, n=2, Tk=9), E), (dict(cu=F + 2, n=2), E), (dict(lse=F + 2), E), (dict(rest=ODD), E), (dict(rest=F, dt=F32), E),
    (dict(B=1 << 20, Tq=1 << 12, Tk=1 << 12), U)])
def test_forward_refuses(lib, kw, want):
    assert fwd(lib, **kw) == want


@pytest.mark.parametrize("kw,want", BAD_HEADS + [
    (dict(out=None), E), (dict(lse=None), E), (dict(g=None), E), (dict(dq=None), E), (dict(dk=None), E), (dict(dv=None), E),
    (dict(ws=None), E), (dict(size=8 * 4 * 4 - 1), E), (dict(dq=ODD), E), (dict(g=ODD), E), (dict(rest=ODD), E), (dict(rest=F, dt=F32), E), (dict(scale=0.0), E)])
def test_gradient_refuses(lib, kw, want):
    assert bwd(lib, **kw) == want


def test_gradient_workspace(lib):
    n = ctypes.c_size_t(7)
    assert lib.kda_attn_bwd_workspace_size(2, 100, 4, ctypes.byref(n)) == OK and n.value == 2 * 100 * 4 * 4
    assert lib.kda_attn_bwd_workspace_size(0, 100, 4, ctypes.byref(n)) == E
    assert lib.kda_attn_bwd_workspace_size(1, 100, 4, None) == E


BAD_CACHE = [(dict(kc=None), E), (dict(vc=ODD), E), (dict(table=None), E), (dict(table=F + 2), E), (dict(pages=0), E),
             (dict(size=0), E), (dict(width=0), E), (dict(width=4, row=3), E), (dict(kp=2 * 16 * 64 - 8), E),
             (dict(vp=2 * 16 * 64 + 4), E), (dict(size=24), U), (dict(size=1 << 17), U)]


@pytest.mark.parametrize("kw,want", BAD_HEADS + BAD_CACHE + [
    (dict(k=None), E), (dict(v=None), E), (dict(q=None), E), (dict(qo=None), E), (dict(lens=None), E), (dict(B=0), E),
    (dict(T=-1), E), (dict(freq=None), E), (dict(rot=-2), E), (dict(rot=66), E), (dict(rot=80), E), (dict(rot=15), E),
    (dict(rot=24), U), (dict(ko=ODD), E), (dict(cu=F, n=0), E), (dict(cu=F, n=2, B=2), E), (dict(ks=129), E),
    (dict(qs=264, qo=F), E)])
def test_append_refuses(lib, kw, want):
    assert append(lib, **kw) == want


@pytest.mark.parametrize("kw,want", BAD_HEADS + BAD_CACHE + [
    (dict(q=None), E), (dict(out=None), E), (dict(lens=None), E), (dict(lens=F + 1), E), (dict(B=0), E), (dict(ws=None), E),
    (dict(ws_bytes=8), E), (dict(ws=ODD), E), (dict(scale=0.0), E), (dict(qs=257), E), (dict(lse=F + 1), E),
    (dict(width=1 << 28, row=0), U)])
def test_decode_refuses(lib, kw, want):
    assert decode(lib, **kw) == want


def test_decode_workspace(lib):
    n = ctypes.c_size_t(0)
    assert lib.kda_attn_decode_workspace_size(4, 8, 2, 128, 1 << 20, B16, ctypes.byref(n)) == OK and n.value > 0
    assert lib.kda_attn_decode_workspace_size(4, 8, 2, 96, 1 << 20, B16, ctypes.byref(n)) == U and n.value == 0
    assert lib.kda_attn_decode_workspace_size(4, 8, 3, 128, 1 << 20, B16, ctypes.byref(n)) == E
    assert lib.kda_attn_decode_workspace_size(4, 8, 2, 128, 0, B16, ctypes.byref(n)) == E


def test_empty_calls_launch_nothing(lib):
    assert append(lib, T=0, k=None, v=None, q=None, qo=None) == OK
    assert fwd(lib, Tq=0, q=None, out=None) == OK


def test_status_name(lib):
    assert lib.kda_status_string(5).decode() == "KDA_ERR_BAD_PAGE"


def test_binding_refuses(lib):
    x = torch.zeros(1, 4, 2, 64)
    i = torch.zeros(1, dtype=torch.int32)
    t = torch.zeros(1, 4, dtype=torch.int32)
    c = torch.zeros(4, 2, 16, 64)
    for call in (lambda: kda.kda_attn_fwd(x, x, x), lambda: kda.kda_attn(x, x, x),              # not on a GPU
                 lambda: kda.kda_kv_append(x, x, c, c, t, i),
                 lambda: kda.kda_attn_decode_step(x[:, 0], c, c, t, i),
                 lambda: kda.kda_attn_fwd(x[0], x, x), lambda: kda.kda_attn_fwd(x, x[:, :3], x),
                 lambda: kda.kda_attn_fwd(x[:, :, :1], x, x),                                    # 1 head over 2
                 lambda: kda.kda_attn_fwd(x, x, x, cu_seqlens_k=i),
                 lambda: kda.kda_attn_fwd(x, x[:, :3], x[:, :3], cu_seqlens=torch.tensor([0, 4], dtype=torch.int32)),
                 lambda: kda.kda_kv_append(x, x, c[:, :1], c[:, :1], t, i),
                 lambda: kda.kda_kv_append(x, x, c.transpose(1, 2), c.transpose(1, 2), t, i),
                 lambda: kda.kda_kv_append(x, x, c, c, t[:0], i),
                 lambda: kda.kda_kv_append(x, x, c, c, t, i[:0]),
                 lambda: kda.kda_attn_decode_step(x[:, 0], c[..., :32], c[..., :32], t, i),
                 lambda: kda.kda_attn_decode_step(x, c, c, t, i)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: kda.kda_attn_fwd(x.half(), x.half(), x.half()), lambda: kda.kda_attn_fwd(x, x.bfloat16(), x),
                 lambda: kda.kda_attn_fwd(x, x, x, cu_seqlens=torch.tensor([0, 4])),
                 lambda: kda.kda_attn_decode_step(x[:, 0], c, c, t, i.long()),
                 lambda: kda.kda_kv_append(x, x, c.bfloat16(), c.bfloat16(), t, i)):
        with pytest.raises(TypeError):
            call()


def test_token_strides(lib):
    """Which layouts are read in place, and with which distance between tokens."""
    _tokens = _native().tokens
    x = torch.zeros(3, 5, 8, 64)
    assert _tokens(x)[1] == 512 and _tokens(x)[0].data_ptr() == x.data_ptr()
    part = x[:, :, 2:4]
    t, step = _tokens(part)
    assert t.data_ptr() == part.data_ptr() and step == 512
    one = x[:, 1:2, :2]   # one token per row: rows are the tokens
    t, step = _tokens(one)
    assert t.data_ptr() == one.data_ptr() and step == 5 * 512
    for odd in (x[:, :3], x[:, ::2], x.transpose(1, 2), x[..., ::2], x[:, :, ::2], x[:1].expand(3, -1, -1, -1)):
        t, step = _tokens(odd)
        assert t.is_contiguous() and step == t.shape[2] * t.shape[3] and torch.equal(t, odd)
    shifted = torch.zeros(3 * 5 * 8 * 64 + 1)[1:].view(3, 5, 8, 64)
    if shifted.data_ptr() % 16:
        assert _tokens(shifted)[0].data_ptr() % 16 == 0


def test_missing_binding_fails_loudly(monkeypatch):
    import gated_delta_rule_86_b200.attention as attention

    def gone(*a):
        raise ImportError("no such module")

    monkeypatch.setattr(attention, "_module", None)
    monkeypatch.setattr(attention.importlib, "import_module", gone)
    with pytest.raises(ImportError, match="build_binding"):
        kda.kda_attn_fwd(None, None, None)


def test_status_becomes_kda_error(lib):
    """The native module raises the package's own error type."""
    err = kda.KdaError(2, "kda_attn_fwd")
    assert err.status == 2 and "KDA_ERR_UNSUPPORTED" in str(err) and isinstance(err, RuntimeError)


def test_binding_refuses_caches_whose_pages_overlap(lib):
    """One page shown several times (a distance of 0, which means dense to the library), and pages that overlap in part."""
    x = torch.zeros(1, 1, 2, 64)
    i = torch.zeros(1, dtype=torch.int32)
    t = torch.zeros(1, 4, dtype=torch.int32)
    c = torch.zeros(4, 2, 16, 64)
    for bad in (c[:1].expand(4, -1, -1, -1), torch.zeros(8 * 2 * 16 * 64).as_strided((4, 2, 16, 64), (1024, 1024, 64, 1))):
        for caches in ((bad, c), (c, bad)):
            for call in (lambda: kda.kda_kv_append(x, x, *caches, t, i), lambda: kda.kda_attn_decode_step(x[:, 0], *caches, t, i)):
                with pytest.raises(ValueError, match="overlap"):
                    call()


def test_forward_mode_is_refused(lib):
    """An input with a tangent: no derivative of zero without a word (found before the device is looked at)."""
    import torch.autograd.forward_ad as fwd_ad
    plain = torch.zeros(1, 4, 2, 64)
    with fwd_ad.dual_level():
        dual = fwd_ad.make_dual(plain, torch.ones_like(plain))
        for i in range(3):
            args = [plain] * 3
            args[i] = dual
            for wants in (False, True):
                args[(i + 1) % 3] = plain.clone().requires_grad_(wants)
                with pytest.raises(NotImplementedError, match="forward-mode"):
                    kda.kda_attn(*args)


def test_append_says_that_it_has_no_gradient(lib):
    x, i, t, c = torch.zeros(1, 1, 2, 64), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(4, 2, 16, 64)
    leaf = x.clone().requires_grad_()
    for k, q in ((leaf, None), (x, leaf)):
        with pytest.warns(UserWarning, match="no gradient"), pytest.raises(ValueError, match="CUDA"):
            kda.kda_kv_append(k, x, c, c, t, i, q=q)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(UserWarning, match="no gradient"):
            kda.kda_kv_append(leaf, x, c, c, t, i)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            kda.kda_kv_append(leaf, x, c, c, t, i)
        with pytest.raises(ValueError, match="CUDA"):
            kda.kda_kv_append(x, x, c, c, t, i, q=x)


def test_binding_is_built_again_for_another_torch(lib, monkeypatch):
    from gated_delta_rule_86_b200 import build
    assert _native().built_for == f"built for torch {torch.__version__}"
    commands = []
    monkeypatch.setattr(build.subprocess, "check_call", commands.append)
    monkeypatch.setattr(build.os, "replace", lambda a, b: None)
    build.build_binding()
    assert not commands
    for other in (torch.__version__ + "1", torch.__version__[:-1], "1.0"):
        monkeypatch.setattr(torch, "__version__", other)
        build.build_binding()
        assert any(f"built for torch {other}" in str(x) for x in commands.pop())
