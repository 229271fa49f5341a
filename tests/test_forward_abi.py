"""C-ABI checks of libspecforward.so that need no GPU: exports as declared, workspace sizes,
and the synchronous refusals (every case fails the host-side checks, so nothing is
enqueued and no pointer is followed)."""
import ctypes
import os
import re
import subprocess

import pytest

import token_verification_amd as tv
from token_verification_amd import forward

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x100000                                               # an aligned address, never followed
S = (ctypes.c_int64 * 3)
CACHE = S(2 * 16 * 64, 16 * 64, 64)


def test_exports_match_header():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "spec_forward.h")).read(), flags=re.S)
    declared = set(re.findall(r"\b(spec_\w+)\s*\(", src))
    out = subprocess.run(["nm", "-D", "--defined-only", forward.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert declared == {s for s in exported if s.startswith("spec_")}


def append(**kw):
    a = dict(k=P, ks=S(6 * 64, 2 * 64, 64), v=P, vs=S(6 * 64, 2 * 64, 64), dtype=1, B=2, R=3, Hkv=2, D=64, kc=P, kcs=CACHE,
             vc=P, vcs=CACHE, cdtype=1, pages=8, page=16, table=P, maxp=4, kv=P, dl=None, ksc=None, vsc=None)
    a.update(kw)
    return tv.forward_lib().spec_kv_append(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=0), -3), (dict(dtype=3), -3), (dict(cdtype=2), -3), (dict(cdtype=0), -3),
    (dict(B=0), -2), (dict(B=(1 << 21) + 1), -2), (dict(R=0), -2), (dict(R=(1 << 20) + 1), -2), (dict(Hkv=0), -2),
    (dict(Hkv=1025), -2), (dict(D=32), -2), (dict(D=96), -2), (dict(pages=0), -2), (dict(page=0), -2), (dict(page=24), -2),
    (dict(page=131072), -2), (dict(maxp=0), -2), (dict(maxp=1 << 27), -2),
    (dict(k=None), -1), (dict(v=None), -1), (dict(kc=None), -1), (dict(table=None), -1), (dict(kv=None), -1),
    (dict(cdtype=3), -1), (dict(ksc=P), -1), (dict(cdtype=3, ksc=P), -1),
    (dict(k=P + 8), -7), (dict(vc=P + 2), -7), (dict(ks=S(6 * 64, 2 * 64, 60)), -7), (dict(kcs=S(2048, 1024, -64)), -7),
    (dict(table=P + 2), -7), (dict(dl=P + 1), -7), (dict(kcs=S(1 << 30, 1 << 29, 1 << 28)), -2),
])
def test_append_refuses(kw, code):
    assert append(**kw) == code
    assert tv.forward_lib().spec_forward_last_error()


def attention(**kw):
    a = dict(q=P, qs=S(12 * 64, 4 * 64, 64), dtype=1, B=2, R=3, Hq=4, Hkv=2, D=64, kc=P, kcs=CACHE, vc=P, vcs=CACHE,
             cdtype=1, pages=8, page=16, table=P, maxp=4, kv=P, dl=None, scale=0.125, softcap=0.0, window=0, slopes=None,
             ksc=None, vsc=None, out=P, ws=P, nws=1 << 30)
    a.update(kw)
    return tv.forward_lib().spec_attention(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=0), -3), (dict(cdtype=2), -3), (dict(R=66), -2), (dict(R=0), -2), (dict(Hq=3), -2), (dict(Hq=1), -2),
    (dict(Hq=1026), -2), (dict(D=80), -2), (dict(q=None), -1), (dict(out=None), -1), (dict(cdtype=3), -1),
    (dict(scale=float("nan")), -9), (dict(scale=float("inf")), -9), (dict(softcap=-1.0), -9),
    (dict(softcap=float("inf")), -9), (dict(softcap=1e-38), -9), (dict(window=-1), -9),
    (dict(q=P + 8), -7), (dict(out=P + 8), -7), (dict(slopes=P + 2), -7), (dict(qs=S(768, 256, 4)), -7),
    (dict(ws=None), -6), (dict(nws=100), -6), (dict(ws=P + 128), -7),
])
def test_attention_refuses(kw, code):
    assert attention(**kw) == code
    assert tv.forward_lib().spec_forward_last_error()


def test_attention_workspace_sizes():
    f = tv.forward_lib().spec_attention_workspace_size
    assert f(0, 1, 4, 2, 64, 1, 16, 4) == f(2, 66, 4, 2, 64, 1, 16, 4) == f(2, 1, 3, 2, 64, 1, 16, 4) == 0
    assert f(2, 1, 4, 2, 96, 1, 16, 4) == f(2, 1, 4, 2, 64, 0, 16, 4) == f(2, 1, 4, 2, 64, 1, 0, 4) == 0
    for args in ((1, 1, 8, 8, 64, 1, 16, 4), (64, 6, 32, 8, 128, 1, 16, 300), (1, 5, 64, 8, 128, 3, 64, 4096),
                 (1, 65, 1024, 1, 256, 2, 16, 9), (1 << 21, 1, 1, 1, 64, 1, 1, 1)):
        n = f(*args)
        assert n > 0 and n % 256 == 0
    # a short cache needs no more ranges than it has units
    assert f(1, 1, 8, 8, 64, 1, 16, 4) < f(1, 1, 8, 8, 64, 1, 16, 4096)


def adjust(**kw):
    a = dict(logits=P, B=2, R=4, V=100, dtype=0, tokens=P, k=3, dl=None, hist=P, H=10, hl=P, pl=P, rep=P, freq=P, pres=P, bt=P,
             bv=P, nb=3, admit=P, na=8, ar=P, out=P + (1 << 20), odtype=0)
    a.update(kw)
    return tv.forward_lib().spec_adjust(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -3), (dict(odtype=1), -3), (dict(odtype=2), -3), (dict(dtype=1, odtype=2), -3),
    (dict(dtype=1, odtype=0, out=P), -3),
    (dict(B=0), -2), (dict(k=65, R=65), -2), (dict(R=2), -2), (dict(R=5), -2), (dict(R=0, k=0), -2), (dict(V=0), -2),
    (dict(V=(1 << 29) + 1), -2), (dict(H=-1), -2), (dict(H=1 << 29), -2), (dict(nb=-1), -2), (dict(nb=65537), -2),
    (dict(ar=None, na=7), -2), (dict(B=1 << 21, V=1 << 29), -2),
    (dict(logits=None), -1), (dict(out=None), -1), (dict(tokens=None), -1), (dict(hist=None), -1), (dict(hl=None), -1),
    (dict(bt=None), -1), (dict(bv=None), -1), (dict(admit=None), -1), (dict(na=0), -1), (dict(admit=None, na=0), -1),
    (dict(logits=P + 2), -7), (dict(out=P + 1), -7), (dict(hl=P + 2), -7), (dict(admit=P + 1), -7), (dict(tokens=P + 2), -7),
])
def test_adjust_refuses(kw, code):
    assert adjust(**kw) == code
    assert tv.forward_lib().spec_forward_last_error()


def test_binding_refuses_cpu_tensors_and_fails_without_library(monkeypatch, tmp_path):
    import torch
    with pytest.raises(ValueError):
        tv.spec_adjust(torch.zeros(1, 1, 8))
    with pytest.raises(ValueError):
        tv.spec_attention(torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16), None, None, None, None)
    with pytest.raises(ValueError):
        tv.spec_kv_append(None, None, None, None, None, None)
    monkeypatch.setattr(forward, "_lib", None)
    monkeypatch.setattr(forward, "LIB_PATH", str(tmp_path / "missing.so"))
    with pytest.raises(tv.SpecVerifyError):
        forward.forward_lib()
