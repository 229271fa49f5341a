"""Inputs, runners and comparisons shared by the CPU (emulated) and GPU tests of the
spec_forward operators. A runner is the public Python API on the device, or the same C
ABI of the library source compiled for the host (tests/emu), on host pointers."""
from __future__ import annotations

import ctypes
import math
import os
import subprocess

import numpy as np
import torch

from oracle import forward as ref

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
NAME = {v: k for k, v in DT.items()}
CODE = {"f32": 0, "bf16": 1, "f16": 2, "e4m3": 3}


# ------------------------------------------------------------------ runners

class Gpu:
    def __init__(self):
        import token_verification_amd as tv
        self.tv = tv

    def _up(self, kw):
        seen = {}

        def up(t):
            if not isinstance(t, torch.Tensor):
                return t
            if id(t) not in seen:
                seen[id(t)] = on_device(t)
            return seen[id(t)]
        return {n: up(t) for n, t in kw.items()}

    def append(self, **kw):
        d = self._up(kw)
        self.tv.spec_kv_append(**d)
        torch.cuda.synchronize()
        return d["k_cache"].cpu(), d["v_cache"].cpu()

    def attention(self, **kw):
        out = self.tv.spec_attention(**self._up(kw))
        torch.cuda.synchronize()
        return out.cpu()

    def adjust(self, **kw):
        out = self.tv.spec_adjust(**self._up(kw))
        torch.cuda.synchronize()
        return out.cpu()


def on_device(t):
    """t on the GPU with t's strides (storage order included)."""
    base = torch.as_strided(t, (t.untyped_storage().nbytes() // t.element_size(),), (1,), 0)
    return torch.as_strided(base.to("cuda:0"), t.shape, t.stride(), t.storage_offset())


class Emu:
    """The library source on the CPU."""

    def __init__(self, path):
        from token_verification_amd import forward
        L = ctypes.CDLL(path)
        src = forward.forward_lib()
        for n in ("spec_kv_append", "spec_attention", "spec_attention_workspace_size", "spec_adjust"):
            getattr(L, n).argtypes = getattr(src, n).argtypes
            getattr(L, n).restype = getattr(src, n).restype
        L.spec_forward_last_error.restype = ctypes.c_char_p
        self.L = L

    def _ok(self, rc):
        assert rc == 0, (rc, self.L.spec_forward_last_error())

    def append(self, k, v, k_cache, v_cache, page_table, kv_len, draft_len=None, k_scale=None, v_scale=None):
        B, R, H, D = k.shape
        self._ok(self.L.spec_kv_append(
            ptr(k), stride(k), ptr(v), stride(v), CODE[NAME[k.dtype]], B, R, H, D, ptr(k_cache), stride(k_cache),
            ptr(v_cache), stride(v_cache), CODE[NAME[k_cache.dtype]], k_cache.shape[0], k_cache.shape[2],
            ptr(page_table), page_table.shape[1], ptr(kv_len), ptr(draft_len), ptr(k_scale), ptr(v_scale), None))
        return k_cache, v_cache

    def attention(self, q, k_cache, v_cache, page_table, kv_len, draft_len=None, scale=None, softcap=0.0, window=0,
                  slopes=None, k_scale=None, v_scale=None):
        B, R, Hq, D = q.shape
        pages, Hkv, ps, _ = k_cache.shape
        code = CODE[NAME[k_cache.dtype]]
        need = self.L.spec_attention_workspace_size(B, R, Hq, Hkv, D, code, ps, page_table.shape[1])
        assert need > 0
        ws = np.frombuffer(os.urandom(1 << 16) * (need // (1 << 16) + 2), np.uint8).copy()
        at = ws.ctypes.data + (-ws.ctypes.data) % 256
        out = aligned_empty((B, R, Hq, D), q.dtype)
        self._ok(self.L.spec_attention(
            ptr(q), stride(q), CODE[NAME[q.dtype]], B, R, Hq, Hkv, D, ptr(k_cache), stride(k_cache), ptr(v_cache),
            stride(v_cache), code, pages, ps, ptr(page_table), page_table.shape[1], ptr(kv_len), ptr(draft_len),
            1.0 / math.sqrt(D) if scale is None else scale, softcap, window, ptr(slopes), ptr(k_scale), ptr(v_scale),
            ptr(out), at, need, None))
        return out

    def adjust(self, logits, tokens=None, history=None, hist_len=None, prompt_len=None, repetition=None,
               frequency=None, presence=None, bias_tokens=None, bias_values=None, admit=None, admit_row=None,
               draft_len=None, out=None, out_dtype=None):
        B, R, V = logits.shape
        if out is None:
            out = aligned_empty((B, R, V), out_dtype or logits.dtype)
        self._ok(self.L.spec_adjust(
            ptr(logits), B, R, V, CODE[NAME[logits.dtype]], ptr(tokens), 0 if tokens is None else tokens.shape[1],
            ptr(draft_len), ptr(history), 0 if history is None else history.shape[1], ptr(hist_len), ptr(prompt_len),
            ptr(repetition), ptr(frequency), ptr(presence), ptr(bias_tokens), ptr(bias_values),
            0 if bias_tokens is None else bias_tokens.shape[1], ptr(admit), 0 if admit is None else admit.shape[0],
            ptr(admit_row), ptr(out), CODE[NAME[out.dtype]], None))
        return out


def ptr(t):
    return None if t is None else t.data_ptr()


def stride(t):
    return (ctypes.c_int64 * 3)(*t.stride()[:3])


def aligned_empty(shape, dtype):
    n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
    raw = torch.from_numpy(np.frombuffer(os.urandom(n + 64), np.uint8).copy())
    o = -raw.data_ptr() % 64
    return raw[o:o + n].view(dtype).view(shape)


def build_emu(name="libspecforward_emu.so", sanitize=False):
    out = os.path.join(HERE, "emu", name)
    cmd = ["/opt/rocm/llvm/bin/clang++", "-std=c++17", "-O1", "-g", "-mf16c", "-fPIC", "-shared",
           "-I", os.path.join(HERE, "emu"), "-I", os.path.join(ROOT, "include"), "-Wno-unknown-pragmas",
           "-Wno-pass-failed", "-Wno-psabi", "-o", out, os.path.join(HERE, "emu", "spec_forward_emu.cpp"), "-lpthread"]
    subprocess.run(cmd, check=True)
    return out


# ------------------------------------------------------------------ inputs

def values(t):
    """float64 values of a tensor (e4m3 by the reference's own table)."""
    if t is None:
        return None
    if t.dtype == torch.float8_e4m3fn:
        return ref.e4m3_value(t.contiguous().view(torch.uint8).numpy())
    return t.double().numpy()


def arr(t):
    return None if t is None else t.numpy()


def paged(rng, B, Hkv, D, page, lens, R, dtype, cache, layout, spare=2, fill=None):
    """Cache tensors [pages, Hkv, page, D], a shuffled page table (unmapped entries -1)
    that maps lens[b] + R positions, and the scales of an e4m3 cache."""
    n = [max(1, -(-(max(0, x) + R) // page)) for x in lens]
    pages, width = sum(n) + spare, max(n) + 1
    order = rng.permutation(pages)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :n[b]] = order[at:at + n[b]]
        at += n[b]
    shape = (pages, Hkv, page, D) if layout == "head" else (pages, page, Hkv, D)
    out = []
    for _ in range(2):
        x = torch.from_numpy(rng.normal(0, 1, shape).astype(np.float32)) if fill is None else torch.full(shape, fill)
        x = (x * 50).to(DT["e4m3"]) if cache == "e4m3" else x.to(DT[dtype])
        out.append(x if layout == "head" else x.transpose(1, 2))
    ks, vs = ((torch.from_numpy(rng.uniform(0.01, 0.03, Hkv).astype(np.float32)) for _ in range(2))
              if cache == "e4m3" else (None, None))
    return out[0], out[1], torch.from_numpy(table), ks, vs


def make_attention(seed, B=2, R=1, Hkv=2, G=2, D=64, page=16, lens=None, dtype="bf16", cache="same", layout="head",
                   slopes=False, draft_len=None, strided=True, sharp=2.0, **kw):
    rng = np.random.default_rng(seed)
    lens = [37] * B if lens is None else list(lens)
    kc, vc, table, ks, vs = paged(rng, B, Hkv, D, page, lens, R, dtype, cache, layout)
    Hq = Hkv * G
    wide = torch.from_numpy(rng.normal(0, sharp, (B, R, Hq + 2 * Hkv, D)).astype(np.float32)).to(DT[dtype])
    q = wide[:, :, Hkv:Hkv + Hq] if strided else wide[:, :, :Hq].contiguous()
    a = dict(q=q, k_cache=kc, v_cache=vc, page_table=table, kv_len=torch.tensor(lens, dtype=torch.int32),
             k_scale=ks, v_scale=vs, **kw)
    if slopes:
        a["slopes"] = torch.from_numpy(np.exp2(-8.0 * np.arange(1, Hq + 1) / Hq).astype(np.float32))
    if draft_len is not None:
        a["draft_len"] = torch.tensor(draft_len, dtype=torch.int32)
    return a


def attention_want(a):
    kw = {n: a[n] for n in ("scale", "softcap", "window") if n in a}
    return ref.attention_ref(values(a["q"]), values(a["k_cache"]), values(a["v_cache"]), arr(a["page_table"]),
                             arr(a["kv_len"]), dtype=NAME[a["q"].dtype], draft_len=arr(a.get("draft_len")),
                             slopes=values(a.get("slopes")), k_scale=values(a.get("k_scale")),
                             v_scale=values(a.get("v_scale")), **kw)


def near(got, want, tol, what=""):
    """got within tol of want element by element; NaN and infinities in the same places."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    inf = np.isinf(want)
    assert np.array_equal(inf, np.isinf(got)) and np.array_equal(got[inf], want[inf]), f"{what}: other infinities"
    fine = np.isfinite(want)
    with np.errstate(invalid="ignore"):
        far = np.abs(got - want)[fine] - np.broadcast_to(tol, want.shape)[fine]
    assert not (far > 0).any(), f"{what}: {int((far > 0).sum())} of {far.size} outside, by up to {far.max():.3g}"


def check_attention(run, a, what=""):
    want, tol = attention_want(a)
    near(run.attention(**a).double().numpy(), want, tol, what)


def make_append(seed, B=2, R=3, Hkv=2, D=64, page=16, lens=None, dtype="bf16", cache="same", layout="head",
                draft_len=None, scale=60.0):
    rng = np.random.default_rng(seed)
    lens = [5 + 11 * b for b in range(B)] if lens is None else list(lens)
    kc, vc, table, ks, vs = paged(rng, B, Hkv, D, page, lens, R, dtype, cache, layout)
    wide = torch.from_numpy(rng.normal(0, scale * 0.02, (B, R, 3 * Hkv, D)).astype(np.float32)).to(DT[dtype])
    a = dict(k=wide[:, :, Hkv:2 * Hkv], v=wide[:, :, 2 * Hkv:], k_cache=kc, v_cache=vc, page_table=table,
             kv_len=torch.tensor(lens, dtype=torch.int32), k_scale=ks, v_scale=vs)
    if draft_len is not None:
        a["draft_len"] = torch.tensor(draft_len, dtype=torch.int32)
    return a


def bits(t):
    t = t.contiguous()
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32).numpy()


def check_append(run, a, what=""):
    want = []
    for n in ("k", "v"):
        s = a[n + "_scale"]
        x = bits(a[n]) if s is None else values(a[n])
        want.append(ref.append_ref(x, bits(a[n + "_cache"]), arr(a["page_table"]), arr(a["kv_len"]),
                                   arr(a.get("draft_len")), None if s is None else s.numpy()))
    got = run.append(**a)
    for g, w, n in zip(got, want, "kv"):
        g = bits(g)
        if a["k_scale"] is not None:                       # both codes 0x7f and 0xff are NaN
            g, w = (np.where(x == 0xff, 0x7f, x) for x in (g, w))
        assert np.array_equal(g, w), f"{what}: {n}"


def make_adjust(seed, B=2, k=3, V=1000, dtype="f32", rows="target", H=40, bias=5, masks=True, out="same",
                draft_len=None, parts=("repetition", "frequency", "presence")):
    rng = np.random.default_rng(seed)
    R = k + 1 if rows == "target" else k
    a = dict(logits=aligned_empty((B, R, V), DT[dtype]).copy_(
        torch.from_numpy(rng.normal(0, 3, (B, R, V)).astype(np.float32))))
    tokens = rng.integers(0, V, (B, k)).astype(np.int32)
    if H:
        hist = (V * rng.uniform(0, 1, (B, H)) ** 3).astype(np.int32)
        n = rng.integers(H // 2, H + 1, B).astype(np.int32)
        a.update(history=torch.from_numpy(hist), hist_len=torch.from_numpy(n),
                 prompt_len=torch.from_numpy((n * rng.uniform(0, 1, B)).astype(np.int32)))
        for b in range(B):
            for j in range(k):
                if n[b] and rng.uniform() < 0.7:
                    tokens[b, j] = hist[b, rng.integers(0, n[b])]
        if k > 2:
            tokens[:, 2] = tokens[:, 0]                    # a draft that repeats a draft
    if k:
        a["tokens"] = torch.from_numpy(tokens)
    if "repetition" in parts:
        a["repetition"] = torch.from_numpy(rng.uniform(0.8, 1.4, B).astype(np.float32))
    if "frequency" in parts:
        a["frequency"] = torch.from_numpy(rng.uniform(-0.2, 0.6, B).astype(np.float32))
    if "presence" in parts:
        a["presence"] = torch.from_numpy(rng.uniform(-0.2, 0.6, B).astype(np.float32))
    if bias:
        bt = rng.integers(0, V, (B, bias)).astype(np.int32)
        if bias > 2:
            bt[:, bias // 2] = bt[:, 0]                    # a token that is biased twice
            bt[:, -1] = -1                                 # padding
        a.update(bias_tokens=torch.from_numpy(bt),
                 bias_values=torch.from_numpy(rng.normal(0, 4, (B, bias)).astype(np.float32)))
    if masks:
        W = (V + 31) // 32
        m = rng.integers(-2 ** 31, 2 ** 31, (B * R + 1, W)).astype(np.int32)
        m[0] = 0                                           # admits nothing
        row = rng.integers(-1, B * R + 1, (B, R)).astype(np.int32)
        a.update(admit=torch.from_numpy(m), admit_row=torch.from_numpy(row))
    if draft_len is not None:
        a["draft_len"] = torch.tensor(draft_len, dtype=torch.int32)
    if out == "f32":
        a["out_dtype"] = torch.float32
    return a


def check_adjust(run, a, what=""):
    k = a["tokens"].shape[1] if a.get("tokens") is not None else 0
    B, R, V = a["logits"].shape
    names = ("history", "hist_len", "prompt_len", "bias_tokens", "admit", "admit_row", "draft_len")
    floats = ("repetition", "frequency", "presence", "bias_values")
    kw = {n: arr(a.get(n)) for n in names} | {n: values(a.get(n)) for n in floats}
    dtype = a.get("out_dtype") or a["logits"].dtype
    given = dict(a)
    before = None
    if a.get("draft_len") is not None and a.get("out") is None:
        given["out"] = aligned_empty((B, R, V), dtype).copy_(torch.full((B, R, V), 7.0))
    if given.get("out") is not None:
        before = values(given["out"])
    want, tol = ref.adjust_ref(values(a["logits"]), np.zeros((B, 0), np.int32) if k == 0 else arr(a["tokens"]),
                               out_dtype=NAME[dtype], before=before, **kw)
    got = run.adjust(**given)
    assert got.dtype == dtype
    near(got.double().numpy(), want, tol, what)
