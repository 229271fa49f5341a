"""A seeded sweep of random shapes, types, masks, layouts and lengths through the
spec_forward operators, against the float64 references."""
import numpy as np
import pytest
import torch

import forward_cases as fc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def run():
    return fc.Gpu()


def log_int(rng, lo, hi):
    return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))


@pytest.mark.parametrize("seed", range(60))
def test_attention(run, seed):
    rng = np.random.default_rng(1000 + seed)
    D = int(rng.choice([64, 128, 256]))
    R = int(rng.choice([1, 1, 2, 4, 6, 9, 17]))
    Hkv, G = int(rng.integers(1, 5)), int(rng.integers(1, 17))
    most = 2.0e7 / (R * G * Hkv * D)                       # keeps the reference to a second
    B = min(log_int(rng, 1, 90), max(1, int(most / 8)))
    L = max(2, min(log_int(rng, 4, 6000), int(most / B)))
    kw = dict(B=B, R=R, Hkv=Hkv, G=G, D=D, page=int(2 ** rng.integers(0, 9)), lens=rng.integers(0, L, B).tolist(),
              dtype=str(rng.choice(["bf16", "f16"])), cache=str(rng.choice(["same", "same", "e4m3"])),
              layout=str(rng.choice(["head", "token"])), slopes=bool(rng.random() < 0.3), sharp=float(rng.choice([0.3, 2, 8])),
              strided=bool(rng.random() < 0.5))
    if rng.random() < 0.3:
        kw["softcap"] = float(rng.choice([1.0, 30.0, 50.0]))
    if rng.random() < 0.4:
        kw["window"] = log_int(rng, 1, 2 * L)
    if rng.random() < 0.3:
        kw["draft_len"] = rng.integers(0, R, B).tolist()
    print(seed, {n: v for n, v in kw.items() if n not in ("lens", "draft_len")}, flush=True)
    fc.check_attention(run, fc.make_attention(seed, **kw))


@pytest.mark.parametrize("seed", range(40))
def test_append(run, seed):
    rng = np.random.default_rng(2000 + seed)
    B, R = log_int(rng, 1, 60), log_int(rng, 1, 200)
    kw = dict(B=B, R=R, Hkv=int(rng.integers(1, 9)), D=int(rng.choice([64, 128, 256])), page=int(2 ** rng.integers(0, 9)),
              lens=rng.integers(0, 50, B).tolist(), dtype=str(rng.choice(["bf16", "f16"])),
              cache=str(rng.choice(["same", "e4m3"])), layout=str(rng.choice(["head", "token"])))
    if rng.random() < 0.4:
        kw["draft_len"] = rng.integers(-1, R + 1, B).tolist()
    print(seed, {n: v for n, v in kw.items() if n not in ("lens", "draft_len")}, flush=True)
    fc.check_append(run, fc.make_append(seed, **kw))


@pytest.mark.parametrize("seed", range(60))
def test_adjust(run, seed):
    rng = np.random.default_rng(3000 + seed)
    k = int(rng.integers(0, 9))
    V = log_int(rng, 1, 60000)
    B = max(1, min(log_int(rng, 1, 40), int(1.5e6 / (V * (k + 1)))))
    parts = tuple(p for p in ("repetition", "frequency", "presence") if rng.random() < 0.7)
    kw = dict(B=B, k=k, V=V, dtype=str(rng.choice(["f32", "bf16"])), rows="draft" if k and rng.random() < 0.3 else "target",
              H=0 if rng.random() < 0.2 else log_int(rng, 1, 9000), bias=int(rng.choice([0, 1, 7, 300])),
              masks=bool(rng.random() < 0.6), parts=parts, out=str(rng.choice(["same", "f32"])))
    if rng.random() < 0.3:
        kw["draft_len"] = rng.integers(0, k + 1, B).tolist()
    print(seed, {n: v for n, v in kw.items() if n != "draft_len"}, flush=True)
    a = fc.make_adjust(seed, **kw)
    fc.check_adjust(run, a)
    if a.get("draft_len") is None and a.get("out_dtype") in (None, a["logits"].dtype):
        x = a["logits"].clone()
        assert np.array_equal(fc.bits(run.adjust(**dict(a, logits=x, out=x))), fc.bits(run.adjust(**a)))
