"""CPU runs of the unchanged spec_forward kernel source (tests/emu) against the float64
references: bad lengths, pages and indices, masks, ragged and empty rows, strides."""
import numpy as np
import pytest
import torch

import forward_cases as fc
from oracle import forward as ref


@pytest.fixture(scope="module")
def run():
    r = fc.Emu(fc.build_emu())
    return r


def test_e4m3_reference_and_emulation(run):
    """Every code's value against torch's, and the rounding of a sweep that holds all ties."""
    codes = np.arange(256, dtype=np.uint8)
    v = ref.e4m3_value(codes)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(v), np.isnan(t)) and np.array_equal(v[~np.isnan(v)], t[~np.isnan(t)])
    pos = np.sort(v[:127])
    x = np.concatenate([pos, (pos[1:] + pos[:-1]) / 2, np.nextafter(pos, 1e9), [500.0, 1e30, np.inf, np.nan, 2.0 ** -20]])
    x = np.concatenate([x, -x]).astype(np.float32)
    clamped = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_code(x.astype(np.float64)) & 127, clamped & 127)
    run.L.spec_forward_emu_e4m3.argtypes = [fc.ctypes.c_float]
    fine = ~np.isinf(x) & (np.abs(x) <= 448) | np.isnan(x)
    assert [run.L.spec_forward_emu_e4m3(float(y)) & 127 for y in x[fine]] == list(clamped[fine] & 127)


APPENDS = [
    dict(), dict(R=1), dict(layout="token", D=128), dict(cache="e4m3"), dict(cache="e4m3", dtype="f16", D=256, page=8),
    dict(B=3, R=20, page=1, lens=[0, 1, 30]), dict(B=3, R=5, draft_len=[0, 4, 2]),
    dict(B=4, R=5, draft_len=[-1, 5, 2 ** 31 - 1, 4]), dict(cache="e4m3", scale=3000.0),
]


@pytest.mark.parametrize("kw", APPENDS, ids=str)
def test_append(run, kw):
    fc.check_append(run, fc.make_append(1, **kw))


def bad_rows(a, page):
    """Lengths and pages out of range: (what is wrong with row b, the changed inputs)."""
    table, kv = a["page_table"].clone(), a["kv_len"].clone()
    width = table.shape[1]
    kv[1] = -1
    kv[2] = width * page                                   # no room for one token
    kv[3] = 2 ** 31 - 1
    table[4, 0] = 2 ** 31 - 1
    table[5, 0] = -7
    return dict(a, page_table=table, kv_len=kv)


def test_append_bad_rows(run):
    a = fc.make_append(2, B=7, lens=[3, 9, 8, 4, 2, 6, 12])
    fc.check_append(run, bad_rows(a, 16))


ATTENTIONS = [
    dict(), dict(lens=[0, 1]), dict(R=4, lens=[0, 60]), dict(R=4, G=5, Hkv=1, D=128, lens=[31, 200]),
    dict(layout="token", D=128, page=8), dict(dtype="f16", D=256, G=1), dict(cache="e4m3"),
    dict(cache="e4m3", dtype="f16", D=128, page=32), dict(cache="e4m3", D=256, R=3),
    dict(R=3, window=7, lens=[0, 100]), dict(R=2, window=1, lens=[50, 63]), dict(R=3, softcap=5.0, sharp=6.0),
    dict(R=2, slopes=True, lens=[90, 17]), dict(R=3, softcap=30.0, window=20, slopes=True, lens=[300, 10]),
    dict(R=5, draft_len=[0, 4], lens=[40, 12]), dict(B=3, R=5, draft_len=[-1, 2, 5], lens=[40, 12, 7]),
    dict(R=9, G=8, Hkv=1, lens=[100, 3]), dict(page=1, lens=[40, 9]), dict(page=1024, lens=[700, 5]),
    dict(B=5, R=2, lens=[0, 500, 3, 129, 64]), dict(B=70, lens=[(11 * b) % 150 for b in range(70)], G=1, Hkv=1),
    dict(R=7, G=5, Hkv=1, lens=[200, 33], D=128), dict(R=6, G=8, Hkv=1, cache="e4m3", lens=[100, 64], D=128),
    dict(R=8, G=8, Hkv=1, cache="e4m3", lens=[70, 0]), dict(R=5, G=7, Hkv=1, window=20, lens=[90, 5], page=8),
    dict(R=9, G=4, Hkv=1, D=256, lens=[40, 65]), dict(R=25, G=8, Hkv=1, lens=[30, 2]), dict(scale=0.0), dict(scale=-0.3), dict(strided=False),
]


@pytest.mark.parametrize("kw", ATTENTIONS, ids=str)
def test_attention(run, kw):
    fc.check_attention(run, fc.make_attention(3, **kw))


@pytest.mark.parametrize("softcap", [255.0, 256.0, 5000.0, 1e8, 1e30, 3e38])
def test_attention_large_softcap(run, softcap):
    """A cap far above the scores leaves them as they are."""
    fc.check_attention(run, fc.make_attention(15, R=2, softcap=softcap, sharp=10.0, lens=[90, 17]))


def test_attention_softcap_between_series_and_exponential(run):
    """Scores on both sides of a quarter of the cap."""
    a = fc.make_attention(16, R=2, G=4, softcap=300.0, sharp=1.0, lens=[120, 40])
    fc.check_attention(run, dict(a, q=a["q"] * torch.tensor([4.0, 20.0, 60.0, 300.0] * 2)[:, None].to(a["q"].dtype)))


@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_attention_float16_sums_of_small_weights(run, cache):
    """Many weights of about 2^-24 of the largest, whose value is zero."""
    a = fc.make_attention(17, B=1, Hkv=1, dtype="f16", cache=cache, lens=[1500])
    ones = torch.ones_like(a["k_cache"].float())
    first = int(a["page_table"][0, 0])
    k, v = ones * 0.0, ones * 200.0
    k[..., 0] = -16.0
    k[first, :, 0], v[first, :, 0] = 0.0, 0.0
    q = torch.zeros_like(a["q"])
    q[..., 0] = torch.tensor([1.0, 1.0166])
    if cache == "e4m3":
        a.update(k_scale=torch.ones(1), v_scale=torch.ones(1))
    fc.check_attention(run, dict(a, q=q, k_cache=k.to(a["k_cache"].dtype), v_cache=v.to(a["v_cache"].dtype), scale=1.0))


def test_attention_bad_rows(run):
    a = fc.make_attention(4, B=7, R=2, lens=[30, 9, 8, 4, 20, 40, 12])
    fc.check_attention(run, bad_rows(a, 16))


def unmap(a, page, window):
    """The pages before every window out of the table."""
    table = a["page_table"].clone()
    for b, kv in enumerate(a["kv_len"].tolist()):
        first = max(0, kv + 1 - window)
        table[b, :first // page] = -1
    return dict(a, page_table=table)


@pytest.mark.parametrize("page", [8, 16, 64])
def test_attention_window_over_unmapped_pages(run, page):
    a = fc.make_attention(5, B=3, R=3, page=page, lens=[200, 70, 5], window=33)
    fc.check_attention(run, unmap(a, page, 33))


def poison(a, R, what, cache=None):
    """NaN or infinities in every cache place that no token in use sees."""
    k, v = a["k_cache"].clone(), a["v_cache"].clone()
    ps = k.shape[2]
    live = torch.zeros(k.shape[0], ps, dtype=torch.bool)
    for b, kv in enumerate(a["kv_len"].tolist()):
        n = R if a.get("draft_len") is None else int(a["draft_len"][b]) + 1
        lo = max(0, kv + 1 - a["window"]) if a.get("window") else 0
        for t in range(lo, kv + n):
            live[a["page_table"][b, t // ps], t % ps] = True
    dead = ~live[:, None, :, None].expand(k.shape)
    if k.dtype == torch.float8_e4m3fn:
        k, v = (torch.where(dead, torch.tensor(0x7f, dtype=torch.uint8), t.view(torch.uint8)).view(k.dtype)
                for t in (k, v))
    else:
        k, v = (t.masked_fill(dead, what) for t in (k, v))
    return dict(a, k_cache=k, v_cache=v)


@pytest.mark.parametrize("kw", [dict(), dict(window=21), dict(cache="e4m3"), dict(draft_len=[1, 0, 3]), dict(G=10),
                                dict(G=10, window=21), dict(G=20, cache="e4m3", draft_len=[3, 2, 0])], ids=str)
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_attention_ignores_places_nobody_sees(run, kw, what):
    a = fc.make_attention(6, B=3, R=4, lens=[77, 0, 30], **kw)
    fc.check_attention(run, poison(a, 4, what))


@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("which", ["k_cache", "v_cache"])
@pytest.mark.parametrize("window", [0, 3])
@pytest.mark.parametrize("G", [2, 9])
def test_attention_bad_value_reaches_only_who_sees_it(run, what, which, window, G):
    """A non-finite key or value of the last draft: the earlier tokens do not see it; one
    just before the first token's window end: the later ones do not."""
    a = fc.make_attention(7, B=2, R=4, lens=[45, 2], window=window, G=G)
    for t, b in ((48, 0), (5, 1), (44, 0)):
        x = a[which].clone()
        ps = x.shape[2]
        x[a["page_table"][b, t // ps], :, t % ps, 5] = what
        a2 = dict(a, **{which: x})
        fc.check_attention(run, a2, f"position {t}")


def test_attention_shared_pages(run):
    """Two sequences that share their first pages (a common prefix), and one page twice in a
    sequence."""
    a = fc.make_attention(16, B=3, R=2, lens=[100, 90, 70])
    table = a["page_table"].clone()
    table[1, :4] = table[0, :4]
    table[2, 2] = table[2, 0]
    fc.check_attention(run, dict(a, page_table=table))


def test_attention_extreme_scores(run):
    """Scores far apart, huge and tiny: the running maximum moves by large steps."""
    a = fc.make_attention(8, B=2, R=2, lens=[300, 40], sharp=60.0, dtype="bf16")
    fc.check_attention(run, a)
    q = a["q"].clone()
    q[0] *= 1e30
    fc.check_attention(run, dict(a, q=q.contiguous()))


ADJUSTS = [
    dict(), dict(k=0), dict(rows="draft"), dict(dtype="bf16"), dict(dtype="bf16", out="f32"), dict(V=1001),
    dict(V=1001, dtype="bf16"), dict(V=1003, dtype="bf16", out="f32"), dict(V=7, H=3, bias=0), dict(V=1, H=2, bias=1),
    dict(V=9000, H=300, bias=40, dtype="bf16"), dict(H=0), dict(H=0, parts=()), dict(H=0, parts=(), bias=0),
    dict(masks=False), dict(parts=("repetition",)), dict(parts=("frequency",)), dict(parts=("presence",)),
    dict(B=3, draft_len=[0, 3, 1]), dict(B=3, rows="draft", draft_len=[0, 3, 1]), dict(B=3, draft_len=[-1, 4, 2]),
    dict(k=9, V=40, H=200), dict(bias=400, V=300), dict(H=1, V=50), dict(B=3, V=4097, H=64),
]


@pytest.mark.parametrize("kw", ADJUSTS, ids=str)
def test_adjust(run, kw):
    fc.check_adjust(run, fc.make_adjust(9, **kw))


@pytest.mark.parametrize("kw", [dict(), dict(masks=False), dict(dtype="bf16", V=1001), dict(B=3, draft_len=[0, 3, -1])],
                         ids=str)
def test_adjust_in_place(run, kw):
    a = fc.make_adjust(10, **kw)
    want = run.adjust(**dict(a, out=a["logits"].clone()))  # (itself checked by test_adjust)
    x = a["logits"].clone()
    got = run.adjust(**dict(a, logits=x, out=x))
    assert np.array_equal(fc.bits(got), fc.bits(want))


def spoiled(a, H, nrows):
    """Bad data of every kind, one per batch row (of 12)."""
    a = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in a.items()}
    a["hist_len"][1] = -1
    a["hist_len"][2] = H + 1
    a["hist_len"][3] = 2 ** 31 - 1
    a["prompt_len"][4] = a["hist_len"][4] + 1
    a["prompt_len"][5] = -1
    a["repetition"][6] = 0.0
    a["repetition"][7] = float("nan")
    a["frequency"][8] = float("inf")
    a["presence"][9] = float("nan")
    a["admit_row"][10, 0] = -2
    a["admit_row"][11, 1] = nrows
    a["history"][0, 0] = -5
    a["history"][0, 1] = 2 ** 31 - 1
    a["tokens"][0, 0] = -1
    a["tokens"][10, 1] = 10 ** 6
    a["bias_tokens"][0, 0] = 2 ** 31 - 1
    a["logits"][0, 0, 3:9] = float("nan")
    a["logits"][0, 1, 3:9] = float("-inf")
    a["logits"][0, 2, 3:9] = float("inf")
    return a


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_adjust_bad_rows(run, dtype):
    a = fc.make_adjust(11, B=12, V=300, dtype=dtype)
    fc.check_adjust(run, spoiled(a, 40, a["admit"].shape[0]))


def test_adjust_misaligned_pointers(run):
    """Tensors that start at an element, not at 16 bytes."""
    a = fc.make_adjust(12, V=515)
    x = torch.empty(a["logits"].numel() + 1)[1:].view(a["logits"].shape)
    x.copy_(a["logits"])
    fc.check_adjust(run, dict(a, logits=x))
