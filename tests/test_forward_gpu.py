"""The spec_forward operators on the GPU, through the public Python API: the cases of the
CPU run and larger ones against the float64 references, bad data, refusals, streams,
graphs, and a whole verify step through the cache, the attention, the adjustment,
spec_verify and spec_commit."""
import numpy as np
import pytest
import torch

import forward_cases as fc
import test_forward_emu as cpu
import token_verification_amd as tv
from oracle import forward as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def run():
    return fc.Gpu()


@pytest.fixture(autouse=True)
def announce(request):
    print(request.node.name, flush=True)


# ------------------------------------------------------------------ against the references

@pytest.mark.parametrize("kw", cpu.APPENDS + [
    dict(B=33, R=7, Hkv=12, D=128, lens=list(range(0, 330, 10))), dict(B=5, R=300, D=256, dtype="f16", page=64),
    dict(B=200, R=4, Hkv=8, D=128, cache="e4m3", lens=[5] * 200, layout="token"),
], ids=str)
def test_append(run, kw):
    fc.check_append(run, fc.make_append(1, **kw))


def test_append_bad_rows(run):
    fc.check_append(run, cpu.bad_rows(fc.make_append(2, B=7, lens=[3, 9, 8, 4, 2, 6, 12]), 16))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_append_e4m3_rounds_every_value(run, dtype):
    """All 65536 bit patterns of the type as keys, against the table."""
    x = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(fc.DT[dtype]).view(4, 64, 4, 64)
    a = fc.make_append(3, B=4, R=64, Hkv=4, D=64, lens=[0, 1, 2, 3], dtype=dtype, cache="e4m3")
    a.update(k=x, v=x.flip(1), k_scale=torch.ones(4), v_scale=torch.full((4,), 0.37))
    fc.check_append(run, a)


@pytest.mark.parametrize("kw", cpu.ATTENTIONS + [
    dict(B=1, Hkv=8, G=4, D=128, lens=[999]), dict(B=1, Hkv=1, G=1, lens=[5000]), dict(B=3, R=5, Hkv=2, G=8, D=128,
                                                                                       lens=[3000, 1, 700]),
    dict(B=40, R=2, Hkv=2, G=2, lens=[(b * 37) % 260 for b in range(40)]), dict(B=1, R=4, Hkv=1, G=3, D=256, lens=[4090]),
    dict(B=2, R=65, Hkv=1, G=2, lens=[100, 0]), dict(B=1, R=17, Hkv=1, G=16, D=128, lens=[513]),
    dict(B=2, R=4, Hkv=3, G=7, D=128, cache="e4m3", lens=[2048, 2047]), dict(B=300, lens=[(7 * b) % 40 for b in range(300)]),
    dict(B=2, R=3, Hkv=2, D=128, window=500, softcap=50.0, lens=[3001, 499], dtype="f16"),
    dict(B=1, Hkv=20, G=1, lens=[1500], slopes=True), dict(B=100, R=2, lens=[(97 * b) % 700 for b in range(100)]),
    dict(B=1, Hkv=20, G=1, lens=[3000]), dict(B=2, R=2, Hkv=8, lens=[6000, 20]),
    dict(B=1, R=5, Hkv=8, G=8, D=128, cache="e4m3", lens=[8000]), dict(B=3, Hkv=16, G=1, lens=[40, 7000, 0], window=6500),
    dict(B=600, Hkv=1, G=2, lens=[(131 * b) % 900 for b in range(600)]), dict(B=2, R=9, G=8, Hkv=2, D=128, lens=[2500, 60]),
    dict(B=2, R=6, G=7, Hkv=2, D=128, cache="e4m3", lens=[3000, 100]), dict(B=1, R=8, G=8, Hkv=1, D=256, lens=[1000]),
    dict(B=2, R=65, G=8, Hkv=1, D=128, lens=[700, 0]), dict(B=1, R=12, G=16, Hkv=1, D=128, lens=[3000], window=1000), dict(B=1, R=2, D=256, cache="e4m3", dtype="f16", lens=[1200], page=128),
], ids=str)
def test_attention(run, kw):
    fc.check_attention(run, fc.make_attention(3, **kw))


@pytest.mark.parametrize("softcap", [255.0, 256.0, 5000.0, 1e8, 1e30, 3e38])
def test_attention_large_softcap(run, softcap):
    cpu.test_attention_large_softcap(run, softcap)


def test_attention_softcap_between_series_and_exponential(run):
    cpu.test_attention_softcap_between_series_and_exponential(run)


@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_attention_float16_sums_of_small_weights(run, cache):
    cpu.test_attention_float16_sums_of_small_weights(run, cache)


def test_attention_bad_rows(run):
    fc.check_attention(run, cpu.bad_rows(fc.make_attention(4, B=7, R=2, lens=[30, 9, 8, 4, 20, 40, 12]), 16))


def test_attention_bad_page_in_a_long_row(run):
    """One bad page among many: the whole batch row is NaN, its neighbours are not."""
    a = fc.make_attention(13, B=3, R=2, lens=[2000, 2000, 2000])
    a["page_table"][1, 77] = a["k_cache"].shape[0]
    fc.check_attention(run, a)


@pytest.mark.parametrize("page", [8, 16, 64])
def test_attention_window_over_unmapped_pages(run, page):
    a = fc.make_attention(5, B=3, R=3, page=page, lens=[200, 70, 5], window=33)
    fc.check_attention(run, cpu.unmap(a, page, 33))


@pytest.mark.parametrize("kw", [dict(), dict(window=21), dict(cache="e4m3"), dict(draft_len=[1, 0, 3]), dict(G=10),
                                dict(G=10, window=21), dict(G=20, cache="e4m3", draft_len=[3, 2, 0])], ids=str)
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_attention_ignores_places_nobody_sees(run, kw, what):
    a = fc.make_attention(6, B=3, R=4, lens=[777, 0, 30], **kw)
    fc.check_attention(run, cpu.poison(a, 4, what))


@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("which", ["k_cache", "v_cache"])
@pytest.mark.parametrize("window", [0, 3])
@pytest.mark.parametrize("G", [2, 9])
def test_attention_bad_value_reaches_only_who_sees_it(run, what, which, window, G):
    cpu.test_attention_bad_value_reaches_only_who_sees_it(run, what, which, window, G)


def test_attention_shared_pages(run):
    cpu.test_attention_shared_pages(run)


def test_attention_extreme_scores(run):
    cpu.test_attention_extreme_scores(run)


def test_attention_offsets_past_32_bits(run):
    """Pages on both sides of 2^32 bytes (and of 2^31 elements) of one cache."""
    a = fc.make_attention(14, B=2, R=2, Hkv=2, D=128, page=16, lens=[100, 35])
    pages, Hkv, ps, D = a["k_cache"].shape
    want, tol = fc.attention_want(a)
    stride = (5 << 30) // 2 // pages // 64 * 64            # elements between pages: the cache spans about 5 GiB
    big = {}
    for n in ("k_cache", "v_cache"):
        store = torch.empty(stride * pages, dtype=torch.bfloat16, device=DEV)
        big[n] = torch.as_strided(store, (pages, Hkv, ps, D), (stride, ps * D, D, 1))
        big[n].copy_(a[n].to(DEV))
    d = {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in a.items()} | big
    fc.near(tv.spec_attention(**d).double().cpu().numpy(), want, tol)
    x = torch.randn((2, 2, Hkv, D), dtype=torch.bfloat16, device=DEV)
    tv.spec_kv_append(x, -x, d["k_cache"], d["v_cache"], d["page_table"], d["kv_len"])
    for b, kv in enumerate(a["kv_len"].tolist()):
        for i in range(2):
            page, slot = int(a["page_table"][b, (kv + i) // ps]), (kv + i) % ps
            assert torch.equal(big["k_cache"][page, :, slot], x[b, i])
            assert torch.equal(big["v_cache"][page, :, slot], -x[b, i])


def test_attention_is_reproducible(run):
    a = fc.make_attention(15, B=5, R=3, Hkv=2, G=4, D=128, lens=[4000, 1, 900, 77, 2500])
    d = {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in a.items()}
    first = tv.spec_attention(**d).clone()
    for _ in range(5):
        assert torch.equal(tv.spec_attention(**d).view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("kw", cpu.ADJUSTS + [
    dict(B=4, k=5, V=151936, dtype="bf16", H=2000, bias=16), dict(B=1, k=0, V=32000, H=512, masks=False, bias=0),
    dict(B=3, k=2, V=50257, H=5000, dtype="bf16", out="f32"), dict(B=1, k=64, V=700, H=100),
    dict(B=2, k=1, V=128256, H=70001, bias=300), dict(B=1, k=3, V=262144, H=0, parts=(), dtype="bf16"),
], ids=str)
def test_adjust(run, kw):
    fc.check_adjust(run, fc.make_adjust(9, **kw))


@pytest.mark.parametrize("kw", [dict(), dict(masks=False), dict(dtype="bf16", V=1001), dict(B=3, draft_len=[0, 3, -1])],
                         ids=str)
def test_adjust_in_place(run, kw):
    a = fc.make_adjust(10, **kw)
    want = run.adjust(**dict(a, out=a["logits"].clone()))
    x = a["logits"].clone()
    got = run.adjust(**dict(a, logits=x, out=x))
    assert np.array_equal(fc.bits(got), fc.bits(want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_adjust_bad_rows(run, dtype):
    a = fc.make_adjust(11, B=12, V=300, dtype=dtype)
    fc.check_adjust(run, cpu.spoiled(a, 40, a["admit"].shape[0]))


def test_adjust_misaligned_pointers(run):
    cpu.test_adjust_misaligned_pointers(run)


# ------------------------------------------------------------------ streams and graphs

def device_inputs(seed=20):
    a = fc.make_attention(seed, B=3, R=4, Hkv=2, G=4, D=128, lens=[1500, 3, 640], strided=False)
    d = {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in a.items()}
    j = fc.make_adjust(seed, B=3, k=3, V=5000, dtype="bf16")
    return d, {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in j.items()}


def step(d, j, k, v):
    cache = {n: d[n] for n in ("k_cache", "v_cache", "page_table", "kv_len")}
    tv.spec_kv_append(k, v, **cache)
    return tv.spec_attention(d["q"], **cache), tv.spec_adjust(**j)


def test_other_streams(run):
    """Every operator on two side streams at once, against the default stream."""
    (d, j), (d2, j2) = device_inputs(20), device_inputs(21)
    new = [torch.randn((3, 4, 2, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    want = [step(x, y, *new) for x, y in ((d, j), (d2, j2))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for s, (x, y) in zip(streams, ((d, j), (d2, j2))):
            with torch.cuda.stream(s):
                got.append(step(x, y, *new))
    torch.cuda.synchronize()
    for n, (o, l) in enumerate(got):
        assert torch.equal(o, want[n % 2][0]) and torch.equal(l, want[n % 2][1])


def test_two_graphs_at_once(run):
    """Two graphs captured on one stream, replayed on two at once with changed inputs, eager
    calls between the replays."""
    (d, j), (d2, j2) = device_inputs(22), device_inputs(23)
    new = [torch.randn((3, 4, 2, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(d, j, *new)
    torch.cuda.synchronize()
    for x, y in ((d, j), (d2, j2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(step(x, y, *new))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for n in range(4):
        for x in (d, d2):
            x["q"].copy_(torch.randn_like(x["q"]))
            x["kv_len"].copy_(torch.tensor([1500 - 300 * n, 3 + n, 640 - 100 * n], dtype=torch.int32))
        for y in (j, j2):
            y["logits"].copy_(torch.randn_like(y["logits"]))
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (x, y), (o, l) in zip(((d, j), (d2, j2)), outs):
            eo, el = step(x, y, *new)
            torch.cuda.synchronize()
            assert torch.equal(o, eo) and torch.equal(l, el), n


# ------------------------------------------------------------------ together

def one_page(x):
    """[tokens, heads, D] as a cache of one page."""
    return x.transpose(1, 0, 2)[None]


@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_verify_steps_through_the_cache(run, cache):
    """Three verify steps of a one-layer toy: its keys, values and queries come from the
    tokens, its logits from the attention. Every step appends, attends, adjusts,
    verifies and commits on the device; a float64 replay of the committed tokens must
    give the attention, and the committed tokens the history the next step sees."""
    rng = np.random.default_rng(30)
    B, k, Hkv, G, D, V, page, H = 4, 3, 2, 2, 64, 500, 8, 64
    R, Hq = k + 1, Hkv * G
    emb = {n: torch.from_numpy(rng.normal(0, 1, (V, h, D)).astype(np.float32)).bfloat16().to(DEV)
           for n, h in (("q", Hq), ("k", Hkv), ("v", Hkv))}
    head = torch.from_numpy(rng.normal(0, 1, (Hq * D, V)).astype(np.float32)).to(DEV)
    kc, vc, table, ks, vs = fc.paged(rng, B, Hkv, D, page, [60] * B, R, "bf16", cache, "head")
    kc, vc, table = kc.to(DEV), vc.to(DEV), table.to(DEV)
    ks, vs = (None, None) if ks is None else (ks.to(DEV), vs.to(DEV))
    kv_len = torch.zeros(B, dtype=torch.int32, device=DEV)
    committed = [[] for _ in range(B)]                     # tokens whose keys are in the cache
    pending = [int(t) for t in rng.integers(0, V, B)]
    rep = torch.full((B,), 1.3, device=DEV)
    pres = torch.full((B,), 0.7, device=DEV)
    for _ in range(3):
        drafts = torch.from_numpy(rng.integers(0, V, (B, k)).astype(np.int32)).to(DEV)
        toks = torch.cat([torch.tensor(pending, dtype=torch.int32, device=DEV)[:, None], drafts], 1).long()
        cached = dict(k_cache=kc, v_cache=vc, page_table=table, kv_len=kv_len, k_scale=ks, v_scale=vs)
        tv.spec_kv_append(emb["k"][toks], emb["v"][toks], **cached)
        o = tv.spec_attention(emb["q"][toks], **cached)
        got = o.double().cpu().numpy()
        for b in range(B):                                 # the replay, from the committed tokens alone
            seq = committed[b] + toks[b].tolist()
            kk, vv = (fc.values(emb[n][torch.tensor(seq, device=DEV)].cpu()) for n in "kv")
            if ks is not None:
                kk, vv = (ref.e4m3_value(ref.e4m3_code(x.astype(np.float32) / s.cpu().numpy()[:, None]))
                          for x, s in ((kk, ks), (vv, vs)))
            want, tol = ref.attention_ref(
                fc.values(emb["q"][toks[b:b + 1]].cpu()), one_page(kk), one_page(vv), np.zeros((1, 1), np.int64),
                np.array([len(committed[b])]), dtype="bf16", k_scale=fc.values(None if ks is None else ks.cpu()),
                v_scale=fc.values(None if vs is None else vs.cpu()))
            fc.near(got[b:b + 1], want, tol, f"row {b}")
        logits = (o.float().view(B, R, -1) @ head) * 0.3
        hist = torch.full((B, H), -1, dtype=torch.int32)
        for b in range(B):
            hist[b, :len(committed[b]) + 1] = torch.tensor(committed[b] + [pending[b]], dtype=torch.int32)
        n = torch.tensor([len(c) + 1 for c in committed], dtype=torch.int32, device=DEV)
        shaped = tv.spec_adjust(logits, drafts, history=hist.to(DEV), hist_len=n, repetition=rep, presence=pres)
        drafts[::2, 0] = shaped[::2, 0].argmax(1).to(torch.int32)   # half of the first drafts are right
        res = tv.spec_verify(shaped, None, drafts, None, 1.0, tv.GREEDY)
        tv.spec_commit(res.accepted_len, k, kv_len)
        acc, out = res.accepted_len.tolist(), res.out_tokens.tolist()
        assert all(a >= 1 for a in acc[::2])
        # the draft put in place above is not the one whose keys were cached: commit the pending token only
        for b in range(B):
            kv_len[b] = len(committed[b]) + 1
            committed[b].append(pending[b])
            pending[b] = out[b][0]
        torch.cuda.synchronize()


# ------------------------------------------------------------------ refusals

def dev(a):
    return {n: t.to(DEV) if isinstance(t, torch.Tensor) and n not in ("k_cache", "v_cache") else
            fc.on_device(t) if isinstance(t, torch.Tensor) else t for n, t in a.items()}


def refused(fn, a, **kw):
    with pytest.raises((ValueError, tv.SpecVerifyError)):
        fn(**dict(a, **kw))


def test_attention_refusals(run):
    a = dev(fc.make_attention(40, B=2, R=2, Hkv=2, G=2, D=64))
    f = tv.spec_attention
    refused(f, a, q=a["q"].float())
    refused(f, a, q=a["q"].half())                         # the cache is bfloat16
    refused(f, a, q=a["q"][..., :32])
    refused(f, a, q=a["q"][:, :, :3])                      # 3 heads over 2
    refused(f, a, q=a["q"].cpu())
    refused(f, a, q=a["q"].transpose(2, 3))
    refused(f, a, k_cache=a["k_cache"][:, :1])
    refused(f, a, k_cache=a["k_cache"].float())
    refused(f, a, k_cache=a["k_cache"][:, :, :12], v_cache=a["v_cache"][:, :, :12])      # 12 tokens a page
    refused(f, a, page_table=a["page_table"].long())
    refused(f, a, page_table=a["page_table"][:1])
    refused(f, a, kv_len=a["kv_len"].long())
    refused(f, a, kv_len=a["kv_len"][:1])
    refused(f, a, draft_len=a["kv_len"].float())
    refused(f, a, slopes=torch.zeros(3, device=DEV))
    refused(f, a, k_scale=torch.ones(2, device=DEV))
    refused(f, a, softcap=-1.0)
    refused(f, a, softcap=float("nan"))
    refused(f, a, scale=float("inf"))
    refused(f, a, window=-1)
    refused(f, a, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    refused(f, a, out=torch.empty((2, 2, 4, 64), device=DEV))
    refused(f, a, window=2 ** 32 + 5)                      # 5, cut to 32 bits
    dense = a["q"].contiguous()
    refused(f, a, q=dense, out=dense)
    refused(f, a, out=a["k_cache"].flatten()[:2 * 2 * 4 * 64].view(2, 2, 4, 64))
    refused(f, a, page_table=torch.empty((2, 2 ** 31 + 3), dtype=torch.int32, device=DEV))
    e = dev(fc.make_attention(40, B=2, R=2, Hkv=2, G=2, D=64, cache="e4m3"))
    refused(f, e, k_scale=None)
    refused(f, e, v_scale=torch.ones(2, dtype=torch.float64, device=DEV))
    wide = torch.zeros((2, 2, 4, 65), dtype=torch.bfloat16, device=DEV)
    refused(f, a, q=wide[..., 1:])                         # rows at odd places
    refused(f, a, q=torch.zeros((2, 66, 4, 64), dtype=torch.bfloat16, device=DEV))


def test_append_refusals(run):
    a = dev(fc.make_append(41))
    f = tv.spec_kv_append
    refused(f, a, k=a["k"].float())
    refused(f, a, k=a["k"][:, :, :1])
    refused(f, a, v=a["v"][:, :2])
    refused(f, a, k_cache=a["k_cache"][:1].expand(a["k_cache"].shape))     # every page at one place
    refused(f, a, v_cache=a["v_cache"].half())
    refused(f, a, draft_len=torch.zeros(3, dtype=torch.int32, device=DEV))
    refused(f, a, kv_len=None)
    refused(f, a, k=a["k"].cpu())


def test_adjust_refusals(run):
    a = dev(fc.make_adjust(42))
    f = tv.spec_adjust
    with pytest.raises(ValueError):                        # 1000 columns, cut to 32 bits
        f(torch.empty((1, 1, 2 ** 32 + 1000), dtype=torch.bfloat16, device=DEV))
    refused(f, a, logits=a["logits"].half())
    refused(f, a, logits=a["logits"][:, :, :999])
    refused(f, a, logits=a["logits"].cpu())
    refused(f, a, tokens=None)
    refused(f, a, tokens=a["tokens"][:, :1].contiguous())
    refused(f, a, tokens=a["tokens"].long())
    refused(f, a, hist_len=None)
    refused(f, a, history=None)
    refused(f, a, history=a["history"].long())
    refused(f, a, repetition=a["repetition"].double())
    refused(f, a, bias_values=None)
    refused(f, a, bias_values=a["bias_values"][:, :2].contiguous())
    refused(f, a, admit=a["admit"][:, :5].contiguous())
    refused(f, a, admit=None)
    refused(f, a, admit_row=None)                          # 9 masks for 8 rows
    refused(f, a, out_dtype=torch.bfloat16)
    refused(f, a, out=torch.empty((2, 4, 999), device=DEV))
    both = torch.empty(2 * 4 * 1000 + 4, device=DEV)
    refused(f, dict(a, logits=both[4:].view(2, 4, 1000)), out=both[:-4].view(2, 4, 1000))


def test_nothing_is_allocated_with_out_and_workspace(run):
    a = dev(fc.make_attention(43, B=2, R=2, Hkv=2, G=2, D=64, lens=[500, 20]))
    out = torch.empty_like(tv.spec_attention(**a))
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    tv.spec_attention(**a, out=out, workspace=ws)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
