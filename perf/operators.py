"""Cases of the operators around a verify step, with their plain forms.

Three operators, the ones a verify forward needs on either side of its model:

* "append": write the keys and values of a step's new tokens into a paged cache
  (bfloat16, float16, or e4m3 with one scale per head);
* "attention": the step's new tokens (one, or the pending token and k drafts)
  over the paged cache, optionally with scores capped by a tanh, a bias that
  grows with the distance, and a sliding window;
* "adjust": penalties for repeated tokens, biases and grammar masks on the
  step's logits, where position i also counts the drafts before it.

A case is a dict of plain values. ``prepare`` makes its inputs from a seed,
``run`` computes it in plain torch (``own`` false) or by the package's calls
(``own`` true), ``exact`` in 64 bits, ``work`` counts what has to be read,
written and multiplied.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0


def device():
    return "cuda" if torch.cuda.is_available() else "cpu"


# ------------------------------------------------------------------ cases

def adjust_case(name, B, k, V, dtype, rows="target", H=0, bias=0, masks="none", out="same"):
    """rows: "target" (k+1 rows per batch row) or "draft" (k rows); H: longest
    history; bias: biased tokens per batch row; masks: "none", "all" (one for
    every position) or "some" (half of the positions are unconstrained);
    out: "same" type as the logits, or "f32"."""
    return {"name": name, "op": "adjust", "B": B, "k": k, "V": V, "dtype": dtype, "rows": rows, "H": H, "bias": bias,
            "masks": masks, "out": out}


def attention_case(name, B, k, Hkv, G, D, L, page, dtype, cache="same", layout="head", softcap=0.0, window=0,
                   slopes=False):
    """G query heads share each of Hkv cache heads; L: longest total length;
    cache: "same" type as the queries, or "e4m3"; layout: "head" (each head's
    tokens of a page together) or "token" (each token's heads together)."""
    return {"name": name, "op": "attention", "B": B, "k": k, "Hkv": Hkv, "G": G, "D": D, "L": L, "page": page,
            "dtype": dtype, "cache": cache, "layout": layout, "softcap": softcap, "window": window, "slopes": slopes}


def append_case(name, B, R, Hkv, D, L, page, dtype, cache="same", layout="head"):
    """R new tokens per sequence behind up to L cached ones."""
    return {"name": name, "op": "append", "B": B, "R": R, "Hkv": Hkv, "D": D, "L": L, "page": page, "dtype": dtype,
            "cache": cache, "layout": layout}


def listed():
    return [
        # one sequence sampling one token with the three penalties: pure latency
        adjust_case("adjust one token", 1, 0, 32000, "f32", H=512),
        # a serving batch of verify steps, every feature in use
        adjust_case("adjust verify", 64, 5, 151936, "bf16", H=2047, bias=16, masks="some"),
        # structured output over a wide batch: masks and biases, no history
        adjust_case("adjust grammar", 256, 3, 128256, "bf16", bias=5, masks="all"),
        # few sequences with very long contexts
        adjust_case("adjust long history", 8, 5, 151936, "f32", H=65537),
        # one sequence, one token, a short context: pure latency
        attention_case("attention one token", 1, 0, 8, 4, 128, 1000, 16, "bf16"),
        # a serving batch of verify steps over ragged contexts
        attention_case("attention verify", 64, 5, 8, 4, 128, 4096, 16, "bf16"),
        # one verify step over one very long context in an 8-bit cache
        attention_case("attention long e4m3", 1, 4, 8, 8, 128, 131071, 64, "bf16", cache="e4m3"),
        # capped scores in a sliding window, wide heads, a cache with each token's heads together
        attention_case("attention cap window", 16, 3, 4, 2, 256, 8191, 32, "f16", layout="token", softcap=50.0,
                       window=4096),
        # single tokens, every head with its own cache, distance bias
        attention_case("attention distance", 32, 0, 32, 1, 64, 2047, 16, "bf16", slopes=True),
        # the cache write of one decoding sequence
        append_case("append one token", 1, 1, 8, 128, 1000, 16, "bf16"),
        # a wide batch of verify steps into an 8-bit cache
        append_case("append verify e4m3", 256, 4, 8, 128, 2047, 64, "bf16", cache="e4m3"),
        # prompts into the cache
        append_case("append prompts", 8, 2049, 8, 128, 100, 16, "f16", layout="token"),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("adjust", "attention", "append"))
    most = 1.0e9
    while True:
        if op == "adjust":
            k = rng.randint(0, 8)
            c = adjust_case("", log_int(rng, 1, 256), k, log_int(rng, 1000, 152000), rng.choice(("f32", "bf16")),
                            rows=rng.choice(("target", "target", "draft")) if k else "target",
                            H=rng.choice((0, log_int(rng, 1, 65536), log_int(rng, 1, 65536))),
                            bias=rng.choice((0, rng.randint(1, 300))), masks=rng.choice(("none", "some", "all")),
                            out=rng.choice(("same", "f32")))
            limit = 5.0e8
            if not c["H"] and not c["bias"] and c["masks"] == "none":       # nothing to do
                continue
        elif op == "attention":
            dtype = rng.choice(("bf16", "f16"))
            c = attention_case("", log_int(rng, 1, 128), rng.randint(0, 8), rng.choice((1, 2, 4, 8, 12)),
                               rng.randint(1, 8), rng.choice((64, 128, 256)), log_int(rng, 10, 131072),
                               rng.choice((8, 16, 32, 64, 128)), dtype, cache=rng.choice(("same", "same", "e4m3")),
                               layout=rng.choice(("head", "token")), softcap=rng.choice((0.0, 0.0, 30.0, 50.0)),
                               window=rng.choice((0, 0, log_int(rng, 1, 8192))), slopes=rng.random() < 0.25)
            limit = most
            if c["B"] * c["Hkv"] * c["L"] * c["D"] > 2.7e8:      # the cache itself, whatever the window reads of it
                continue
        else:
            c = append_case("", log_int(rng, 1, 256), log_int(rng, 1, 4096), rng.choice((1, 2, 4, 8, 12)),
                            rng.choice((64, 128, 256)), log_int(rng, 1, 4096), rng.choice((8, 16, 32, 64, 128)),
                            rng.choice(("bf16", "f16")), cache=rng.choice(("same", "e4m3")),
                            layout=rng.choice(("head", "token")))
            limit = 2.0e8
            if c["B"] * c["Hkv"] * (c["L"] + c["R"]) * c["D"] > 2.0e8:
                continue
        if work(c)["bytes"] <= limit:
            del c["name"]
            return c


def rows_of(case):
    return case["k"] + 1 if case["rows"] == "target" else case["k"]


def work(case):
    if case["op"] == "adjust":
        B, k, V, H, nb = case["B"], case["k"], case["V"], case["H"], case["bias"]
        R, es = rows_of(case), 4 if case["dtype"] == "f32" else 2
        eo = 4 if case["out"] == "f32" else es
        share = {"none": 0.0, "some": 0.5, "all": 1.0}[case["masks"]]
        n = B * R * V
        by = n * (es + eo) + share * B * R * ((V + 31) // 32) * 4 + B * k * 4
        by += B * (0.75 * H * 4 + 20 if H else 0) + B * nb * 8 + (B * R * 4 if share else 0)
        return {"bytes": by, "flops": B * R * (0.75 * H + nb) * 4}
    D, Hkv = case["D"], case["Hkv"]
    es = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "append":
        n = case["B"] * case["R"] * Hkv * D * 2
        return {"bytes": n * (2 + es) + case["B"] * 4 + case["B"] * (case["R"] / case["page"] + 1) * 4, "flops": 0}
    B, R = case["B"], case["k"] + 1
    mean = 0.75 * case["L"] if case["L"] > 2 * R else max(R, 0.75 * case["L"])
    seen = min(mean, case["window"] + R - 1) if case["window"] else mean
    M = R * case["G"]
    by = B * (2 * Hkv * seen * D * es + seen / case["page"] * 4 + 2 * M * Hkv * D * 2 + 4)
    return {"bytes": by, "flops": 4.0 * B * Hkv * M * seen * D}


# ------------------------------------------------------------------ inputs

def gen(seed):
    g = torch.Generator(device=device())
    g.manual_seed(int(seed))
    return g


def ints(g, lo, hi, shape):
    return torch.randint(lo, hi, shape, generator=g, device=device(), dtype=torch.int32)


def prepare(case, seed):
    g, dev = gen(seed), device()
    if case["op"] == "adjust":
        return prepare_adjust(case, g, dev)
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    dtype = DTYPES[case["dtype"]]
    R = case["R"] if case["op"] == "append" else case["k"] + 1
    most = case["L"] if case["op"] == "append" else max(0, case["L"] - R)
    kv_len = ints(g, most // 2, most + 1, (B,))
    pages = (most + R + page - 1) // page
    table = torch.randperm(B * pages, generator=g, device=dev).to(torch.int32).view(B, pages)
    shape = (B * pages, Hkv, page, D) if case["layout"] == "head" else (B * pages, page, Hkv, D)
    s = {"case": dict(case), "kv_len": kv_len, "table": table, "k_scale": None, "v_scale": None}
    e4m3 = case["cache"] == "e4m3"
    if e4m3:
        s["k_scale"] = 0.01 + 0.02 * torch.rand(Hkv, generator=g, device=dev)
        s["v_scale"] = 0.01 + 0.02 * torch.rand(Hkv, generator=g, device=dev)
    if case["op"] == "append":
        # keys and values are slices of the fused projection's output, with as many query heads beside them
        qkv = torch.randn((B, R, 3 * Hkv, D), generator=g, device=dev).to(dtype)
        s["k"], s["v"] = qkv[:, :, Hkv:2 * Hkv], qkv[:, :, 2 * Hkv:]
        cache = [torch.zeros(shape, device=dev, dtype=torch.uint8).view(DTYPES["e4m3"]) if e4m3
                 else torch.zeros(shape, device=dev, dtype=dtype) for _ in range(2)]
    else:
        G = case["G"]
        qkv = torch.randn((B, R, (G + 2) * Hkv, D), generator=g, device=dev).mul_(2.0).to(dtype)
        s["q"] = qkv[:, :, :G * Hkv]
        if e4m3:
            cache = [torch.randn(shape, generator=g, device=dev, dtype=torch.float16).mul_(50.0).to(DTYPES["e4m3"])
                     for _ in range(2)]
        else:
            cache = [torch.randn(shape, generator=g, device=dev, dtype=dtype) for _ in range(2)]
        Hq = G * Hkv
        s["slopes"] = (torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=dev, dtype=torch.float32) / Hq)
                       if case["slopes"] else None)
    if case["layout"] == "token":
        cache = [c.transpose(1, 2) for c in cache]
    s["k_cache"], s["v_cache"] = cache
    return s


def prepare_adjust(case, g, dev):
    B, k, V, H, nb = case["B"], case["k"], case["V"], case["H"], case["bias"]
    R = rows_of(case)
    s = {"case": dict(case), "tokens": ints(g, 0, V, (B, k)), "history": None, "hist_len": None, "prompt_len": None,
         "repetition": None, "frequency": None, "presence": None, "bias_tokens": None, "bias_values": None,
         "admit": None, "admit_row": None}
    s["logits"] = torch.randn((B, R, V), generator=g, device=dev).mul_(3.0).to(DTYPES[case["dtype"]])
    if H:
        # frequent tokens come back often, as in text
        u = torch.rand((B, H), generator=g, device=dev)
        s["history"] = (V * u * u * u).to(torch.int32).clamp_(max=V - 1)
        s["hist_len"] = ints(g, H // 2, H + 1, (B,))
        s["prompt_len"] = (s["hist_len"] * torch.rand(B, generator=g, device=dev)).to(torch.int32)
        s["repetition"] = 1.0 + 0.3 * torch.rand(B, generator=g, device=dev)
        s["frequency"] = 0.5 * torch.rand(B, generator=g, device=dev)
        s["presence"] = 0.5 * torch.rand(B, generator=g, device=dev)
        if k:
            some = torch.rand((B, k), generator=g, device=dev) < 0.5      # drafts repeat the context, and each other
            at = (torch.rand((B, k), generator=g, device=dev) * s["hist_len"][:, None]).long().clamp_(max=H - 1)
            s["tokens"] = torch.where(some, s["history"].gather(1, at), s["tokens"])
    if nb:
        first = ints(g, 0, V, (B, 1))
        step = max(1, V // nb)
        s["bias_tokens"] = ((first + torch.arange(nb, device=dev, dtype=torch.int32) * step) % V).contiguous()
        s["bias_values"] = 4.0 * torch.randn((B, nb), generator=g, device=dev)
    if case["masks"] != "none":
        # a grammar state admits most tokens, about half, or few
        n, W = B * R, (V + 31) // 32
        bits = [torch.randint(-2 ** 31, 2 ** 31, (n, W), generator=g, device=dev, dtype=torch.int64).to(torch.int32)
                for _ in range(3)]
        kind = torch.arange(n, device=dev)[:, None] % 3
        few, many = bits[0] & bits[1] & bits[2], bits[0] | bits[1] | bits[2]
        s["admit"] = torch.where(kind == 0, few, torch.where(kind == 1, bits[0], many)).contiguous()
        s["admit_row"] = torch.arange(n, device=dev, dtype=torch.int32).view(B, R)
        if case["masks"] == "some":
            s["admit_row"] = torch.where(torch.rand((B, R), generator=g, device=dev) < 0.5, -1, s["admit_row"])
            s["admit_row"] = s["admit_row"].to(torch.int32).contiguous()
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"adjust": own_adjust, "attention": own_attention, "append": own_append}[op](state)
    return {"adjust": plain_adjust, "attention": plain_attention, "append": plain_append}[op](state)


def own_adjust(s):
    import token_verification_amd as tv
    return tv.spec_adjust(s["logits"], s["tokens"], history=s["history"], hist_len=s["hist_len"],
                          prompt_len=s["prompt_len"], repetition=s["repetition"], frequency=s["frequency"],
                          presence=s["presence"], bias_tokens=s["bias_tokens"], bias_values=s["bias_values"],
                          admit=s["admit"], admit_row=s["admit_row"],
                          out_dtype=torch.float32 if s["case"]["out"] == "f32" else None)


def own_attention(s):
    import token_verification_amd as tv
    c = s["case"]
    return tv.spec_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_len"], softcap=c["softcap"],
                             window=c["window"], slopes=s["slopes"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def own_append(s):
    import token_verification_amd as tv
    tv.spec_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["kv_len"], k_scale=s["k_scale"],
                      v_scale=s["v_scale"])
    return {"k": s["k_cache"], "v": s["v_cache"]}


def plain_adjust(s):
    x = s["logits"].float()
    B, R, V = x.shape
    dev, tokens = x.device, s["tokens"].long()
    k = tokens.shape[1]
    if s["history"] is not None:
        hist, H = s["history"].long(), s["history"].shape[1]
        at = torch.arange(H, device=dev)
        live = at < s["hist_len"][:, None]
        made = live & (at >= s["prompt_len"][:, None])
        zero = torch.zeros((B, V), device=dev)
        seen = zero.scatter_add(1, hist, live.float())[:, None]
        count = zero.scatter_add(1, hist, made.float())[:, None]
        if k:
            before = (torch.arange(k, device=dev) < torch.arange(R, device=dev)[:, None]).float()
            drafts = torch.zeros((B, R, V), device=dev).scatter_add_(
                2, tokens[:, None].expand(B, R, k), before.expand(B, R, k).contiguous())
            seen, count = seen + drafts, count + drafts
        rep = s["repetition"][:, None, None]
        x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
        x = x - s["frequency"][:, None, None] * count - s["presence"][:, None, None] * (count > 0)
    if s["bias_tokens"] is not None:
        x = x + torch.zeros((B, V), device=dev).scatter_add_(1, s["bias_tokens"].long(), s["bias_values"])[:, None]
    if s["admit"] is not None:
        at = torch.arange(V, device=dev)
        row = s["admit_row"].long()
        word = s["admit"][row.clamp(min=0)][:, :, at >> 5]
        admitted = ((word >> (at & 31).to(torch.int32)) & 1).bool() | (row < 0)[:, :, None]
        x = x.masked_fill(~admitted, -math.inf)
    return x if s["case"]["out"] == "f32" else x.to(s["logits"].dtype)


def codes(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def gathered(cache, table, scale):
    """[B, Hkv, pages * page, D] in float32."""
    c = codes(cache)[table.long()].view(cache.dtype).float()
    B, n, Hkv, page, D = c.shape
    c = c.transpose(1, 2).reshape(B, Hkv, n * page, D)
    return c if scale is None else c * scale[:, None, None]


def plain_attention(s):
    case, q = s["case"], s["q"].float()
    B, R, Hq, D = q.shape
    Hkv = case["Hkv"]
    G = Hq // Hkv
    K = gathered(s["k_cache"], s["table"], s["k_scale"])
    V = gathered(s["v_cache"], s["table"], s["v_scale"])
    j = torch.arange(K.shape[2], device=q.device)
    pos = s["kv_len"][:, None] + torch.arange(R, device=q.device)                      # [B, R]
    far = (j - pos[:, :, None])[:, None, :, None, :]                                   # [B, 1, R, 1, L]
    x = q.view(B, R, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, D)
    x = torch.matmul(x, K.transpose(2, 3).contiguous()).view(B, Hkv, R, G, -1) * (1.0 / math.sqrt(D))
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    if s["slopes"] is not None:
        x = x + s["slopes"].view(1, Hkv, 1, G, 1) * far
    hidden = far > 0
    if case["window"]:
        hidden = hidden | (far <= -case["window"])
    x = x.masked_fill(hidden, -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    total = x.sum(-1, keepdim=True)
    V = V.masked_fill((j >= s["kv_len"][:, None] + R)[:, None, :, None], 0.0)
    o = torch.matmul(x.view(B, Hkv, R * G, -1), V).view(B, Hkv, R, G, D) / total
    return o.permute(0, 2, 1, 3, 4).reshape(B, R, Hq, D).to(s["q"].dtype)


def plain_append(s):
    B, R, Hkv, D = s["k"].shape
    page = s["case"]["page"]
    pos = s["kv_len"].long()[:, None] + torch.arange(R, device=s["k"].device)
    at, slot = s["table"].long().gather(1, pos // page), pos % page
    put(s["k_cache"], at, slot, s["k"], s["k_scale"])
    put(s["v_cache"], at, slot, s["v"], s["v_scale"])
    return {"k": s["k_cache"], "v": s["v_cache"]}


def put(cache, at, slot, x, scale):
    if scale is not None:
        x = (x.float() / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)
    codes(cache)[at, :, slot] = codes(x)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"adjust": exact_adjust, "attention": exact_attention, "append": exact_append}[case["op"]](s)


def exact_adjust(s):
    x = s["logits"].double()
    B, R, V = x.shape
    for b in range(B):
        if s["history"] is not None:
            n, p = int(s["hist_len"][b]), int(s["prompt_len"][b])
            line = s["history"][b].long()
            seen, count = torch.bincount(line[:n], minlength=V), torch.bincount(line[p:n], minlength=V)
            r, f, q = (float(s[w][b]) for w in ("repetition", "frequency", "presence"))
            for i in range(R):
                if i:
                    t = int(s["tokens"][b, i - 1])
                    seen[t] += 1
                    count[t] += 1
                v = x[b, i]
                v[seen > 0] = torch.where(v > 0, v / r, v * r)[seen > 0]
                v -= f * count.double()
                v -= q * (count > 0).double()
        if s["bias_tokens"] is not None:
            x[b].index_add_(1, s["bias_tokens"][b].long(), s["bias_values"][b].double().expand(R, -1).contiguous())
        if s["admit"] is not None:
            for i in range(R):
                m = int(s["admit_row"][b, i])
                if m >= 0:
                    bit = torch.arange(32, device=x.device, dtype=torch.int32)
                    ok = ((s["admit"][m][:, None] >> bit) & 1).reshape(-1)[:V].bool()
                    x[b, i][~ok] = -math.inf
    return x


def exact_attention(s):
    case, page = s["case"], s["case"]["page"]
    B, R, Hq, D = s["q"].shape
    Hkv = case["Hkv"]
    G = Hq // Hkv
    out = torch.zeros((B, R, Hq, D), dtype=torch.float64, device=s["q"].device)
    for b in range(B):
        n = int(s["kv_len"][b])
        used = s["table"][b, :(n + R + page - 1) // page].long()
        k, v = (codes(c)[used].view(c.dtype).double().transpose(0, 1).reshape(Hkv, -1, D)
                for c in (s["k_cache"], s["v_cache"]))
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"].double()[:, None, None], v * s["v_scale"].double()[:, None, None]
        for i in range(R):
            lo = max(0, n + i + 1 - case["window"]) if case["window"] else 0
            q = s["q"][b, i].double().view(Hkv, G, D)
            x = torch.matmul(k[:, lo:n + i + 1], q.transpose(1, 2)) / math.sqrt(D)      # [Hkv, seen, G]
            if case["softcap"]:
                x = torch.tanh(x / case["softcap"]) * case["softcap"]
            if s["slopes"] is not None:
                away = torch.arange(lo - n - i, 1, device=x.device, dtype=torch.float64)
                x = x + away[None, :, None] * s["slopes"].double().view(Hkv, 1, G)
            p = torch.softmax(x, 1)
            out[b, i] = torch.matmul(p.transpose(1, 2), v[:, lo:n + i + 1]).reshape(Hq, D)
    return out


def to_e4m3(x):
    """The nearest e4m3 value (ties to even), saturating, in 64 bits."""
    a = x.abs().clamp(max=E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign(torch.clamp(torch.round(a / step) * step, max=E4M3_MAX), x)


def exact_append(s):
    page, got = s["case"]["page"], {}
    B, R = s["k"].shape[:2]
    for name in ("k", "v"):
        cache = s[name + "_cache"].double()
        x = s[name].double()
        if s[name + "_scale"] is not None:
            x = to_e4m3(x / s[name + "_scale"].double()[:, None])
        for b in range(B):
            pos = int(s["kv_len"][b]) + torch.arange(R, device=x.device)
            cache[s["table"][b].long()[pos // page], :, pos % page] = x[b]
        got[name] = cache
    return got
