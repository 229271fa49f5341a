"""float64 references of the operators around a verify step's model, in plain numpy:
the paged KV cache's write and attention and the adjustment of the logits.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``.

They follow the definitions in include/spec_forward.h one batch row at a time and
share no code with the HIP path. Tensors come as float64 arrays of the exact values
the library sees (e4m3 codes as uint8). attention_ref and adjust_ref also return
how far a correct float32 evaluation with the stated roundings may be from the
exact result, element by element (derived at each function).
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24                                           # half a step, relative to the value
HALF_STEP = {"f32": U32, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -24, "bf16": 2.0 ** -126}
# the absolute half step of a weight below the smallest normal, where the largest weight is 1
WEIGHT = {"f16": 2.0 ** -25 / 2.0 ** 7, "bf16": 2.0 ** -126}


def e4m3_value(codes: np.ndarray) -> np.ndarray:
    """The values of e4m3 codes (OCP: bias 7, no infinities, S.1111.111 = NaN)."""
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(c & 128, -v, v)


def e4m3_code(x: np.ndarray) -> np.ndarray:
    """Codes of the nearest e4m3 values (ties to the even code), saturating at +-448."""
    table = e4m3_value(np.arange(127, dtype=np.uint8))     # 0 .. 448, ascending
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(table, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - table[lo], table[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code)
    return (code | np.where(np.signbit(x) & ~np.isnan(x), 128, 0)).astype(np.uint8)


def seq_rows(kv_len: int, draft_len, R: int, positions: int) -> int:
    """Tokens in use of a batch row, 0 if its lengths are out of range."""
    n = R if draft_len is None else int(draft_len) + 1
    return 0 if kv_len < 0 or n < 1 or n > R or kv_len + n > positions else n


def append_ref(x, cache, table, kv_len, draft_len=None, scale=None):
    """x [B, R, H, D] (float64 values, or any array for a plain copy) into a copy of
    cache [pages, H, page_size, D]; with scale, cache holds e4m3 codes."""
    cache = cache.copy()
    B, R = x.shape[:2]
    pages, _, ps, _ = cache.shape
    for b in range(B):
        for i in range(seq_rows(int(kv_len[b]), None if draft_len is None else draft_len[b], R, table.shape[1] * ps)):
            t = int(kv_len[b]) + i
            page = int(table[b, t // ps])
            if 0 <= page < pages:
                y = x[b, i]
                if scale is not None:                      # the quotient in float32, as defined
                    with np.errstate(all="ignore"):
                        y = e4m3_code(y.astype(np.float32) / scale.astype(np.float32)[:, None])
                cache[page, :, t % ps] = y
    return cache


def attention_ref(q, k_cache, v_cache, table, kv_len, *, dtype, draft_len=None, scale=None, softcap=0.0, window=0,
                  slopes=None, k_scale=None, v_scale=None):
    """(out, tolerance), both [B, R, Hq, D].

    Tolerance, with u half a step of dtype: the weights exp(s - m) are rounded to
    dtype (u each; below dtype's smallest normal an absolute half step, WEIGHT of the
    largest weight), the scores
    carry the rounding of a D-term float32 product sum ((D + 4) U32 of sum |q k|
    scale), of the factors and the bias (8 U32 of the largest term; a tanh's absolute
    2^-21 of the cap, or, for caps of 256 and more, where that is less, 2^-19 of the score:
    the series' next term is 2^-21.5 of it below a quarter of the cap; above it, with
    A = 2^-23, the argument's rounding moves 1 - 2 / (1 + e) by at most 0.45 A, exp2 by
    0.5 A, the sum by 0.38 A, the reciprocal by 0.76 A and the difference by 0.5 A, together
    2.6 A of at least tanh(1/4) = 0.245) and of exp2 (2^-21 with its argument's reduction), the sums over
    n tokens n U32 of their absolute value, and the result u of itself. A relative
    error d_t of weight t moves the result by p_t d_t (v_t - out).
    """
    B, R, Hq, D = q.shape
    pages, Hkv, ps, _ = k_cache.shape
    G = Hq // Hkv
    u = HALF_STEP[dtype]
    out = np.zeros((B, R, Hq, D))
    tol = np.zeros((B, R, Hq, D))
    sc = 1.0 / np.sqrt(D) if scale is None else scale
    for b in range(B):
        kv = int(kv_len[b])
        n = seq_rows(kv, None if draft_len is None else draft_len[b], R, table.shape[1] * ps)
        if n == 0:
            out[b] = np.nan
            continue
        lo = max(0, kv + 1 - window) if window else 0
        ids = table[b, np.arange(lo, kv + n) // ps]
        if ((ids < 0) | (ids >= pages)).any():
            out[b] = np.nan
            continue
        slot = np.arange(lo, kv + n) % ps
        for h in range(Hkv):
            K, V = k_cache[ids, h, slot], v_cache[ids, h, slot]
            if k_scale is not None:
                K, V = K * k_scale[h], V * v_scale[h]
            for i in range(n):
                first = max(lo, kv + i + 1 - window) if window else 0
                Kv, Vv = K[first - lo:kv + i + 1 - lo], V[first - lo:kv + i + 1 - lo]
                for g in range(G):
                    x = q[b, i, h * G + g]
                    with np.errstate(all="ignore"):
                        s = sc * (Kv @ x)
                        raw = sc * (np.abs(Kv) @ np.abs(x))
                        ds = (D + 4) * U32 * raw + 8 * U32 * np.abs(s)
                        if softcap:
                            s = softcap * np.tanh(s / softcap)
                            ds = ds + np.minimum(2.0 ** -21 * softcap, 2.0 ** -19 * np.abs(s) if softcap >= 256 else np.inf)
                        if slopes is not None:
                            away = slopes[h * G + g] * (np.arange(first, kv + i + 1) - (kv + i))
                            s = s + away
                            ds = ds + 8 * U32 * np.abs(away)
                        p = np.exp(s - s.max())
                        o = (p @ Vv) / p.sum()
                        d = u + ds + 2.0 ** -21 + len(s) * U32
                        t = ((p * d) @ np.abs(Vv) + (p * d).sum() * np.abs(o)) / p.sum()
                        t = t + WEIGHT[dtype] * np.abs(Vv).sum(0) / p.sum()
                        out[b, i, h * G + g] = o
                        tol[b, i, h * G + g] = 1.01 * t + u * (np.abs(o) + 1.01 * t) + TINY[dtype]
    return out, tol


def adjust_ref(logits, tokens, *, out_dtype, before=None, history=None, hist_len=None, prompt_len=None, repetition=None,
               frequency=None, presence=None, bias_tokens=None, bias_values=None, admit=None, admit_row=None,
               draft_len=None):
    """(out, tolerance), both [B, R, V]; `before` is what rows not in use keep.

    Tolerance: each float32 step is off by U32 of its result, and no intermediate
    result is larger than |x'| + |frequency| count + |presence| + sum |bias| (x' the
    logit after the repetition penalty); there are at most n_bias + 6 steps. Then
    half a step of out_dtype.
    """
    B, R, V = logits.shape
    k = tokens.shape[1]
    out = np.array(before if before is not None else np.zeros((B, R, V)), dtype=np.float64)
    tol = np.zeros((B, R, V))
    for b in range(B):
        rows = R
        if draft_len is not None:
            if not 0 <= int(draft_len[b]) <= k:
                continue
            rows = R - k + int(draft_len[b])
        n = 0 if history is None else int(hist_len[b])
        p = 0 if history is None or prompt_len is None else int(prompt_len[b])
        r = 1.0 if repetition is None else float(repetition[b])
        f = 0.0 if frequency is None else float(frequency[b])
        c = 0.0 if presence is None else float(presence[b])
        if n < 0 or (history is not None and n > history.shape[1]) or not 0 <= p <= n or not (0 < r < np.inf) \
                or not np.isfinite(f) or not np.isfinite(c):
            out[b, :rows] = np.nan
            continue
        line = [] if history is None else [int(t) for t in history[b, :n]]
        bias, size, nb = np.zeros(V), np.zeros(V), 0
        biased = np.zeros(V, bool)
        if bias_tokens is not None:
            nb = bias_tokens.shape[1]
            for t, w in zip(bias_tokens[b], bias_values[b]):
                if 0 <= t < V:
                    bias[t] += w
                    size[t] += abs(w)
                    biased[t] = True
        for i in range(rows):
            m = -1
            if admit is not None:
                m = int(admit_row[b, i]) if admit_row is not None else b * R + i
                if not -1 <= m < len(admit):
                    out[b, i] = np.nan
                    continue
            drafts = [int(t) for t in tokens[b, :i]]
            seen, count = np.zeros(V, bool), np.zeros(V)
            for t in line + drafts:
                if 0 <= t < V:
                    seen[t] = True
            for t in line[p:] + drafts:
                if 0 <= t < V:
                    count[t] += 1
            with np.errstate(all="ignore"):
                x = logits[b, i].astype(np.float64)
                x = np.where(seen, np.where(x > 0, x / r, x * r), x)
                most = np.abs(x) + abs(f) * count + abs(c) + size
                y = x - f * count - np.where(count > 0, c, 0.0)
                y = np.where(biased, y + bias, y)
                e = np.where(seen | biased, (nb + 6) * U32 * most, 0.0)
                e = np.where(np.isfinite(e), e, 0.0)
                if m >= 0:
                    bits = (admit[m][:, None].astype(np.uint32) >> np.arange(32, dtype=np.uint32)) & 1
                    ok = bits.reshape(-1)[:V].astype(bool)
                    y, e = np.where(ok, y, -np.inf), np.where(ok, e, 0.0)
                u = HALF_STEP[out_dtype]
                out[b, i] = y
                tol[b, i] = e + u * (np.abs(np.where(np.isfinite(y), y, 0.0)) + e) + (TINY[out_dtype] if r != 1 else 0)
    return out, tol
