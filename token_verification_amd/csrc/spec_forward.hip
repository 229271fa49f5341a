// spec_forward.hip -- the operators around a verify step's model for MI355X (gfx950):
// the paged KV cache's write and attention, and the adjustment of the logits.
//
// What is computed is stated in include/spec_forward.h.
//
// Every reduction uses a fixed order, so results are bitwise reproducible.

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "spec_forward.h"

namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float F32_MAX = 3.402823466e38f;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float E4M3_MAX = 448.0f;

// ------------------------------------------------------------------ element types

__device__ inline float bits_f32(unsigned u) { return __builtin_bit_cast(float, u); }

struct Bf16 {
    using type = __bf16;
    __device__ static inline float lo(unsigned w) { return bits_f32(w << 16); }
    __device__ static inline float hi(unsigned w) { return bits_f32(w & 0xffff0000u); }
};

struct F16 {
    using type = _Float16;
    __device__ static inline float lo(unsigned w) {
        return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<unsigned short>(w)));
    }
    __device__ static inline float hi(unsigned w) {
        return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<unsigned short>(w >> 16)));
    }
};

// two floats to two 16-bit values, each rounded to nearest even
template <class T>
__device__ inline unsigned pack2(float a, float b) {
    typedef typename T::type v2 __attribute__((ext_vector_type(2)));
    const v2 p = {static_cast<typename T::type>(a), static_cast<typename T::type>(b)};
    return __builtin_bit_cast(unsigned, p);
}

// ------------------------------------------------------------------ paged cache

struct Cache {
    char* k;
    char* v;
    long long ks[3], vs[3];    // bytes between pages, heads, tokens
    const int* table;          // [B, max_pages]
    const int* kv_len;         // [B]
    const int* draft_len;      // [B] or null
    const float* k_scale;      // [Hkv], e4m3 only
    const float* v_scale;
    long long pages;
    int max_pages, shift;      // page_size = 1 << shift
    int B, R, Hkv;
};

// The first position and the number of tokens in use of batch row b; 0 tokens
// if its length is out of range (a row in use has at least one).
__device__ inline int seq_rows(const Cache& C, int b, int& kv) {
    kv = C.kv_len[b];
    const int n = C.draft_len ? C.draft_len[b] + 1 : C.R;
    const long long cap = static_cast<long long>(C.max_pages) << C.shift;
    // a draft_len of INT_MAX wraps to a negative n: also out of range
    return kv < 0 || n < 1 || n > C.R || static_cast<long long>(kv) + n > cap ? 0 : n;
}

__device__ inline bool page_ok(const Cache& C, int page) { return page >= 0 && page < C.pages; }

// ------------------------------------------------------------------ cache write
//
// Bound by memory: every new key and value is read and written once. One
// thread moves 16 bytes of the cache for keys and for values, so that a wave's
// stores cover whole head rows (D * 2 bytes, 256 at D = 128, contiguous in
// either cache order), and finds its place itself: two dependent loads (length,
// page id), served by L2 for all but the first threads of a token.

constexpr int NTA = 256;

struct AppendParams {
    Cache c;
    const char* k;
    const char* v;
    long long xk[3], xv[3];    // bytes between batch rows, tokens, heads
    unsigned cph_shift;        // 16-byte cache chunks per head row = 1 << cph_shift
    unsigned cpt;              // chunks per token (all heads)
    long long chunks;          // B * R * cpt
};

// e4m3 codes of four values x / s, saturating; NaN stays NaN
template <class T>
__device__ inline unsigned e4m3x4(unsigned a, unsigned b, float s) {
    float x[4] = {T::lo(a) / s, T::hi(a) / s, T::lo(b) / s, T::hi(b) / s};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = x[j] != x[j] ? x[j] : fminf(fmaxf(x[j], -E4M3_MAX), E4M3_MAX);
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    return static_cast<unsigned>(__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true));
}

template <class T, bool E4M3>
__device__ inline void append_chunk(const char* x, char* cache, float s) {
    if constexpr (E4M3) {
        const u32x4 a = reinterpret_cast<const u32x4*>(x)[0], b = reinterpret_cast<const u32x4*>(x)[1];
        u32x4 o;
        o.x = e4m3x4<T>(a.x, a.y, s); o.y = e4m3x4<T>(a.z, a.w, s);
        o.z = e4m3x4<T>(b.x, b.y, s); o.w = e4m3x4<T>(b.z, b.w, s);
        *reinterpret_cast<u32x4*>(cache) = o;
    } else {
        *reinterpret_cast<u32x4*>(cache) = *reinterpret_cast<const u32x4*>(x);
    }
}

template <class T, bool E4M3>
__global__ __launch_bounds__(NTA) void append_kernel(AppendParams A) {
    const Cache& C = A.c;
    const long long step = static_cast<long long>(gridDim.x) * NTA;
    for (long long n = static_cast<long long>(blockIdx.x) * NTA + threadIdx.x; n < A.chunks; n += step) {
        const long long tok = n / A.cpt;
        const unsigned r = static_cast<unsigned>(n - tok * A.cpt);
        const int h = static_cast<int>(r >> A.cph_shift), c = static_cast<int>(r & ((1u << A.cph_shift) - 1));
        const int b = static_cast<int>(tok / C.R), i = static_cast<int>(tok - static_cast<long long>(b) * C.R);
        int kv;
        if (i >= seq_rows(C, b, kv)) continue;
        const int t = kv + i;
        const int page = C.table[static_cast<long long>(b) * C.max_pages + (t >> C.shift)];
        if (!page_ok(C, page)) continue;
        const int slot = t & ((1 << C.shift) - 1);
        const long long in = 16ll * c * (E4M3 ? 2 : 1);
        append_chunk<T, E4M3>(A.k + b * A.xk[0] + i * A.xk[1] + h * A.xk[2] + in,
                              C.k + page * C.ks[0] + h * C.ks[1] + slot * C.ks[2] + 16ll * c,
                              E4M3 ? C.k_scale[h] : 1.0f);
        append_chunk<T, E4M3>(A.v + b * A.xv[0] + i * A.xv[1] + h * A.xv[2] + in,
                              C.v + page * C.vs[0] + h * C.vs[1] + slot * C.vs[2] + 16ll * c,
                              E4M3 ? C.v_scale[h] : 1.0f);
    }
}

// ------------------------------------------------------------------ attention

struct AttnParams {
    Cache c;
    const char* q;
    long long qs[3];           // bytes between batch rows, tokens, heads
    const float* slopes;       // [Hq] or null
    char* out;                 // [B, R, Hq, D]
    float scale, softcap;
    int window, Hq, G;
};

constexpr int NTQ = 256;

// One workgroup per query row: scores of 256 tokens at a time, one per thread,
// then one output element per thread.
template <class T, int D, bool E4M3>
__global__ __launch_bounds__(NTQ) void attn_kernel(AttnParams A) {
    const Cache& C = A.c;
    __shared__ float q[D], p[NTQ], red[NTQ];
    __shared__ const char* vrow[NTQ];
    __shared__ int bad;
    const int t = static_cast<int>(threadIdx.x);
    const int hq = static_cast<int>(blockIdx.x) % A.Hq, bi = static_cast<int>(blockIdx.x) / A.Hq;
    const int b = bi / C.R, i = bi % C.R, h = hq / A.G;
    typename T::type* out = reinterpret_cast<typename T::type*>(A.out) + static_cast<long long>(blockIdx.x) * D;
    int kv;
    const int n = seq_rows(C, b, kv);
    if (i >= n) {
        if (t < D) out[t] = static_cast<typename T::type>(n ? 0.0f : NAN);
        return;
    }
    const int pos = kv + i, lo = A.window > 0 ? max(0, pos + 1 - A.window) : 0;
    if (t == 0) bad = 0;
    if (t < D)
        q[t] = static_cast<float>(reinterpret_cast<const typename T::type*>(A.q + b * A.qs[0] + i * A.qs[1] +
                                                                             hq * A.qs[2])[t]);
    __syncthreads();
    const float ksc = E4M3 ? C.k_scale[h] : 1.0f, vsc = E4M3 ? C.v_scale[h] : 1.0f;
    auto value = [&](const char* row, int j) -> float {
        if constexpr (E4M3) {
            typedef __bf16 v2 __attribute__((ext_vector_type(2)));
            const v2 f = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(reinterpret_cast<const unsigned char*>(row)[j],
                                                                   1.0f, false);
            return static_cast<float>(f.x);
        } else {
            return static_cast<float>(reinterpret_cast<const typename T::type*>(row)[j]);
        }
    };
    float m = -F32_MAX, l = 0.0f, o = 0.0f;
    for (int t0 = lo; t0 <= pos; t0 += NTQ) {
        const int tok = t0 + t;
        float x = -INFINITY;
        if (tok <= pos) {
            int page = C.table[static_cast<long long>(b) * C.max_pages + (tok >> C.shift)];
            if (!page_ok(C, page)) { bad = 1; page = 0; }
            const int slot = tok & ((1 << C.shift) - 1);
            const char* krow = C.k + page * C.ks[0] + h * C.ks[1] + slot * C.ks[2];
            vrow[t] = C.v + page * C.vs[0] + h * C.vs[1] + slot * C.vs[2];
            float s = 0.0f;
            for (int j = 0; j < D; ++j) s += q[j] * value(krow, j);
            x = s * A.scale * ksc;
            if (A.softcap > 0.0f) x = A.softcap * tanhf(x / A.softcap);
            if (A.slopes) x += A.slopes[hq] * static_cast<float>(tok - pos);
        }
        red[t] = x;
        __syncthreads();
        float mx = m;
        for (int j = 0; j < NTQ; ++j) mx = fmaxf(mx, red[j]);
        const float e = exp2f((x - mx) * LOG2E), r = exp2f((m - mx) * LOG2E);
        p[t] = x == -INFINITY && tok > pos ? 0.0f : e;
        m = mx;
        __syncthreads();
        l *= r;
        o *= r;
        const int cnt = min(NTQ, pos + 1 - t0);
        for (int j = 0; j < cnt; ++j) {
            l += p[j];
            if (t < D) o += p[j] * value(vrow[j], t);
        }
        __syncthreads();
    }
    if (t < D) out[t] = static_cast<typename T::type>(bad ? NAN : o / l * vsc);
}

// ------------------------------------------------------------------ logit adjustment
//
// Bound by memory: the logits are read and written once, the masks and the
// histories are small beside them. A workgroup owns a segment of the
// vocabulary for all R rows of a batch row. It counts the segment's tokens of
// the history in LDS (integer atomics, so the order does not matter), streams
// the segment of every row through registers with the mask applied, and then
// goes over the few tokens with a count or a bias once more, taking their
// logits from the input again and overwriting what it had stored. The streaming
// part so has no lookups, and rows whose start is not 16-byte aligned (an odd
// V) differ only in the head and tail elements that are moved one by one.

constexpr int NTJ = 256;
constexpr int SEG_MAX = 8192;                              // most tokens of a segment
constexpr unsigned SEEN = 0x80000000u;                     // count word: the token is in the prompt
constexpr unsigned NOBIAS = 0xffffffffu;

struct AdjustParams {
    const char* in;
    char* out;
    const int* tokens;         // [B, k] or null
    const int* draft_len;
    const int* history;        // [B, H] or null
    const int* hist_len;
    const int* prompt_len;
    const float* rep;
    const float* freq;
    const float* pres;
    const int* bias_tok;       // [B, nb]
    const float* bias_val;
    const unsigned* admit;     // [n_admit, W] or null
    const int* admit_row;      // [B, R] or null
    int B, R, V, k, H, nb, n_admit, W;
    int seg, nseg;
    int vec;                   // 16-byte vectors usable
    int inplace;               // out is the input
};

struct InF32 {
    static constexpr int VE = 4, ES = 4;
    __device__ static inline float one(const char* p, long long n) { return reinterpret_cast<const float*>(p)[n]; }
};
struct InBf16 {
    static constexpr int VE = 8, ES = 2;
    __device__ static inline float one(const char* p, long long n) {
        return bits_f32(static_cast<unsigned>(reinterpret_cast<const unsigned short*>(p)[n]) << 16);
    }
};

// I: input type; OF: float32 output (else the input's type)
template <class I, bool OF>
__device__ inline void put_one(char* p, long long n, float x) {
    if constexpr (OF || I::ES == 4) reinterpret_cast<float*>(p)[n] = x;
    else reinterpret_cast<__bf16*>(p)[n] = static_cast<__bf16>(x);
}

// the admit bits of tokens v..v+VE-1 (all < V) in the low bits
template <int VE>
__device__ inline unsigned admit_bits(const unsigned char* row, int v) {
    const unsigned lo = row[v >> 3], hi = row[(v + VE - 1) >> 3];
    return (lo | hi << 8) >> (v & 7);
}

template <class I, bool OF, bool MASK>
__device__ inline void put_vec(char* out, long long n, u32x4 w, unsigned bits) {
    if constexpr (I::ES == 4) {
        if constexpr (MASK) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = (bits >> j) & 1 ? w[j] : 0xff800000u;
        }
        *reinterpret_cast<u32x4*>(out + 4 * n) = w;
    } else if constexpr (!OF) {
        if constexpr (MASK) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const unsigned lo = (bits >> (2 * j)) & 1 ? w[j] & 0xffffu : 0xff80u;
                const unsigned hi = (bits >> (2 * j + 1)) & 1 ? w[j] & 0xffff0000u : 0xff800000u;
                w[j] = lo | hi;
            }
        }
        *reinterpret_cast<u32x4*>(out + 2 * n) = w;
    } else {
        u32x4 a, b;
        a.x = w.x << 16; a.y = w.x & 0xffff0000u; a.z = w.y << 16; a.w = w.y & 0xffff0000u;
        b.x = w.z << 16; b.y = w.z & 0xffff0000u; b.z = w.w << 16; b.w = w.w & 0xffff0000u;
        if constexpr (MASK) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a[j] = (bits >> j) & 1 ? a[j] : 0xff800000u;
                b[j] = (bits >> (4 + j)) & 1 ? b[j] : 0xff800000u;
            }
        }
        *reinterpret_cast<u32x4*>(out + 4 * n) = a;
        *reinterpret_cast<u32x4*>(out + 4 * n + 16) = b;
    }
}

template <class I, bool OF>
__global__ __launch_bounds__(NTJ) void adjust_kernel(AdjustParams A) {
    __shared__ unsigned cnt[SEG_MAX], own[SEG_MAX];
    __shared__ int dup;
    const int t = static_cast<int>(threadIdx.x);
    const int b = static_cast<int>(blockIdx.x) / A.nseg, s = static_cast<int>(blockIdx.x) % A.nseg;
    const int v0 = s * A.seg, v1 = min(A.V, v0 + A.seg), len = v1 - v0;
    int rows = A.R;                                        // rows in use
    if (A.draft_len) {
        const int kb = A.draft_len[b];
        if (kb < 0 || kb > A.k) return;
        rows = A.R - A.k + kb;
    }
    const int n = A.history ? A.hist_len[b] : 0, p = A.history && A.prompt_len ? A.prompt_len[b] : 0;
    const float rep = A.rep ? A.rep[b] : 1.0f, freq = A.freq ? A.freq[b] : 0.0f, pres = A.pres ? A.pres[b] : 0.0f;
    const bool bad = n < 0 || n > A.H || p < 0 || p > n || !(rep > 0.0f && rep <= F32_MAX) ||
                     !(fabsf(freq) <= F32_MAX) || !(fabsf(pres) <= F32_MAX);
    const bool counts = (A.rep || A.freq || A.pres) && !bad;
    const bool any = (counts && (n > 0 || A.k > 0)) || A.nb > 0;
    if (any) {
        for (int v = t; v < len; v += NTJ) { cnt[v] = 0; own[v] = NOBIAS; }
        if (t == 0) dup = 0;
        __syncthreads();
        if (counts) {
            const int* h = A.history + static_cast<long long>(b) * A.H;
            for (int j = t; j < n; j += NTJ) {
                const unsigned v = static_cast<unsigned>(h[j]) - static_cast<unsigned>(v0);
                if (v < static_cast<unsigned>(len)) {
                    if (j < p) atomicOr(&cnt[v], SEEN);
                    else atomicAdd(&cnt[v], 1u);
                }
            }
        }
        // the first entry of a biased token owns it; further ones are rare
        for (int j = t; j < A.nb; j += NTJ) {
            const unsigned v = static_cast<unsigned>(A.bias_tok[static_cast<long long>(b) * A.nb + j]) -
                               static_cast<unsigned>(v0);
            if (v < static_cast<unsigned>(len) && atomicMin(&own[v], static_cast<unsigned>(j)) != NOBIAS) dup = 1;
        }
    }
    // stream
    for (int i = 0; i < rows; ++i) {
        const long long row = static_cast<long long>(b) * A.R + i, n0 = row * A.V;
        int ar = A.admit ? (A.admit_row ? A.admit_row[row] : static_cast<int>(row)) : -1;
        if (bad || ar < -1 || (A.admit && ar >= A.n_admit)) {
            for (int v = v0 + t; v < v1; v += NTJ) put_one<I, OF>(A.out, n0 + v, NAN);
            continue;
        }
        const unsigned char* mask =
            ar >= 0 ? reinterpret_cast<const unsigned char*>(A.admit + static_cast<long long>(ar) * A.W) : nullptr;
        if (A.inplace && !mask) continue;                  // nothing to change
        const int head = A.vec ? min(len, static_cast<int>(-(n0 + v0) & (I::VE - 1))) : len;
        const int nvec = (len - head) / I::VE, tail = len - head - nvec * I::VE;
        for (int q = t; q < nvec; q += NTJ) {
            const int v = v0 + head + q * I::VE;
            const u32x4 w = *reinterpret_cast<const u32x4*>(A.in + (n0 + v) * I::ES);
            if (mask) put_vec<I, OF, true>(A.out, n0 + v, w, admit_bits<I::VE>(mask, v));
            else put_vec<I, OF, false>(A.out, n0 + v, w, 0);
        }
        for (int q = t; q < head + tail; q += NTJ) {
            const int v = q < head ? v0 + q : v1 - tail + (q - head);
            const bool ok = !mask || (mask[v >> 3] >> (v & 7) & 1);
            put_one<I, OF>(A.out, n0 + v, ok ? I::one(A.in, n0 + v) : -INFINITY);
        }
    }
    if (!any || bad) return;
    __builtin_amdgcn_s_waitcnt(0);                         // the stores above land before those below
    __syncthreads();
    // the tokens with a count or a bias
    const int* tok = A.tokens + static_cast<long long>(b) * A.k;
    if (counts) {
        // drafts without a count of their own yet: mark them so that they are visited
        for (int j = t; j < min(A.k, rows - 1); j += NTJ) {
            const unsigned v = static_cast<unsigned>(tok[j]) - static_cast<unsigned>(v0);
            if (v < static_cast<unsigned>(len)) atomicOr(&cnt[v], 0x40000000u);
        }
        __syncthreads();
    }
    for (int v = t; v < len; v += NTJ) {
        const unsigned c = cnt[v], o = own[v];
        if (c == 0 && o == NOBIAS) continue;
        const unsigned long long bo = static_cast<unsigned long long>(b) * A.nb;
        float bias = 0.0f;
        if (o != NOBIAS) {
            bias = A.bias_val[bo + o];
            if (dup)
                for (int j = static_cast<int>(o) + 1; j < A.nb; ++j)
                    if (A.bias_tok[bo + j] == v0 + v) bias += A.bias_val[bo + j];
        }
        unsigned num = c & 0x3fffffffu;
        bool seen = (c & SEEN) != 0 || num > 0;
        for (int i = 0; i < rows; ++i) {
            if (i > 0 && counts && tok[i - 1] == v0 + v) { ++num; seen = true; }
            const long long row = static_cast<long long>(b) * A.R + i, at = row * A.V + v0 + v;
            const int ar = A.admit ? (A.admit_row ? A.admit_row[row] : static_cast<int>(row)) : -1;
            if (ar < -1 || (A.admit && ar >= A.n_admit)) continue;
            if (ar >= 0 && !(A.admit[static_cast<long long>(ar) * A.W + ((v0 + v) >> 5)] >> ((v0 + v) & 31) & 1))
                continue;
            float x = I::one(A.in, at);
            if (seen) x = x > 0.0f ? x / rep : x * rep;
            if (num > 0) x = x - freq * static_cast<float>(num) - pres;
            if (o != NOBIAS) x += bias;
            put_one<I, OF>(A.out, at, x);
        }
    }
}

// ------------------------------------------------------------------ host side

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return code;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int launched() {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? SPEC_OK : fail(SPEC_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
}

constexpr int64_t MAX_STRIDE = int64_t(1) << 40;           // elements; 3 strides times their extents stay below 2^63

bool strides_ok(const int64_t* s, int es, long long (&bytes)[3]) {
    for (int j = 0; j < 3; ++j) {
        if (s[j] < 0 || s[j] > MAX_STRIDE || s[j] * es % 16 != 0) return false;
        bytes[j] = s[j] * es;
    }
    return true;
}

// The checks that the cache write and the attention share.
int check_cache(int dtype, int32_t B, int32_t R, int32_t max_R, int32_t Hkv, int32_t D, const void* k_cache,
                const int64_t* ks, const void* v_cache, const int64_t* vs, int cache_dtype, int64_t pages,
                int32_t page_size, const int32_t* table, int32_t max_pages, const int32_t* kv_len,
                const int32_t* draft_len, const float* k_scale, const float* v_scale, Cache& C) {
    if (dtype != SPEC_DTYPE_BF16 && dtype != SPEC_DTYPE_F16)
        return fail(SPEC_ERR_DTYPE, "dtype %d is not SPEC_DTYPE_BF16 or SPEC_DTYPE_F16", dtype);
    if (cache_dtype != dtype && cache_dtype != SPEC_DTYPE_E4M3)
        return fail(SPEC_ERR_DTYPE, "the cache's dtype %d is neither dtype %d nor SPEC_DTYPE_E4M3", cache_dtype, dtype);
    if (B < 1 || B > (1 << 21) || R < 1 || R > max_R || Hkv < 1 || Hkv > 1024 || (D != 64 && D != 128 && D != 256))
        return fail(SPEC_ERR_SHAPE, "need 1 <= B <= 2^21, 1 <= R <= %d, 1 <= Hkv <= 1024, D 64, 128 or 256 "
                    "(got B=%d R=%d Hkv=%d D=%d)", max_R, B, R, Hkv, D);
    if (pages < 1 || pages > (int64_t(1) << 31) || max_pages < 1 || page_size < 1 || page_size > SPEC_MAX_PAGE ||
        (page_size & (page_size - 1)) != 0)
        return fail(SPEC_ERR_SHAPE, "need pages >= 1, max_pages >= 1 and a page_size that is a power of two up to %d "
                    "(got %lld, %d, %d)", SPEC_MAX_PAGE, static_cast<long long>(pages), max_pages, page_size);
    if (static_cast<int64_t>(max_pages) * page_size > (int64_t(1) << 30))
        return fail(SPEC_ERR_SHAPE, "max_pages * page_size exceeds 2^30 positions");
    const bool e4m3 = cache_dtype == SPEC_DTYPE_E4M3;
    if (!k_cache || !v_cache || !ks || !vs || !table || !kv_len)
        return fail(SPEC_ERR_NULL, "a cache, stride, page_table or kv_len pointer is NULL");
    if (e4m3 != (k_scale != nullptr) || e4m3 != (v_scale != nullptr))
        return fail(SPEC_ERR_NULL, "k_scale and v_scale are required for an e4m3 cache and must be NULL otherwise");
    const int es = e4m3 ? 1 : 2;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !strides_ok(ks, es, C.ks) || !strides_ok(vs, es, C.vs))
        return fail(SPEC_ERR_ALIGN, "cache pointers must be 16-byte aligned and their strides multiples of 16 bytes");
    if (!aligned(table, 4) || !aligned(kv_len, 4) || (draft_len && !aligned(draft_len, 4)) ||
        (k_scale && (!aligned(k_scale, 4) || !aligned(v_scale, 4))))
        return fail(SPEC_ERR_ALIGN, "a tensor pointer is not aligned to its element size");
    C.k = const_cast<char*>(static_cast<const char*>(k_cache));
    C.v = const_cast<char*>(static_cast<const char*>(v_cache));
    C.table = table; C.kv_len = kv_len; C.draft_len = draft_len;
    C.k_scale = k_scale; C.v_scale = v_scale;
    C.pages = pages; C.max_pages = max_pages;
    C.shift = __builtin_ctz(static_cast<unsigned>(page_size));
    C.B = B; C.R = R; C.Hkv = Hkv;
    return SPEC_OK;
}

template <class T, int D>
void launch_attn_d(const AttnParams& A, bool e4m3, unsigned grid, hipStream_t s) {
    if (e4m3) hipLaunchKernelGGL((attn_kernel<T, D, true>), dim3(grid), dim3(NTQ), 0, s, A);
    else hipLaunchKernelGGL((attn_kernel<T, D, false>), dim3(grid), dim3(NTQ), 0, s, A);
}

template <class T>
void launch_attn(const AttnParams& A, int D, bool e4m3, unsigned grid, hipStream_t s) {
    if (D == 64) launch_attn_d<T, 64>(A, e4m3, grid, s);
    else if (D == 128) launch_attn_d<T, 128>(A, e4m3, grid, s);
    else launch_attn_d<T, 256>(A, e4m3, grid, s);
}

}  // namespace

extern "C" {

int spec_kv_append(const void* k, const int64_t* k_stride, const void* v, const int64_t* v_stride, int dtype,
                   int32_t B, int32_t R, int32_t Hkv, int32_t D, void* k_cache, const int64_t* k_cache_stride,
                   void* v_cache, const int64_t* v_cache_stride, int cache_dtype, int64_t pages,
                   int32_t page_size, const int32_t* page_table, int32_t max_pages, const int32_t* kv_len,
                   const int32_t* draft_len, const float* k_scale, const float* v_scale, void* stream) {
    AppendParams A{};
    const int rc = check_cache(dtype, B, R, 1 << 20, Hkv, D, k_cache, k_cache_stride, v_cache, v_cache_stride,
                               cache_dtype, pages, page_size, page_table, max_pages, kv_len, draft_len, k_scale,
                               v_scale, A.c);
    if (rc != SPEC_OK) return rc;
    if (!k || !v || !k_stride || !v_stride) return fail(SPEC_ERR_NULL, "k, v or one of their strides is NULL");
    if (!aligned(k, 16) || !aligned(v, 16) || !strides_ok(k_stride, 2, A.xk) || !strides_ok(v_stride, 2, A.xv))
        return fail(SPEC_ERR_ALIGN, "k and v must be 16-byte aligned and their strides multiples of 8 elements");
    const bool e4m3 = cache_dtype == SPEC_DTYPE_E4M3;
    A.k = static_cast<const char*>(k);
    A.v = static_cast<const char*>(v);
    const int cph = D * (e4m3 ? 1 : 2) / 16;
    A.cph_shift = static_cast<unsigned>(__builtin_ctz(static_cast<unsigned>(cph)));
    A.cpt = static_cast<unsigned>(Hkv * cph);
    A.chunks = static_cast<long long>(B) * R * A.cpt;
    const long long want = (A.chunks + NTA - 1) / NTA;
    const unsigned grid = static_cast<unsigned>(want < (1 << 20) ? want : (1 << 20));
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == SPEC_DTYPE_BF16) {
        if (e4m3) hipLaunchKernelGGL((append_kernel<Bf16, true>), dim3(grid), dim3(NTA), 0, s, A);
        else hipLaunchKernelGGL((append_kernel<Bf16, false>), dim3(grid), dim3(NTA), 0, s, A);
    } else {
        if (e4m3) hipLaunchKernelGGL((append_kernel<F16, true>), dim3(grid), dim3(NTA), 0, s, A);
        else hipLaunchKernelGGL((append_kernel<F16, false>), dim3(grid), dim3(NTA), 0, s, A);
    }
    return launched();
}

size_t spec_attention_workspace_size(int32_t B, int32_t R, int32_t Hq, int32_t Hkv, int32_t D, int cache_dtype,
                                     int32_t page_size, int32_t max_pages) {
    if (B < 1 || B > (1 << 21) || R < 1 || R > SPEC_MAX_K + 1 || Hkv < 1 || Hkv > 1024 || Hq < Hkv || Hq > 1024 ||
        Hq % Hkv != 0 || (D != 64 && D != 128 && D != 256) || page_size < 1 || page_size > SPEC_MAX_PAGE ||
        max_pages < 1 || (cache_dtype != SPEC_DTYPE_BF16 && cache_dtype != SPEC_DTYPE_F16 &&
                          cache_dtype != SPEC_DTYPE_E4M3))
        return 0;
    return 256;
}

int spec_attention(const void* q, const int64_t* q_stride, int dtype, int32_t B, int32_t R, int32_t Hq, int32_t Hkv,
                   int32_t D, const void* k_cache, const int64_t* k_cache_stride, const void* v_cache,
                   const int64_t* v_cache_stride, int cache_dtype, int64_t pages, int32_t page_size,
                   const int32_t* page_table, int32_t max_pages, const int32_t* kv_len, const int32_t* draft_len,
                   float scale, float softcap, int32_t window, const float* slopes, const float* k_scale,
                   const float* v_scale, void* out, void* workspace, size_t workspace_bytes, void* stream) {
    AttnParams A{};
    const int rc = check_cache(dtype, B, R, SPEC_MAX_K + 1, Hkv, D, k_cache, k_cache_stride, v_cache, v_cache_stride,
                               cache_dtype, pages, page_size, page_table, max_pages, kv_len, draft_len, k_scale,
                               v_scale, A.c);
    if (rc != SPEC_OK) return rc;
    if (Hq < Hkv || Hq > 1024 || Hq % Hkv != 0)
        return fail(SPEC_ERR_SHAPE, "Hq must be a multiple of Hkv up to 1024 (got Hq=%d Hkv=%d)", Hq, Hkv);
    if (!(fabsf(scale) <= F32_MAX) || !(softcap >= 0.0f && softcap <= F32_MAX) || window < 0)
        return fail(SPEC_ERR_VALUE, "scale must be finite, softcap finite and >= 0, window >= 0 (got %g, %g, %d)",
                    static_cast<double>(scale), static_cast<double>(softcap), window);
    if (!q || !q_stride || !out) return fail(SPEC_ERR_NULL, "q, its strides or out is NULL");
    if (!aligned(q, 16) || !strides_ok(q_stride, 2, A.qs) || !aligned(out, 16))
        return fail(SPEC_ERR_ALIGN, "q and out must be 16-byte aligned and q's strides multiples of 8 elements");
    if (slopes && !aligned(slopes, 4)) return fail(SPEC_ERR_ALIGN, "slopes is not aligned to its element size");
    const size_t need = spec_attention_workspace_size(B, R, Hq, Hkv, D, cache_dtype, page_size, max_pages);
    if (!workspace || workspace_bytes < need)
        return fail(SPEC_ERR_WORKSPACE, "workspace needs %zu bytes (got %zu%s)", need, workspace_bytes,
                    workspace ? "" : ", NULL");
    if (!aligned(workspace, 256)) return fail(SPEC_ERR_ALIGN, "workspace must be 256-byte aligned");
    A.q = static_cast<const char*>(q);
    A.slopes = slopes;
    A.out = static_cast<char*>(out);
    A.scale = scale; A.softcap = softcap; A.window = window;
    A.Hq = Hq; A.G = Hq / Hkv;
    const long long grid = static_cast<long long>(B) * R * Hq;
    if (grid > (1ll << 31) - 1) return fail(SPEC_ERR_SHAPE, "B * R * Hq exceeds 2^31 - 1");
    const bool e4m3 = cache_dtype == SPEC_DTYPE_E4M3;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == SPEC_DTYPE_BF16) launch_attn<Bf16>(A, D, e4m3, static_cast<unsigned>(grid), s);
    else launch_attn<F16>(A, D, e4m3, static_cast<unsigned>(grid), s);
    return launched();
}

int spec_adjust(const void* logits, int32_t B, int32_t R, int32_t V, int dtype, const int32_t* draft_tokens, int32_t k,
                const int32_t* draft_len, const int32_t* history, int32_t H, const int32_t* hist_len,
                const int32_t* prompt_len, const float* repetition, const float* frequency, const float* presence,
                const int32_t* bias_tokens, const float* bias_values, int32_t n_bias, const uint32_t* admit,
                int32_t n_admit, const int32_t* admit_row, void* out, int out_dtype, void* stream) {
    if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16)
        return fail(SPEC_ERR_DTYPE, "dtype %d is not SPEC_DTYPE_F32 or SPEC_DTYPE_BF16", dtype);
    if (out_dtype != SPEC_DTYPE_F32 && out_dtype != dtype)
        return fail(SPEC_ERR_DTYPE, "out_dtype %d is neither SPEC_DTYPE_F32 nor dtype %d", out_dtype, dtype);
    if (B < 1 || B > (1 << 21) || k < 0 || k > SPEC_MAX_K || R < 1 || (R != k + 1 && R != k) || V < 1 || V > (1 << 29))
        return fail(SPEC_ERR_SHAPE, "need 1 <= B <= 2^21, 0 <= k <= %d, R = k or k + 1 and >= 1, 1 <= V <= 2^29 "
                    "(got B=%d k=%d R=%d V=%d)", SPEC_MAX_K, B, k, R, V);
    if (static_cast<unsigned long long>(B) * R * static_cast<unsigned long long>(V) > (1ull << 46))
        return fail(SPEC_ERR_SHAPE, "B*R*V is too large");
    if (H < 0 || H > (1 << 30) - 1 || n_bias < 0 || n_bias > 65536 || n_admit < 0)
        return fail(SPEC_ERR_SHAPE, "need 0 <= H < 2^30, 0 <= n_bias <= 65536, n_admit >= 0 (got %d, %d, %d)", H,
                    n_bias, n_admit);
    if (!logits || !out) return fail(SPEC_ERR_NULL, "logits or out is NULL");
    if (k > 0 && !draft_tokens) return fail(SPEC_ERR_NULL, "draft_tokens is NULL");
    if (H > 0 && (!history || !hist_len)) return fail(SPEC_ERR_NULL, "history and hist_len are required when H > 0");
    if (n_bias > 0 && (!bias_tokens || !bias_values))
        return fail(SPEC_ERR_NULL, "bias_tokens and bias_values are required when n_bias > 0");
    if ((admit != nullptr) != (n_admit > 0) || (admit_row && !admit))
        return fail(SPEC_ERR_NULL, "admit and n_admit > 0 go together, and admit_row needs them");
    if (admit && !admit_row && static_cast<long long>(n_admit) != static_cast<long long>(B) * R)
        return fail(SPEC_ERR_SHAPE, "admit without admit_row must hold B * R rows (got %d)", n_admit);
    const size_t es = dtype == SPEC_DTYPE_F32 ? 4 : 2, eo = out_dtype == SPEC_DTYPE_F32 ? 4 : 2;
    if (!aligned(logits, es) || !aligned(out, eo))
        return fail(SPEC_ERR_ALIGN, "logits or out is not aligned to its element size");
    const void* words[] = {draft_tokens, draft_len, history, hist_len, prompt_len, repetition, frequency, presence,
                           bias_tokens, bias_values, admit, admit_row};
    for (const void* p : words)
        if (p && !aligned(p, 4)) return fail(SPEC_ERR_ALIGN, "a tensor pointer is not aligned to its element size");
    if (out == logits && es != eo) return fail(SPEC_ERR_DTYPE, "out may be logits only with the same dtype");
    AdjustParams A{};
    A.in = static_cast<const char*>(logits);
    A.out = static_cast<char*>(out);
    A.tokens = draft_tokens; A.draft_len = draft_len;
    A.history = H > 0 ? history : nullptr; A.hist_len = hist_len; A.prompt_len = prompt_len;
    A.rep = repetition; A.freq = frequency; A.pres = presence;
    A.bias_tok = bias_tokens; A.bias_val = bias_values;
    A.admit = admit; A.admit_row = admit_row;
    A.B = B; A.R = R; A.V = V; A.k = k; A.H = H; A.nb = n_bias; A.n_admit = n_admit;
    A.W = (V + 31) / 32;
    A.vec = aligned(logits, 16) && aligned(out, 16);
    A.inplace = out == logits;
    A.seg = 4096;
    A.nseg = (V + A.seg - 1) / A.seg;
    const long long grid = static_cast<long long>(B) * A.nseg;
    if (grid > (1ll << 31) - 1) return fail(SPEC_ERR_SHAPE, "B * V is too large");
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == SPEC_DTYPE_F32)
        hipLaunchKernelGGL((adjust_kernel<InF32, false>), dim3(static_cast<unsigned>(grid)), dim3(NTJ), 0, s, A);
    else if (out_dtype == SPEC_DTYPE_BF16)
        hipLaunchKernelGGL((adjust_kernel<InBf16, false>), dim3(static_cast<unsigned>(grid)), dim3(NTJ), 0, s, A);
    else
        hipLaunchKernelGGL((adjust_kernel<InBf16, true>), dim3(static_cast<unsigned>(grid)), dim3(NTJ), 0, s, A);
    return launched();
}

const char* spec_forward_last_error(void) { return g_err; }

}  // extern "C"
