// spec_forward.hip -- the operators around a verify step's model for MI355X (gfx950):
// the paged KV cache's write and attention, and the adjustment of the logits.
//
// What is computed is stated in include/spec_forward.h.
//
// Every sum of floats is taken in a fixed order (atomics only count integers), so results
// are bitwise reproducible.

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
    static constexpr bool IS_BF16 = true;
    static constexpr unsigned EXP = 0x7f80u;               // exponent bits: all set = not finite
    // log2 of the weight of a running maximum when it is set, and of the largest weight
    static constexpr float TOP = 0.0f, LAZY = 8.0f;
    __device__ static inline float lo(unsigned w) { return bits_f32(w << 16); }
    __device__ static inline float hi(unsigned w) { return bits_f32(w & 0xffff0000u); }
};

struct F16 {
    using type = _Float16;
    static constexpr bool IS_BF16 = false;
    static constexpr unsigned EXP = 0x7c00u;
    // (near the top of the type's range, so that small weights keep their bits: the smallest
    // normal one is 2^-21 of the maximum's)
    static constexpr float TOP = 7.0f, LAZY = 15.0f;
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
    // (a draft_len of INT_MAX wraps to a negative n: also out of range)
    const int n = C.draft_len ? static_cast<int>(static_cast<unsigned>(C.draft_len[b]) + 1u) : C.R;
    const long long cap = static_cast<long long>(C.max_pages) << C.shift;
    return kv < 0 || n < 1 || n > C.R || static_cast<long long>(kv) + n > cap ? 0 : n;
}

__device__ inline bool page_ok(const Cache& C, int page) { return page >= 0 && page < C.pages; }

// ------------------------------------------------------------------ cache write
//
// Bound by memory: every new key and value is read and written once. One
// thread moves 16 bytes of the cache for keys and for values, so that a wave's
// stores cover whole head rows (D * 2 bytes, 256 at D = 128, contiguous in
// either cache order), and finds its place itself: two dependent loads (length,
// page id), served by L2 for all but the first threads of a token. 134 MB of prompts in
// 23 us, 5.8 TB/s read + written (a large copy: 5.1, partly from the memory-side cache
// here); 64 rows of 6 tokens into an 8-bit cache 4.7 us, one token 2.0 us (one launch).

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
//
// For one batch row and cache head the R * G query rows (R tokens, G query heads that
// share the cache head) all read the same keys and values, so the cache crosses HBM
// once while every row is computed from it on the matrix cores; the kernel is bound by
// that stream (at R * G = 24, D = 128 the products need less than a tenth of their
// peak while HBM is saturated).
//
// With X = K Q^T as 16 x 16 tiles (keys are the MFMA's A operand), lane l holds scores
// of ONE query row (l % 16) for keys 4 (l / 16) + 0..3 of the tile: the softmax is
// arithmetic within the lane. Two such tiles (32 keys) give, in the same registers,
// the B operand of O^T = V^T P^T, if the contraction takes the keys in the order
// {4g..4g+3, 16+4g..16+4g+3} for lane group g; the A operand, columns of V in that
// order, comes from LDS by transposing reads (ds_read_b64_tr_b16, or _tr_b8 for e4m3).
// No score or weight ever crosses lanes. The running maximum of a row moves only when
// a score exceeds it by 2^8 in weight (checked by a vote), so the two
// exchanges and the rescaling that go with a new maximum are rare; weights are then
// at most 2^8 (float16: 2^15, from 2^7 on), and sums and accumulators are float32.
//
// Each of a workgroup's four waves walks its own tiles of 32 keys with its own
// accumulators, through its own part of LDS, and never waits for another wave: keys
// and values go from memory straight into LDS (16 bytes per lane, the lane fetching
// the chunk that belongs at its place, see `chunk`), the next tile's keys in flight
// during the softmax and the product with V, its values during the product with K.
// The waves' results are joined through LDS at the end.
//
// Split over the length: the batch's sequences are cut into units of 128 keys, and W
// workgroups per cache head (together one resident round) take equal, contiguous
// ranges of the units, whatever the lengths are; the ranges are found on the device
// from kv_len. A sequence inside one range is finished there. Of a sequence that
// crosses ranges each workgroup leaves its unnormalised result and statistics in the
// workspace (at most two such pieces per workgroup: the first and the last of its
// range), and join_kernel merges them.
//
// Measured (this kernel alone, MI355X; a large read reaches 5.97 TB/s): 64 rows of 6 tokens, 8
// cache heads x 4, D = 128, bfloat16, 812 MB of cache: 149 us, 5.4 TB/s. One row of 5 tokens,
// 8 x 8, 8-bit cache, 134 to 268 MB: 47 to 57 us. 16 rows of 4, 4 x 2, D = 256, window, cap,
// 269 MB: 54 us, 5.0 TB/s. 32 rows of one token, 32 x 1, D = 64, 403 MB: 67 us, 6.0 TB/s. One
// row of one token over 1000 keys: 9 us, a chain of dependent loads.

constexpr int NTQ = 256;
constexpr int NWQ = NTQ / 64;
constexpr int TT = 32;                                     // keys of a wave's tile
constexpr int TU = TT * NWQ;                               // keys of a unit
constexpr int CUS = 256;
constexpr int NT_LOAD = 2;                                 // cache policy: non-temporal (read once)
constexpr float CAP_FINE = 256.0f;                         // softcaps from here on take the more exact tanh

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef __attribute__((address_space(3))) i16x4* lds_i16x4;
typedef __attribute__((address_space(3))) i32x2* lds_i32x2;
typedef __attribute__((address_space(1))) const void* glb_ptr;

struct AttnParams {
    Cache c;
    const char* q;
    long long qs[3];           // bytes between batch rows, tokens, heads
    const float* slopes;       // [Hq] or null
    char* out;                 // [B, R, Hq, D]
    float* ws;                 // W RangeRec, then per (w, head, block): two slots of M16 * (D + 2) floats
    long long slots_at;        // floats before the slots
    float scale, softcap;
    int window, Hq, G, D;
    int M;                     // R * G query rows per cache head
    int MB;                    // row blocks of M16 rows
    int M16;                   // query rows of a workgroup
    int W;                     // workgroups per cache head and row block, at most
    int one;                   // ... with one per CU (no more than W)
    int direct;                // join_kernel goes by batch row (else by border between ranges)
    int slices;                // join_kernel: threads that share a sequence's pieces
};

// a batch row's keys: positions [lo, hi) are seen by some token in use
struct Seq {
    int kv, n;                 // first new position, tokens in use (0: bad lengths)
    int lo, hi, base;          // base: lo rounded down to a tile of any shape
    int units;
};

__device__ inline Seq seq_from(const AttnParams& A, int kv, int n) {
    Seq s;
    s.kv = kv;
    s.n = n;
    if (n == 0) { s.lo = s.hi = s.base = 0; s.units = 1; return s; }
    s.lo = A.window > 0 ? max(0, kv + 1 - A.window) : 0;
    s.hi = kv + n;
    s.base = s.lo & ~(2 * TT - 1);                         // (the larger tile)
    s.units = (s.hi - s.base + TU - 1) / TU;
    return s;
}

__device__ inline Seq seq_of(const AttnParams& A, int b) {
    int kv;
    const int n = seq_rows(A.c, b, kv);
    return seq_from(A, kv, n);
}

template <int N>
struct Int {
    static constexpr int value = N;
};

struct Plan {
    unsigned wave[NWQ];
    long long pre;
    int b, kv, n;
};

__device__ inline unsigned wave_inclusive(unsigned v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const unsigned u = __shfl_up(v, d, 64);
        if (lane >= d) v += u;
    }
    return v;
}

// Inclusive scan over the workgroup of v; total is its sum (256 rows of at most 2^23 units
// stay below 2^32).
__device__ inline unsigned block_inclusive(Plan& P, unsigned v, unsigned& total) {
    const int w = threadIdx.x >> 6;
    const unsigned x = wave_inclusive(v);
    __syncthreads();                                       // the last scan's sums have been read
    if ((threadIdx.x & 63) == 63) P.wave[w] = x;
    __syncthreads();
    unsigned before = 0;
    total = 0;
#pragma unroll
    for (int j = 0; j < NWQ; ++j) {
        if (j < w) before += P.wave[j];
        total += P.wave[j];
    }
    return before + x;
}

// x, hidden from the compiler: what is computed from it in a rare branch, or once per sequence,
// is then computed there, not ahead of the loops and held in a register (or spilled) across
// them. It saves the attention kernels 20 to 28 registers; an 8-bit cache with R * G = 40
// spilled without it (201 MB of keys and values: 67 us, 58.5 with it).
__device__ inline int fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

__device__ inline long long fresh(long long x) {
    asm volatile("" : "+v"(x));
    return x;
}

// The batch's units, cut into `ranges` contiguous ranges whose sizes differ by at most one.
struct Ranges {
    long long size, more;                                  // the first `more` ranges hold size + 1
    int ranges;

    __device__ long long start(int w) const { return size * w + (w < more ? w : more); }
    __device__ int holding(long long u) const {
        const long long n = fresh(size), c = more * (n + 1);
        return static_cast<int>(u < c ? u / (n + 1) : more + (u - c) / n);
    }
};

// What join_kernel needs of a batch row (of the row in which range w starts): the first and
// last range that hold units of it. Each of them has a piece of it in its slot 0, the
// first range, where the row begins, in its slot 1.
struct RangeRec {
    int b, n_tok, wa, wb;
};

// x, the same in every lane, as a scalar
__device__ inline int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ inline long long uniform(long long x) {
    const unsigned lo = static_cast<unsigned>(uniform(static_cast<int>(x)));
    const int hi = uniform(static_cast<int>(x >> 32));
    return static_cast<long long>(static_cast<unsigned long long>(static_cast<unsigned>(hi)) << 32 | lo);
}

// At most A.W ranges, but one workgroup per CU (A.one) where that leaves no more than four
// units to each, in sequences of more than 16 on average: fewer pieces then save more than a
// second workgroup's loads gain (one row of 5 tokens, 8 x 4, D = 128: 8192 keys 20.9 us
// against 25.6, 16384 keys 25.8 against 28.9). With shorter sequences the longer ranges take
// parts of several, one after the other (4 rows of 1000 to 2000 keys: 25.1 us against 22.9;
// 100 rows of 4 tokens, 150 keys: 40 against 30).
__device__ inline Ranges cut(const AttnParams& A, long long total) {
    Ranges r;
    const int most = total <= 4ll * A.one && total > 16ll * A.c.B ? A.one : A.W;
    r.ranges = total < most ? static_cast<int>(total) : most;
    if (total <= 0x7fffffff) {
        r.size = static_cast<int>(total) / r.ranges;
    } else {
        r.size = total / r.ranges;
    }
    r.more = total - r.size * r.ranges;
    return r;
}

// Where range w starts: batch row (with its first new position and its tokens in use) and
// the units before it. The same in every lane. Up to 64 batch rows each wave finds it by
// itself; more are scanned by the workgroup, 256 at a time.
__device__ inline Ranges locate(const AttnParams& A, Plan& P, int w, int& b, int& kv, int& n, long long& pre) {
    const int t = static_cast<int>(threadIdx.x), B = A.c.B;
    if (B <= 64) {
        const int lane = t & 63;
        int lkv = 0, ln = 0;
        unsigned u = 0;
        if (lane < B) {
            ln = seq_rows(A.c, lane, lkv);
            u = static_cast<unsigned>(seq_from(A, lkv, ln).units);
        }
        const unsigned inc = wave_inclusive(u);
        const Ranges r = cut(A, uniform(static_cast<int>(__shfl(inc, 63, 64))));
        const unsigned target = static_cast<unsigned>(r.start(w));
        b = w < r.ranges ? uniform(__ffsll(__ballot(inc > target)) - 1) : 0;
        kv = uniform(__shfl(lkv, b, 64));
        n = uniform(__shfl(ln, b, 64));
        pre = uniform(static_cast<int>(__shfl(inc - u, b, 64)));
        return r;
    }
    Seq s;
    s.kv = s.n = s.units = 0;
    if (t < B) s = seq_of(A, t);
    unsigned chunk, u = static_cast<unsigned>(s.units);
    long long inc = block_inclusive(P, u, chunk), total = chunk;
    for (int b0 = NTQ; b0 < B; b0 += NTQ) {
        unsigned sum;
        block_inclusive(P, b0 + t < B ? static_cast<unsigned>(seq_of(A, b0 + t).units) : 0u, sum);
        total += sum;
    }
    const Ranges r = cut(A, uniform(total));
    if (w >= r.ranges) return r;
    const long long target = r.start(w);
    long long run = 0;
    for (int b0 = 0;;) {
        if (target >= inc - u && target < inc) { P.b = b0 + t; P.kv = s.kv; P.n = s.n; P.pre = inc - u; }
        run += chunk;
        b0 += NTQ;
        if (run > target) break;                           // the same in every lane
        s.units = 0;
        if (b0 + t < B) s = seq_of(A, b0 + t);
        u = static_cast<unsigned>(s.units);
        inc = run + block_inclusive(P, u, chunk);
    }
    __syncthreads();
    b = uniform(P.b);
    kv = uniform(P.kv);
    n = uniform(P.n);
    pre = uniform(P.pre);
    return r;
}

// Loads into LDS are waited for by hand (wait_loads): the compiler would have each LDS
// read wait for every load in flight, since they go to one array. It does so unless it
// cannot tell that a load's destination is that array.
__device__ inline lds_ptr untraced(lds_ptr p) {
    asm volatile("" : "+r"(p));
    return p;
}

// s_waitcnt: at most `vm` loads in flight / no LDS read in flight; nothing moves across
template <int VM>
__device__ inline void wait_loads() {
    static_assert(VM <= 63, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (7 << 4) | (15 << 8));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
__device__ inline void wait_lds() {
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// 2^(x - m) for x whose maximum m is (within 2^8 in weight): the difference of the rounded
// scores. Fused with the multiplication that gave x it would hold x's rounding error,
// which for scores beyond 2^30 is a power of two that overflows.
__device__ inline float exp2_diff(float x, float m) {
#pragma clang fp contract(off)
    return __builtin_amdgcn_exp2f(x - m);
}

template <class T>
__device__ inline f32x4 mfma(i32x4 a, i32x4 b, f32x4 c) {
    typedef typename T::type v8 __attribute__((ext_vector_type(8)));
    if constexpr (T::IS_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
}

// eight e4m3 codes to eight values of T (exact: T has more exponents and bits)
template <class T>
__device__ inline i32x4 widen8(i32x2 w) {
    typedef typename T::type v2 __attribute__((ext_vector_type(2)));
    i32x4 o;
    if constexpr (T::IS_BF16) {
        o.x = __builtin_bit_cast(int, (v2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.x, 1.0f, false));
        o.y = __builtin_bit_cast(int, (v2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.x, 1.0f, true));
        o.z = __builtin_bit_cast(int, (v2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.y, 1.0f, false));
        o.w = __builtin_bit_cast(int, (v2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.y, 1.0f, true));
    } else {
        o.x = __builtin_bit_cast(int, (v2)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w.x, 1.0f, false));
        o.y = __builtin_bit_cast(int, (v2)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w.x, 1.0f, true));
        o.z = __builtin_bit_cast(int, (v2)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w.y, 1.0f, false));
        o.w = __builtin_bit_cast(int, (v2)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w.y, 1.0f, true));
    }
    return o;
}

// Makes zeros of the values in these 16 bytes that are NaN or infinite; whether there were any.
template <class T, bool E4M3>
__device__ inline bool strip(i32x4& w) {
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        unsigned u = static_cast<unsigned>(w[j]);
#pragma unroll
        for (int q = 0; q < (E4M3 ? 4 : 2); ++q) {
            const unsigned e = E4M3 ? 0x7fu << (8 * q) : T::EXP << (16 * q), all = E4M3 ? 0xffu << (8 * q) : 0xffffu << (16 * q);
            if ((u & e) == e) { odd = true; u &= ~all; }
        }
        w[j] = static_cast<int>(u);
    }
    return odd;
}

// element d of a value in the cache
template <class T, bool E4M3>
__device__ inline float value_at(const char* row, int d) {
    if constexpr (E4M3) {
        const i32x4 w = widen8<T>(i32x2{static_cast<int>(reinterpret_cast<const unsigned char*>(row)[d]), 0});
        return T::lo(static_cast<unsigned>(w.x));
    } else {
        return T::lo(reinterpret_cast<const unsigned short*>(row)[d]);
    }
}

template <int D, bool E4M3>
struct TileShape {
    static constexpr int RB = D * (E4M3 ? 1 : 2);          // bytes of a row (one key or value)
    static constexpr int CPR = RB / 16;                    // 16-byte chunks of a row
    static constexpr int RPI = 64 / CPR;                   // rows one load instruction of a wave fills
    static constexpr int RPI_SHIFT = RPI == 16 ? 4 : RPI == 8 ? 3 : RPI == 4 ? 2 : 1;
    static constexpr int NL = TT / RPI;                    // load instructions per tile
    // In LDS the rows of one load instruction are contiguous (1 KB), with PAD bytes between
    // instructions, and row r's 16-byte chunk c is at place c ^ mix(r % RPI) of its row. So
    // the 16 lanes that read one chunk of 16 consecutive rows touch 16 different 16-byte
    // columns of the banks, and a lane's addresses for other chunks, rows 16 further
    // on, and other load instructions differ by constants (the instructions' offsets).
    static constexpr int PAD = CPR == 32 ? 32 : CPR == 4 ? 0 : 64;
    static constexpr int GAP = 1024 + PAD;
    __device__ static inline int mix(int lrow) { return CPR >= 16 ? lrow : CPR == 8 ? lrow >> 1 : lrow >> 2; }
    __device__ static inline int place(int row) { return row / RPI * GAP + row % RPI * RB; }
    static constexpr int NEXT16 = 16 / RPI * GAP;          // from row r to row r + 16
    // Column blocks of the values whose addresses differ by more than constants.
    static constexpr int AV = E4M3 ? 4 : CPR == 32 ? 1 : 2;
};

// How a workgroup's waves share the work. KEYS: each takes other keys, with all the query
// rows (up to 32). ROWS, for more query rows: each takes other rows, MT * 16 of them, and
// all walk the same tiles, which they load together; one barrier a tile.
template <int D, int MT, bool E4M3, bool ROWS>
struct AttnShape : TileShape<D, E4M3> {
    using S = TileShape<D, E4M3>;
    static constexpr int SUB = ROWS && S::NL < NWQ ? NWQ / S::NL : 1;      // steps of 32 keys a tile holds
    static constexpr int KT = TT * SUB;                    // keys of a tile
    static constexpr int NLW = ROWS ? S::NL * SUB / NWQ : S::NL;           // a wave's loads for its keys
    static constexpr int HALF = KT / S::RPI * S::GAP;      // bytes of a tile's keys (or values)
    static constexpr int STAGE = (ROWS ? 2 : 2 * NWQ) * HALF;              // of one tile (or one per wave)
    static constexpr int M16 = 16 * MT * (ROWS ? NWQ : 1); // query rows
    static constexpr int PARTS = ROWS ? 1 : NWQ;           // partial results per query row
    // Row tiles whose queries stand in LDS, one copy for all waves, and are read for every tile
    // of keys: where the registers of two waves per SIMD do not hold them (8-bit cache, R * G =
    // 40, 201 MB of keys and values: 55.6 us, 58.5 with all of them in registers, which spills).
    static constexpr int QL = D == 128 && MT == 3 && E4M3 && !ROWS ? 1 : 0;
    // Workgroups per CU (waves per SIMD): at most what the registers allow, that is, the
    // accumulators, the queries, scores and weights, one tile's operands and about 70 more.
    // Of these, what has the most tiles in flight on the CU, for more loads in flight get
    // nearer to HBM's rate (with ROWS one tile is not in flight but in use), and of these the
    // most waves. 8-bit cache, D = 128, R * G = 8, 32 rows of 2048 keys: two workgroups of
    // two tiles per wave 32.5 us, three of one 37.2; D = 64 in 16 bits, R * G = 24, 32 rows of
    // 2048: two of two 34.2 us, three of one 39.0; R * G = 1, 32 rows of 1024: four of one
    // 47.9 us, three of one 49.0.
    static constexpr int LDS_CU = 160 * 1024, MORE = 4 * 1024;             // per CU; beside the tiles
    static constexpr int REGS = 512 / (D * MT / 4 + D * (MT - QL) / 8 + 12 * MT + D / (E4M3 ? 8 : 4) + 70);
    static constexpr int tiles(int occ) {
        const int n = (LDS_CU / occ - MORE) / STAGE, most = ROWS ? 6 : 4;
        return n < most ? n : most;
    }
    static constexpr int occupancy() {
        const int most = REGS < 1 ? 1 : REGS > (ROWS ? 3 : 4) ? (ROWS ? 3 : 4) : REGS, idle = ROWS ? 1 : 0;
        int best = 1;
        for (int occ = 2; occ <= most; ++occ)
            if (tiles(occ) > 2 * idle && occ * (tiles(occ) - idle) >= best * (tiles(best) - idle)) best = occ;
        return best;
    }
    static constexpr int OCC = occupancy();
    static constexpr int NS = tiles(OCC);
    static_assert(NS >= (ROWS ? 2 : 1) && (2 * NS - 1) * NLW <= 63, "tiles");
};

template <class T, int D, int MT, bool E4M3, bool ROWS>
__global__ __launch_bounds__(NTQ, (AttnShape<D, MT, E4M3, ROWS>::OCC)) void attn_kernel(AttnParams A) {
    using S = AttnShape<D, MT, E4M3, ROWS>;
    constexpr int M16 = S::M16, ND = D / 16, NC = D / 32, NS = S::NS, NP = S::PARTS, KT = S::KT;
    constexpr int STRIDE = ROWS ? 1 : NWQ;                 // from a wave's tile to its next
    __shared__ __attribute__((aligned(16))) unsigned char lds[NS * S::STAGE];
    __shared__ float st_m[NP][M16], st_l[NP][M16], fin[M16];
    __shared__ Plan plan;
    __shared__ int odd_any;                                // some edge value was not finite
    __shared__ i32x4 q_lds[S::QL > 0 ? S::QL * NC * 64 : 1];
    const Cache& C = A.c;
    const int t = static_cast<int>(threadIdx.x), lane = t & 63, wv = __builtin_amdgcn_readfirstlane(t >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    // the MB row blocks of one range read the same keys: workgroups 8 apart, on one XCD
    const int per = 8 * A.MB, sub = static_cast<int>(blockIdx.x) % per;
    const int x = static_cast<int>(blockIdx.x) / per * 8 + sub % 8, mb = sub / 8;
    if (x >= A.W * C.Hkv) return;
    const int h = x % C.Hkv, w = x / C.Hkv;
    if (t == 0) odd_any = 0;
    __syncthreads();
    int b = 0, next_kv = 0, next_n = 0;
    long long pre = 0;
    const Ranges ranges = locate(A, plan, w, b, next_kv, next_n, pre);
    RangeRec* recs = reinterpret_cast<RangeRec*>(A.ws);
    const bool scribe = A.W > 1 && h == 0 && mb == 0 && t == 0;
    if (w >= ranges.ranges) {
        if (scribe && !A.direct) recs[w] = RangeRec{0, 0, -1, -1};
        return;
    }
    long long at = ranges.start(w);
    const long long end = ranges.start(w + 1);
    bool first = true;
    unsigned char* tiles_at = lds + (ROWS ? 0 : wv * (NS * 2 * S::HALF));  // [stage][keys, values]
    const char* kbase = C.k + h * C.ks[1];
    const char* vbase = C.v + h * C.vs[1];
    const float ksc = E4M3 ? C.k_scale[h] : 1.0f, vsc = E4M3 ? C.v_scale[h] : 1.0f;
    const float scale = A.scale * ksc;
    const int slot_mask = (1 << C.shift) - 1;
    // where this lane reads its operands in a tile: key r16, and (transposed) the piece of
    // the values that it fetches for its group
    const int k_at = S::place(r16) + (g ^ S::mix(r16 % S::RPI)) * 16;
    int v_at[S::AV];
#pragma unroll
    for (int i = 0; i < S::AV; ++i) {
        const int rr = r16 >> 1, row = !E4M3 ? 4 * g + (r16 >> 2) : rr < 4 ? 4 * g + rr : 12 + 4 * g + rr;
        const int chunk = E4M3 ? i : 2 * i + (rr & 1);
        v_at[i] = S::place(row) + (chunk ^ S::mix(row % S::RPI)) * 16 + (r16 & 1) * 8;
    }
    const int m0 = mb * M16, mw = ROWS ? wv * 16 * MT : 0; // the block's and, in it, the wave's first row

    while (at < end) {
        const Seq sq = first ? seq_from(A, next_kv, next_n) : seq_of(A, b);
        // the same in every lane: scalars
        const int kv = __builtin_amdgcn_readfirstlane(sq.kv), n_tok = __builtin_amdgcn_readfirstlane(sq.n);
        const int lo = __builtin_amdgcn_readfirstlane(sq.lo), hi = __builtin_amdgcn_readfirstlane(sq.hi);
        const int base = __builtin_amdgcn_readfirstlane(sq.base), units = __builtin_amdgcn_readfirstlane(sq.units);
        const int u0 = __builtin_amdgcn_readfirstlane(static_cast<int>(at - pre));
        const int u1 = __builtin_amdgcn_readfirstlane(static_cast<int>(end - pre < units ? end - pre : units));
        at += u1 - u0;
        if (scribe && (A.direct ? u0 == 0 : first))
            recs[A.direct ? b : w] = RangeRec{b, n_tok, ranges.holding(pre), ranges.holding(pre + units - 1)};
        first = false;
        if (n_tok == 0) {                                  // bad lengths: one unit, NaN
            for (int i = fresh(t); i < M16 * D; i += NTQ) {
                const int m = m0 + i / D;
                if (m < A.M) {
                    const long long row = (static_cast<long long>(b) * C.R + m / A.G) * A.Hq + h * A.G + m % A.G;
                    reinterpret_cast<typename T::type*>(A.out)[row * D + i % D] = static_cast<typename T::type>(NAN);
                }
            }
            pre += 1;
            ++b;
            continue;
        }
        const bool whole = u0 == 0 && u1 == units;
        const int beg = base + u0 * TU, stop = min(hi, base + u1 * TU);
        const int tiles = (stop - beg + KT - 1) / KT;
        const int* table = C.table + static_cast<long long>(b) * C.max_pages;
        int bad = 0;
        // the page of the tile's key lane % KT; keys nobody sees are taken from the
        // nearest that somebody does (and masked)
        auto key_of = [&](int tile, int row) { return min(max(beg + tile * KT + row, lo), hi - 1); };
        auto page_at = [&](int tile) { return table[key_of(tile, lane & (KT - 1)) >> C.shift]; };
        auto checked = [&](int p) {
            if (!page_ok(C, p)) { bad = 1; p = 0; }
            return p;
        };
        // A load instruction fills RPI consecutive, aligned rows. They lie in one page
        // unless pages are shorter, so page and place are scalars; rows of keys nobody
        // sees then stand in a page that somebody needs.
        auto issue = [&](unsigned char* dst, const char* cache, const long long (&str)[3], int tile, int pages) {
            const int j0 = ROWS ? wv * S::NLW : 0;
            const int lrow = lane / S::CPR;
            const unsigned off = static_cast<unsigned>(lrow) * static_cast<unsigned>(str[2]) +
                                 static_cast<unsigned>((lane % S::CPR) ^ S::mix(lrow)) * 16u;
            if (C.shift >= S::RPI_SHIFT) {
#pragma unroll
                for (int j = 0; j < S::NLW; ++j) {
                    const int row = (j0 + j) * S::RPI;
                    const int page = __builtin_amdgcn_readlane(pages, row);
                    const int slot = (beg + tile * KT + row) & slot_mask;
                    const char* src = cache + page * str[0] + slot * str[2];
                    __builtin_amdgcn_global_load_lds((glb_ptr)(src + off), untraced((lds_ptr)(dst + (j0 + j) * S::GAP)),
                                                     16, 0, NT_LOAD);
                }
            } else {
                const int l = fresh(lane), lrow = l / S::CPR;
#pragma unroll 1
                for (int j = j0; j < j0 + S::NLW; ++j) {
                    const int row = j * S::RPI + lrow;
                    const int page = __shfl(pages, row, 64);
                    const int slot = key_of(tile, row) & slot_mask;
                    const char* src = cache + page * str[0] + slot * str[2] + ((l % S::CPR) ^ S::mix(lrow)) * 16;
                    __builtin_amdgcn_global_load_lds((glb_ptr)src, untraced((lds_ptr)(dst + j * S::GAP)), 16, 0, NT_LOAD);
                }
            }
        };
        // the first tiles (all but one of the places with ROWS), and the next one's pages
        constexpr int AHEAD = ROWS ? NS - 1 : NS;
        int tile = ROWS ? 0 : wv, stage = 0;
        int pages = 0;
        if (tile < tiles) {
            int p[AHEAD + 1];
#pragma unroll
            for (int j = 0; j <= AHEAD; ++j) p[j] = page_at(tile + j * STRIDE);    // (past the last tile: the last key's)
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                if (tile + j * STRIDE >= tiles) break;
                const int now = checked(p[j]);
                issue(tiles_at + j * 2 * S::HALF, kbase, C.ks, tile + j * STRIDE, now);
                issue(tiles_at + j * 2 * S::HALF + S::HALF, vbase, C.vs, tile + j * STRIDE, now);
            }
            pages = checked(p[AHEAD]);
        }
        // this lane's query rows: the MFMA's B operand, and where each one stands
        constexpr int REG_Q = MT - S::QL;                  // row tiles with their queries in registers
        i32x4 qf[REG_Q][NC];
        int pos[MT];                                       // the row's position
        float slope[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int m = m0 + mw + mt * 16 + fresh(r16), G = fresh(A.G);
            const int i = m < A.M ? m / G : 0, hq = h * G + (m < A.M ? m % G : 0);
            const char* row = A.q + b * A.qs[0] + i * A.qs[1] + hq * A.qs[2];
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                // the products with 8 bits take 16 consecutive elements of a key per lane
                const int d = E4M3 ? (c / 2) * 64 + g * 16 + (c & 1) * 8 : c * 32 + g * 8;
                i32x4 qv = *reinterpret_cast<const i32x4*>(row + d * 2);
                if (m >= A.M) qv = i32x4{0, 0, 0, 0};
                if (mt < REG_Q) qf[mt < REG_Q ? mt : 0][c] = qv;
                else if (wv == 0) q_lds[((mt - REG_Q) * NC + c) * 64 + lane] = qv;
            }
            pos[mt] = kv + min(i, n_tok - 1);
            slope[mt] = A.slopes ? A.slopes[hq] * LOG2E : 0.0f;
        }
        if constexpr (S::QL > 0) __syncthreads();
        f32x4 acc[ND][MT];
        float mx[MT], sum[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            mx[mt] = -F32_MAX;
            sum[mt] = 0.0f;
#pragma unroll
            for (int d = 0; d < ND; ++d) acc[d][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        // A weight of zero does not cancel a value that is not finite. Values that nobody sees
        // become zeros; of those that only some rows see what is not finite does, and is
        // added to the rows that see it at the end.
        auto clean = [&](unsigned char* vt, int tok0, int from, int by) {
            for (int c = fresh(from); c < KT * S::CPR; c += by) {
                i32x4* at16 = reinterpret_cast<i32x4*>(vt + c / 64 * S::GAP + c % 64 * 16);
                const int key = tok0 + c / S::CPR;
                if (key < lo || key >= hi) {
                    *at16 = i32x4{0, 0, 0, 0};
                } else if (key > kv || (A.window > 0 && key <= hi - 1 - A.window)) {
                    i32x4 v = *at16;
                    if (strip<T, E4M3>(v)) { *at16 = v; odd_any = 1; }
                }
            }
        };
        // One tile; MORE: AHEAD tiles on there is another. Loads in flight are counted in
        // their order: keys and values of a tile, then of the next. KEYS loads the other
        // tile into this one's place as soon as the operands are read. ROWS loads it into
        // the place of the tile before this one, which everyone is done with at the barrier.
        auto step = [&](auto MORE) {
            constexpr bool more = decltype(MORE)::value != 0;
            unsigned char* kt = tiles_at + (NS > 1 ? stage : 0) * 2 * S::HALF;
            unsigned char* vt = kt + S::HALF;
            const int tok0 = beg + tile * KT;
            const int pages_now = pages;
            if constexpr (ROWS) {
                wait_loads<(more ? (NS - 2) * 2 * S::NLW : 0)>();
                __syncthreads();
                if constexpr (more) {
                    unsigned char* to = tiles_at + (stage ? stage - 1 : NS - 1) * 2 * S::HALF;
                    issue(to, kbase, C.ks, tile + AHEAD, pages_now);
                    issue(to + S::HALF, vbase, C.vs, tile + AHEAD, pages_now);
                    pages = checked(page_at(tile + AHEAD + 1));
                }
            } else {
                wait_loads<(more ? (2 * NS - 1) * S::NLW : NS > 1 ? 0 : S::NLW)>();        // the keys are in
            }
            const bool edge = tok0 + KT - 1 > kv || (A.window > 0 && tok0 <= hi - 1 - A.window);
            if (ROWS && edge) {
                clean(vt, tok0, t, NTQ);
                wait_lds();
                __syncthreads();
            }
#pragma unroll
            for (int sub = 0; sub < S::SUB; ++sub) {
            const int tok = tok0 + sub * TT;
            const unsigned char* kr = kt + k_at + sub * 2 * S::NEXT16;
            unsigned char* vr = vt + sub * 2 * S::NEXT16;
            i32x4 kf[2][E4M3 ? NC / 2 : NC];
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int c = 0; c < (E4M3 ? NC / 2 : NC); ++c)
                    kf[a][c] = *reinterpret_cast<const i32x4*>(kr + a * S::NEXT16 + c * 64);
            if constexpr (!ROWS) {
                wait_lds();                                // their place is free
                if constexpr (more) {
                    issue(kt, kbase, C.ks, tile + NS * NWQ, pages_now);
                    pages = checked(page_at(tile + (NS + 1) * NWQ));
                }
            }
            i32x4 qt[S::QL > 0 ? S::QL : 1][NC];
#pragma unroll
            for (int i = 0; i < S::QL * NC; ++i) qt[i / NC][i % NC] = q_lds[i * 64 + lane];
            f32x4 sc[2][MT];
#pragma unroll
            for (int a = 0; a < 2; ++a) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) sc[a][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    i32x4 k;
                    if constexpr (E4M3) {
                        const i32x4 k16 = kf[a][c / 2];
                        k = widen8<T>(c & 1 ? i32x2{k16.z, k16.w} : i32x2{k16.x, k16.y});
                    } else {
                        k = kf[a][c];
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        sc[a][mt] = mfma<T>(k, mt < REG_Q ? qf[mt < REG_Q ? mt : 0][c] : qt[mt < REG_Q ? 0 : mt - REG_Q][c], sc[a][mt]);
                }
            }
            // scores in units of log2, masked
            if (A.softcap >= CAP_FINE) {
                // The form below is off by 2^-21 of the cap, which for a large one is more than
                // the scores' own rounding. Here small y = v / cap take tanh's series (its
                // next term is 2^-21 of it at y = 1/4).
                const float by = scale / A.softcap, factor = scale * LOG2E;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float v = sc[j / 4][mt][j % 4], y = v * by, y2 = y * y;
                        const float e = __builtin_amdgcn_exp2f(y * (2.0f * LOG2E));
                        const float far = (1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + e)) * A.softcap * LOG2E;
                        const float near = v * factor * (1.0f + y2 * (-1.0f / 3 + y2 * (2.0f / 15 - y2 * (17.0f / 315))));
                        sc[j / 4][mt][j % 4] = fabsf(y) < 0.25f ? near : far;
                    }
            } else if (A.softcap > 0.0f) {                 // cap tanh(v / cap) = cap (1 - 2 / (1 + e^(2 v / cap)))
                const float c = A.softcap * LOG2E, e2 = scale / A.softcap * 2.0f * LOG2E;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float e = __builtin_amdgcn_exp2f(sc[j / 4][mt][j % 4] * e2);
                        sc[j / 4][mt][j % 4] = c - 2.0f * c * __builtin_amdgcn_rcpf(1.0f + e);
                    }
            } else {
                const float factor = scale * LOG2E;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sc[j / 4][mt][j % 4] *= factor;
            }
            if (A.slopes) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const int away = tok + 4 * fresh(g) - pos[mt];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        sc[j / 4][mt][j % 4] += slope[mt] * static_cast<float>(away + 16 * (j / 4) + j % 4);
                }
            }
            if (edge) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const int away = tok + 4 * fresh(g) - pos[mt];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int k = away + 16 * (j / 4) + j % 4;
                        if (k > 0 || (A.window > 0 && k <= -A.window)) sc[j / 4][mt][j % 4] = -INFINITY;
                    }
                }
            }
            bool up = false;
            float top[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                top[mt] = fmaxf(sc[0][mt][0], sc[0][mt][1]);
#pragma unroll
                for (int j = 2; j < 8; ++j) top[mt] = fmaxf(top[mt], sc[j / 4][mt][j % 4]);
                up = up || top[mt] > mx[mt] + T::LAZY;
            }
            if (__any(up)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    float n = top[mt];
                    n = fmaxf(n, __shfl_xor(n, 16, 64));
                    n = fmaxf(n, __shfl_xor(n, 32, 64));
                    n = fmaxf(n - T::TOP, mx[mt]);
                    const float f = __builtin_amdgcn_exp2f(mx[mt] - n);
                    mx[mt] = n;
                    sum[mt] *= f;
#pragma unroll
                    for (int d = 0; d < ND; ++d) acc[d][mt] *= f;
                }
            }
            i32x4 pf[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    float p[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        p[r] = exp2_diff(sc[a][mt][r], mx[mt]);
                        sum[mt] += p[r];
                    }
                    // rounded once to the operand type of the matrix cores
                    pf[mt][2 * a] = static_cast<int>(pack2<T>(p[0], p[1]));
                    pf[mt][2 * a + 1] = static_cast<int>(pack2<T>(p[2], p[3]));
                }
            }
            if constexpr (!ROWS) {
                wait_loads<(more ? (2 * NS - 1) * S::NLW : 0)>();          // the values are in
                if (edge) {
                    clean(vt, tok0, lane, 64);
                    wait_lds();
                }
            }
            // columns 16 d .. 16 d + 15 of the values as the MFMA's A operand
            i32x2 vf[ND][E4M3 ? 1 : 2];
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                unsigned char* at_v = vr + v_at[d % S::AV] + d / S::AV * (S::AV * (E4M3 ? 16 : 32));
                if constexpr (E4M3) {
                    vf[d][0] = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2)at_v);
                } else {
#pragma unroll
                    for (int a = 0; a < 2; ++a)
                        vf[d][a] = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                                 (lds_i16x4)(at_v + a * S::NEXT16)));
                }
            }
            if constexpr (!ROWS) {
                wait_lds();                                // their place is free
                if constexpr (more) issue(vt, vbase, C.vs, tile + NS * NWQ, pages_now);
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                i32x4 v;
                if constexpr (E4M3) v = widen8<T>(vf[d][0]);
                else v = i32x4{vf[d][0].x, vf[d][0].y, vf[d][1].x, vf[d][1].y};
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) acc[d][mt] = mfma<T>(v, pf[mt], acc[d][mt]);
            }
            }
            tile += STRIDE;
            if (NS > 1) stage = stage + 1 < NS ? stage + 1 : 0;
        };
        if (tile < tiles) {
            while (tile + AHEAD * STRIDE < tiles) step(Int<1>());
            do step(Int<0>()); while (tile < tiles);
        }
        // ---- join the waves (KEYS), normalise, write
        const bool nan = __any(bad);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float l = sum[mt];
            l += __shfl_xor(l, 16, 64);
            l += __shfl_xor(l, 32, 64);
            if (nan) l = NAN;
            if (g == 0) {
                st_m[ROWS ? 0 : wv][mw + mt * 16 + r16] = mx[mt];
                st_l[ROWS ? 0 : wv][mw + mt * 16 + r16] = l;
            }
        }
        __syncthreads();                                   // the statistics are in, the tiles are free
        const bool odd = odd_any != 0;
        float* slot = A.ws + A.slots_at + (static_cast<long long>(w * C.Hkv + h) * A.MB + mb) * (2ll * M16 * (D + 2)) +
                      (u0 == 0 ? M16 * (D + 2) : 0);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int m = mw + mt * 16 + r16;
            float n = st_m[0][m], l = st_l[0][m];
            if constexpr (!ROWS) {
#pragma unroll
                for (int j = 1; j < NP; ++j) n = fmaxf(n, st_m[j][m]);
                l = 0.0f;
#pragma unroll
                for (int j = 0; j < NP; ++j) l += st_l[j][m] * __builtin_amdgcn_exp2f(st_m[j][m] - n);
                const float f = __builtin_amdgcn_exp2f(mx[mt] - n);
#pragma unroll
                for (int d = 0; d < ND; ++d) acc[d][mt] *= f;
            }
            if (g == 0 && (ROWS || wv == 0)) {
                fin[m] = l;
                if (!whole) {
                    slot[M16 * D + 2 * m] = n;
                    slot[M16 * D + 2 * m + 1] = l;
                }
            }
        }
        // through LDS as [part][16-element column block][row][16]: the writes of a wave and the
        // reads of consecutive threads are contiguous
        constexpr int FIT = NS * S::STAGE / (NP * M16 * 64);       // column blocks that fit
        constexpr int DC = FIT >= ND ? ND : FIT >= 8 ? 8 : FIT >= 4 ? 4 : FIT >= 2 ? 2 : 1;
        static_assert(FIT >= 1, "exchange");
        float* ex = reinterpret_cast<float*>(lds);
#pragma unroll
        for (int d0 = 0; d0 < ND; d0 += DC) {
#pragma unroll
            for (int d = 0; d < DC; ++d)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    *reinterpret_cast<f32x4*>(ex + (((ROWS ? 0 : wv) * DC + d) * M16 + mw + mt * 16 + fresh(r16)) * 16 + 4 * g) =
                        acc[d0 + d][mt];
            __syncthreads();
            if (t == 0) odd_any = 0;                       // (everyone has read it)
            for (int i = fresh(t); i < M16 * DC * 4; i += NTQ) {
                const int m = i / 4 % M16, block = d0 + i / (4 * M16), d = block * 16 + i % 4 * 4;
                if (m0 + m >= A.M) continue;
                f32x4 o = *reinterpret_cast<const f32x4*>(ex + 4 * i);
#pragma unroll
                for (int j = 1; j < NP; ++j) o += *reinterpret_cast<const f32x4*>(ex + j * M16 * DC * 16 + 4 * i);
                if (odd) {
                    const int at_pos = kv + min((m0 + fresh(m)) / A.G, n_tok - 1);
                    const int from = max(beg, lo), past = min(stop, hi), seen_by_all = hi - A.window;
                    for (int key = from; key < past; ++key) {
                        if (key <= kv && (A.window <= 0 || key >= seen_by_all)) {
                            key = kv;                      // on to those after the first position
                            continue;
                        }
                        if (key > at_pos || (A.window > 0 && key <= at_pos - A.window)) continue;
                        const int page = table[key >> C.shift];
                        if (!page_ok(C, page)) continue;
                        const char* row = vbase + page * C.vs[0] + (key & slot_mask) * C.vs[2];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float v = value_at<T, E4M3>(row, d + j);
                            if (!(fabsf(v) <= F32_MAX)) o[j] += v;
                        }
                    }
                }
                if (whole) {
                    const int tk = (m0 + m) / A.G, hq = h * A.G + (m0 + m) % A.G;
                    u32x2 y = {0, 0};
                    if (tk < n_tok) {
                        const float inv = vsc / fin[m];
                        y.x = pack2<T>(o.x * inv, o.y * inv);
                        y.y = pack2<T>(o.z * inv, o.w * inv);
                    }
                    const long long row = (static_cast<long long>(b) * C.R + tk) * A.Hq + hq;
                    *reinterpret_cast<u32x2*>(A.out + (row * D + d) * 2) = y;
                } else {
                    *reinterpret_cast<f32x4*>(slot + (block * M16 + m) * 16 + i % 4 * 4) = o;
                }
            }
            __syncthreads();
        }
        if (u1 == units) { pre += units; ++b; }
    }
}

// Merges the pieces of every sequence that crosses ranges. A workgroup takes some rows of
// one sequence: those of a batch row or, when there are at least as many batch rows as
// ranges, of the sequence that the border before range w cuts (the first border inside
// a sequence stands for it). D / 4 threads hold a row; `slices` of such groups share its
// pieces, four loads of each in flight, and meet in LDS. Bound by the latency of its chain
// (launch, record, pieces): 4 us for few pieces, 7 us where 512 workgroups left 32 to 48
// rows each (8 to 13 MB); eight loads in flight measure the same.
template <class T>
__global__ __launch_bounds__(NTQ) void join_kernel(AttnParams A) {
    __shared__ float st[NTQ][2];
    __shared__ f32x4 so[NTQ];
    const Cache& C = A.c;
    const int t = static_cast<int>(threadIdx.x), cols = A.D / 4, rows = NTQ / cols / A.slices;
    const int groups = (A.M16 + rows - 1) / rows;
    int x = static_cast<int>(blockIdx.x);
    const int gr = x % groups; x /= groups;
    const int mb = x % A.MB; x /= A.MB;
    const int h = x % C.Hkv; x /= C.Hkv;
    const RangeRec rec = reinterpret_cast<const RangeRec*>(A.ws)[A.direct ? x : x + 1];
    const int wa = rec.wa, wb = rec.wb;
    if (wa >= wb || (!A.direct && wa != x)) return;
    const int col = t % cols, row = t / cols % rows, sl = t / cols / rows;
    const int m = gr * rows + row, q = mb * A.M16 + m;
    const bool live = m < A.M16 && q < A.M;
    const long long size = static_cast<long long>(A.M16) * (A.D + 2);
    float n = -F32_MAX, l = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int w0 = wa + sl; live && w0 <= wb; w0 += 4 * A.slices) {
        float pm[4], pl[4];
        f32x4 po[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int w = w0 + j * A.slices;
            pm[j] = -F32_MAX;
            pl[j] = 0.0f;
            po[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (w <= wb) {
                const float* slot = A.ws + A.slots_at + ((static_cast<long long>(w) * C.Hkv + h) * A.MB + mb) * 2 * size +
                                    (w == wa ? size : 0);
                pm[j] = slot[A.M16 * A.D + 2 * m];
                pl[j] = slot[A.M16 * A.D + 2 * m + 1];
                po[j] = *reinterpret_cast<const f32x4*>(slot + (col / 4 * A.M16 + m) * 16 + col % 4 * 4);
            }
        }
        float nn = n;
#pragma unroll
        for (int j = 0; j < 4; ++j) nn = fmaxf(nn, pm[j]);
        const float f = __builtin_amdgcn_exp2f(n - nn);
        l *= f;
        o *= f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float e = __builtin_amdgcn_exp2f(pm[j] - nn);
            l += pl[j] * e;
            o += po[j] * e;
        }
        n = nn;
    }
    if (A.slices > 1) {
        st[t][0] = n;
        st[t][1] = l;
        so[t] = o;
        __syncthreads();
        if (sl > 0) return;
        for (int j = 1; j < A.slices; ++j) {
            const int u = t + j * cols * rows;
            const float nn = fmaxf(n, st[u][0]);
            const float f = __builtin_amdgcn_exp2f(n - nn), e = __builtin_amdgcn_exp2f(st[u][0] - nn);
            n = nn;
            l = l * f + st[u][1] * e;
            o = o * f + so[u] * e;
        }
    }
    if (!live) return;
    u32x2 y = {0, 0};
    const int tk = q / A.G;
    if (tk < rec.n_tok) {
        const float inv = (C.v_scale ? C.v_scale[h] : 1.0f) / l;
        y.x = pack2<T>(o.x * inv, o.y * inv);
        y.y = pack2<T>(o.z * inv, o.w * inv);
    }
    const long long at = (static_cast<long long>(rec.b) * C.R + tk) * A.Hq + h * A.G + q % A.G;
    *reinterpret_cast<u32x2*>(A.out + (at * A.D + col * 4) * 2) = y;
}

// ------------------------------------------------------------------ logit adjustment
//
// Bound by memory: the logits are read and written once, the masks and the histories are
// small beside them. A workgroup owns a segment of the vocabulary for all R rows of a
// batch row. It counts the segment's tokens of the history in LDS (integer atomics, so the
// order does not matter), lists the few tokens with a count or a bias, streams the segment
// of every row through registers with the mask applied, and overwrites the listed tokens,
// whose logits it took before the stream. The streaming loop so has no lookups, and rows
// whose start is not 16-byte aligned (an odd V) differ only in the up to 15 elements at
// the segment's ends that are moved one by one. A segment with many such tokens (those of
// a text cluster) is instead adjusted element by element in the stream.
//
// Measured (MI355X; a large copy reaches 5.12 TB/s read + written): [64, 6, 151936] bfloat16
// with histories of up to 2047, 16 biases and masks on half of the rows 62 us (237 MB: 3.8
// TB/s; 280 MB move, since listed tokens are read ahead of the stream and written behind
// it); every segment adjusted in the stream 335 us (registers spill), a second pass of all
// threads over the counts in place of the list 181 us. [256, 4, 128256] bfloat16 with biases
// and masks 109 us, 5.0 TB/s. One row of 32000 float32: 6 us, a chain of dependent loads.

constexpr int NTJ = 512;
constexpr int SEG_MAX = 8192;                              // most tokens of a segment (32 KB of counts)
constexpr int SEG_MAX_BIAS = 5120;                         // ... with as many 16-bit owners of biases beside them
constexpr int SEG_MIN = 512;
constexpr int ADJ_SLOTS = 4 * CUS;                         // resident workgroups
// Many: more than one token in 32. 8, 16, 32 and 64 measure 56.4, 54.3, 54.3 and 56.9 us on
// [64, 6, 151936] bfloat16 with penalties only, 80.6, 78.0, 77.0 and 75.9 on [64, 6, 128256]
// float32 with masks.
constexpr int DENSE = 32;
// count word: the low bits count the token behind the prompt
constexpr unsigned SEEN = 0x80000000u;                     // it is in the prompt
constexpr unsigned DRAFT = 0x40000000u;                    // it is among the drafts
constexpr unsigned BIASED = 0x20000000u;                   // it has a bias
constexpr unsigned COUNT = BIASED - 1;
constexpr int OPEN = -1, BROKEN = -2;                      // a row's mask: none; the row becomes NaN

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
    static constexpr unsigned NANS = 0x7fc00000u;
    __device__ static inline float one(const char* p, long long n) { return reinterpret_cast<const float*>(p)[n]; }
};
struct InBf16 {
    static constexpr int VE = 8, ES = 2;
    static constexpr unsigned NANS = 0x7fc07fc0u;
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

// The admit bits of tokens v..v+VE-1 (all < V) in the low bits; `whole`: they never cross a byte.
template <int VE>
__device__ inline unsigned admit_bits(const unsigned char* row, int v, bool whole) {
    unsigned w = row[static_cast<unsigned>(v) >> 3];
    if (!whole) w |= static_cast<unsigned>(row[static_cast<unsigned>(v + VE - 1) >> 3]) << 8;
    return w >> (v & 7);
}

template <class I>
__device__ inline void unpack(u32x4 w, float (&y)[I::VE]) {
    if constexpr (I::ES == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = bits_f32(w[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) { y[2 * j] = bits_f32(w[j] << 16); y[2 * j + 1] = bits_f32(w[j] & 0xffff0000u); }
    }
}

template <class I, bool OF>
__device__ inline void put_floats(char* out, const float (&y)[I::VE]) {
    if constexpr (OF || I::ES == 4) {
#pragma unroll
        for (int j = 0; j < I::VE; j += 4)
            reinterpret_cast<f32x4*>(out)[j / 4] = f32x4{y[j], y[j + 1], y[j + 2], y[j + 3]};
    } else {
        *reinterpret_cast<u32x4*>(out) = u32x4{pack2<Bf16>(y[0], y[1]), pack2<Bf16>(y[2], y[3]),
                                               pack2<Bf16>(y[4], y[5]), pack2<Bf16>(y[6], y[7])};
    }
}

// w where the mask's bits are set, else -infinity
__device__ inline unsigned pick(unsigned mask, unsigned w, unsigned inf) { return (w & mask) | (inf & ~mask); }
// all ones if bit j of bits is set, else zero
__device__ inline unsigned spread(unsigned bits, int j) {
    return static_cast<unsigned>(static_cast<int>(bits << (31 - j)) >> 31);
}

template <class I, bool OF, bool MASK>
__device__ inline void put_vec(char* out, u32x4 w, unsigned bits) {
    if constexpr (I::ES == 4) {
        if constexpr (MASK) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pick(spread(bits, j), w[j], 0xff800000u);
        }
        *reinterpret_cast<u32x4*>(out) = w;
    } else if constexpr (!OF) {
        if constexpr (MASK) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = pick((spread(bits, 2 * j) & 0xffffu) | (spread(bits, 2 * j + 1) & 0xffff0000u), w[j], 0xff80ff80u);
        }
        *reinterpret_cast<u32x4*>(out) = w;
    } else {
        u32x4 a, b;
        a.x = w.x << 16; a.y = w.x & 0xffff0000u; a.z = w.y << 16; a.w = w.y & 0xffff0000u;
        b.x = w.z << 16; b.y = w.z & 0xffff0000u; b.z = w.w << 16; b.w = w.w & 0xffff0000u;
        if constexpr (MASK) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a[j] = pick(spread(bits, j), a[j], 0xff800000u);
                b[j] = pick(spread(bits, 4 + j), b[j], 0xff800000u);
            }
        }
        reinterpret_cast<u32x4*>(out)[0] = a;
        reinterpret_cast<u32x4*>(out)[1] = b;
    }
}

template <class I, bool OF, bool BIAS>
__global__ __launch_bounds__(NTJ, 8) void adjust_kernel(AdjustParams A) {
    constexpr int SEG = BIAS ? SEG_MAX_BIAS : SEG_MAX, VE = I::VE, U = 4;
    __shared__ __attribute__((aligned(16))) unsigned cnt[SEG];
    __shared__ unsigned short own[BIAS ? SEG : 1], list[SEG / DENSE];
    __shared__ int mask_of[SPEC_MAX_K + 1], drafts[SPEC_MAX_K + 1];
    __shared__ int dup, listed;
    const int t = static_cast<int>(threadIdx.x);
    // Low segments first: vocabularies put frequent tokens there, so these take longest. Batch
    // rows are rotated, so that the segments of one do not meet on one XCD and read its
    // history through the same channels of that L2 at the same time.
    const int s = static_cast<int>(blockIdx.x) / A.B, b = (static_cast<int>(blockIdx.x) % A.B + s) % A.B;
    const int v0 = s * A.seg, len = min(A.V - v0, A.seg);
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
    const bool any = (counts && (n > 0 || A.k > 0)) || (BIAS && !bad);
    const long long row0 = static_cast<long long>(b) * A.R;
    if (t < rows) {
        const int ar = A.admit ? (A.admit_row ? A.admit_row[row0 + t] : static_cast<int>(row0 + t)) : OPEN;
        mask_of[t] = bad || ar < OPEN || (A.admit && ar >= A.n_admit) ? BROKEN : ar;
    }
    if (t < A.k)                                           // (0 .. len - 1: in the segment)
        drafts[t] = static_cast<int>(static_cast<unsigned>(A.tokens[static_cast<long long>(b) * A.k + t]) -
                                     static_cast<unsigned>(v0));
    // The stream's items are 64 consecutive 16-byte vectors of a row, one per lane, wave by
    // wave: row, place and mask are scalars.
    constexpr int EO = OF ? 4 : I::ES;
    const int lane = t & 63, wv = uniform(t >> 6);
    const int chunks = A.vec ? (len / VE + 63) / 64 : 0;
    const bool whole = A.V % 8 == 0;
    struct Item {
        int row, chunk;
    };
    auto advance = [&](Item& it) {
        it.chunk += NTJ / 64;
        while (it.chunk >= chunks) { it.chunk -= chunks; ++it.row; }
    };
    auto row_at = [&](int row) { return (row0 + row) * A.V + v0; };
    // the lane's first token; it has a vector if the VE tokens are in the segment
    auto token = [&](const Item& it) {
        return static_cast<int>(-row_at(it.row) & (VE - 1)) + (it.chunk * 64 + lane) * VE;
    };
    Item it0{0, wv - NTJ / 64};
    if (chunks > 0) advance(it0);
    else it0.row = rows;
    auto load = [&](const Item& it) {                      // read once (or, where adjusted, just before)
        const unsigned v = static_cast<unsigned>(token(it));
        if (it.row >= rows || v + VE > static_cast<unsigned>(len)) return u32x4{0, 0, 0, 0};
        return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(A.in + row_at(it.row) * I::ES + v * I::ES));
    };
    // the first items' logits come in while the history is counted
    u32x4 x[U];
    {
        Item it = it0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = u32x4{0, 0, 0, 0};
            if (!A.inplace && chunks > 0) {
                x[u] = load(it);
                advance(it);
            }
        }
    }
    if (any) {
        for (int v = 4 * t; v < len; v += 4 * NTJ) *reinterpret_cast<u32x4*>(cnt + v) = u32x4{0, 0, 0, 0};
        if (t == 0) dup = listed = 0;
    }
    __syncthreads();
    if (any) {
        if (counts) {
            const int* h = A.history + static_cast<long long>(b) * A.H;
            auto count = [&](int token, int j) {
                const unsigned v = static_cast<unsigned>(token) - static_cast<unsigned>(v0);
                if (v < static_cast<unsigned>(len)) {
                    if (j < p) atomicOr(&cnt[v], SEEN);
                    else atomicAdd(&cnt[v], 1u);
                }
            };
            // 16-byte loads, four in flight, between the unaligned ends
            const int head = min(n, static_cast<int>(-(reinterpret_cast<uintptr_t>(h) / 4) & 3)), quads = (n - head) / 4;
            for (int q0 = t; q0 < quads; q0 += U * NTJ) {
                i32x4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int q = q0 + u * NTJ;
                    v[u] = q < quads ? *reinterpret_cast<const i32x4*>(h + head + 4 * q) : i32x4{-1, -1, -1, -1};
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) count(v[u][j], head + 4 * (q0 + u * NTJ) + j);
            }
            if (t < head) count(h[t], t);
            if (t < n - head - 4 * quads) count(h[head + 4 * quads + t], head + 4 * quads + t);
            if (t < min(A.k, rows - 1) && static_cast<unsigned>(drafts[t]) < static_cast<unsigned>(len))
                atomicOr(&cnt[drafts[t]], DRAFT);
        }
        if constexpr (BIAS) {
            for (int j = t; j < A.nb; j += NTJ) {
                const unsigned v = static_cast<unsigned>(A.bias_tok[static_cast<long long>(b) * A.nb + j]) -
                                   static_cast<unsigned>(v0);
                if (v < static_cast<unsigned>(len)) {
                    if (atomicOr(&cnt[v], BIASED) & BIASED) dup = 1;       // a token twice in the list: rare
                    else own[v] = static_cast<unsigned short>(j);
                }
            }
        }
        __syncthreads();
        for (int v4 = 4 * t; v4 < len; v4 += 4 * NTJ) {
            const u32x4 c = *reinterpret_cast<const u32x4*>(cnt + v4);
            if ((c.x | c.y | c.z | c.w) == 0) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c[j] != 0) {
                    const int at = atomicAdd(&listed, 1);
                    if (at < SEG / DENSE) list[at] = static_cast<unsigned short>(v4 + j);
                }
        }
        __syncthreads();
    }
    const int active = any ? listed : 0;
    const bool dense = active > min(len, SEG) / DENSE;
    const unsigned long long bo = static_cast<unsigned long long>(b) * A.nb;
    const unsigned char* admit = reinterpret_cast<const unsigned char*>(A.admit);
    auto mask_row = [&](int m) { return admit + static_cast<long long>(m) * (4ll * A.W); };
    // the adjusted logit of the segment's token v in row i
    auto adjusted = [&](float y, int v, int i) {
        const unsigned c = cnt[v];
        unsigned num = c & COUNT;
        if ((c & DRAFT) != 0)
            for (int j = 0; j < i; ++j) num += drafts[j] == v;
        if ((c & SEEN) != 0 || num > 0) y = y > 0.0f ? y / rep : y * rep;
        if (num > 0) y = y - freq * static_cast<float>(num) - pres;
        if constexpr (BIAS) {
            if ((c & BIASED) != 0) {
                if (!dup) {
                    y += A.bias_val[bo + own[v]];
                } else {
                    float bias = 0.0f;
                    for (int j = 0; j < A.nb; ++j)
                        if (A.bias_tok[bo + j] == v0 + v) bias += A.bias_val[bo + j];
                    y += bias;
                }
            }
        }
        return y;
    };
    // the first U of a thread's listed tokens: entry e % active in row e / active
    const int todo = dense ? 0 : rows * active;
    const float share = 1.0f / static_cast<float>(max(active, 1));
    auto entry = [&](int e, int& i, int& v) {
        i = static_cast<int>((static_cast<float>(e) + 0.5f) * share);
        v = e < todo ? list[e - i * active] : 0;
        const int m = e < todo ? mask_of[i] : BROKEN;
        return m == OPEN || (m >= 0 && (mask_row(m)[(v0 + v) >> 3] >> ((v0 + v) & 7) & 1));
    };
    float early[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        int i, v;
        early[u] = 0.0f;
        if (t + u * NTJ < todo && entry(t + u * NTJ, i, v)) early[u] = I::one(A.in, (row0 + i) * A.V + v0 + v);
    }
    bool first = !A.inplace;
    for (Item it = it0; it.row < rows; first = false) {
        unsigned bits[U];
        Item at[U];
        int m[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            at[u] = it;
            bits[u] = 0;
            m[u] = OPEN;
            if (it.row >= rows) continue;
            m[u] = uniform(mask_of[it.row]);
            if (!first && (!A.inplace || m[u] != OPEN || dense)) x[u] = load(it);
            const int v = token(it);
            if (m[u] >= 0 && v + VE <= len) bits[u] = admit_bits<VE>(mask_row(m[u]), v0 + v, whole);
            advance(it);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = token(at[u]);
            if (at[u].row >= rows || v + VE > len || (A.inplace && m[u] == OPEN && !dense)) continue;
            char* out = A.out + row_at(at[u].row) * EO + static_cast<unsigned>(v) * EO;
            if (m[u] == BROKEN) {
                put_vec<I, OF, false>(out, u32x4{I::NANS, I::NANS, I::NANS, I::NANS}, 0);
            } else if (dense) {
                float y[VE];
                unpack<I>(x[u], y);
#pragma unroll
                for (int j = 0; j < VE; ++j) {
                    if (cnt[v + j] != 0) y[j] = adjusted(y[j], v + j, at[u].row);
                    if (m[u] >= 0 && !((bits[u] >> j) & 1)) y[j] = -INFINITY;
                }
                put_floats<I, OF>(out, y);
            } else if (m[u] >= 0) {
                put_vec<I, OF, true>(out, x[u], bits[u]);
            } else {
                put_vec<I, OF, false>(out, x[u], 0);
            }
        }
    }
    // the elements before and behind the vectors (all of them where the tensors are not
    // 16-byte aligned), with their adjustment
    const int ends = A.vec ? 2 * VE : len;
    for (int e = t; e < rows * ends; e += NTJ) {
        const int i = e / ends, m = mask_of[i];
        const int head = A.vec ? min(len, static_cast<int>(-row_at(i) & (VE - 1))) : len;
        const int tail = (len - head) / VE * VE + head;    // the first behind the vectors
        const int v = e % ends < head ? e % ends : tail + (e % ends - head);
        if (v >= len || (A.inplace && m == OPEN && !dense)) continue;
        const bool ok = m < 0 || (mask_row(m)[(v0 + v) >> 3] >> ((v0 + v) & 7) & 1);
        float y = m == BROKEN ? NAN : ok ? I::one(A.in, row_at(i) + v) : -INFINITY;
        if (dense && ok && m != BROKEN && cnt[v] != 0) y = adjusted(y, v, i);
        put_one<I, OF>(A.out, row_at(i) + v, y);
    }
    if (todo == 0) return;
    __builtin_amdgcn_s_waitcnt(0);                         // the stores above land before those below
    __syncthreads();
    for (int e0 = t; e0 < todo; e0 += U * NTJ) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int i, v;
            const int e = e0 + u * NTJ;
            if (e >= todo || !entry(e, i, v)) continue;
            const long long n = (row0 + i) * A.V + v0 + v;
            put_one<I, OF>(A.out, n, adjusted(e0 == t ? early[u] : I::one(A.in, n), v, i));
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
    if (C.ks[2] > (1 << 27) || C.vs[2] > (1 << 27))
        return fail(SPEC_ERR_SHAPE, "a cache's tokens are more than 2^27 bytes apart");
    C.k = const_cast<char*>(static_cast<const char*>(k_cache));
    C.v = const_cast<char*>(static_cast<const char*>(v_cache));
    C.table = table; C.kv_len = kv_len; C.draft_len = draft_len;
    C.k_scale = k_scale; C.v_scale = v_scale;
    C.pages = pages; C.max_pages = max_pages;
    C.shift = __builtin_ctz(static_cast<unsigned>(page_size));
    C.B = B; C.R = R; C.Hkv = Hkv;
    return SPEC_OK;
}

// Row blocks, ranges and workspace of an attention call.
struct AttnPlan {
    int M, MB, MT, M16, W, one;
    bool rows;                 // the waves share the query rows (else the keys)
    size_t slots_at, bytes;
};

template <int D, bool E4M3>
int attn_occupancy(bool rows, int MT) {
    if constexpr (E4M3 && D < 256) {
        if (!rows && MT == 3) return AttnShape<D, 3, E4M3, false>::OCC;
    }
    if (!rows) return MT == 1 ? AttnShape<D, 1, E4M3, false>::OCC : AttnShape<D, 2, E4M3, false>::OCC;
    if constexpr (D < 256) {
        if (MT == 3) return AttnShape<D, 3, E4M3, true>::OCC;
    }
    return MT == 1 ? AttnShape<D, 1, E4M3, true>::OCC : AttnShape<D, 2, E4M3, true>::OCC;
}

AttnPlan attn_plan(int B, int R, int Hq, int Hkv, int D, bool e4m3, int page_size, int max_pages) {
    AttnPlan p;
    p.M = R * (Hq / Hkv);
    const int tiles = (p.M + 15) / 16;
    // Up to 32 query rows the waves take keys each, beyond that rows each: accumulators for 48
    // rows leave a wave of 16-bit keys too few registers (R * G = 40, 16 rows of 8192 keys,
    // bfloat16: 104.8 us by rows, 110.1 by keys with some queries in LDS). The exception are
    // 8-bit caches, which every wave widens for itself: by rows that is four times the work
    // (R * G = 40, 131071 keys: 74 us by rows, 65 by keys).
    p.rows = tiles > (e4m3 && D < 256 ? 3 : 2);
    p.MB = 1;
    p.MT = tiles;
    if (p.rows) {
        const int most = NWQ * (D == 256 ? 2 : 3);
        p.MB = (tiles + most - 1) / most;
        p.MT = (tiles + NWQ * p.MB - 1) / (NWQ * p.MB);
    }
    p.M16 = 16 * p.MT * (p.rows ? NWQ : 1);
    // one resident round, but no more ranges than there can be units
    const int lanes = Hkv * p.MB;
    const int occ = D == 64 ? (e4m3 ? attn_occupancy<64, true>(p.rows, p.MT) : attn_occupancy<64, false>(p.rows, p.MT))
                  : D == 128 ? (e4m3 ? attn_occupancy<128, true>(p.rows, p.MT) : attn_occupancy<128, false>(p.rows, p.MT))
                             : (e4m3 ? attn_occupancy<256, true>(p.rows, p.MT) : attn_occupancy<256, false>(p.rows, p.MT));
    long long w = CUS * occ / lanes;
    const long long units = B * ((static_cast<long long>(max_pages) * page_size + 2 * TT + TU - 1) / TU);
    if (w > units) w = units;
    p.W = w < 1 ? 1 : static_cast<int>(w);
    p.one = (CUS + lanes - 1) / lanes < p.W ? (CUS + lanes - 1) / lanes : p.W;
    p.slots_at = (p.W * sizeof(RangeRec) + 255) & ~static_cast<size_t>(255);
    p.bytes = p.slots_at + static_cast<size_t>(lanes) * p.W * 2 * p.M16 * (D + 2) * sizeof(float);
    p.bytes = p.W == 1 ? 256 : (p.bytes + 255) & ~static_cast<size_t>(255);
    return p;
}

template <class T, int D, bool E4M3>
void launch_attn_m(const AttnParams& A, const AttnPlan& p, unsigned grid, hipStream_t s) {
    if (!p.rows) {
        if constexpr (E4M3 && D < 256) {
            if (p.MT == 3) {
                hipLaunchKernelGGL((attn_kernel<T, D, 3, E4M3, false>), dim3(grid), dim3(NTQ), 0, s, A);
                return;
            }
        }
        if (p.MT == 1) hipLaunchKernelGGL((attn_kernel<T, D, 1, E4M3, false>), dim3(grid), dim3(NTQ), 0, s, A);
        else hipLaunchKernelGGL((attn_kernel<T, D, 2, E4M3, false>), dim3(grid), dim3(NTQ), 0, s, A);
        return;
    }
    if constexpr (D < 256) {
        if (p.MT == 3) {
            hipLaunchKernelGGL((attn_kernel<T, D, 3, E4M3, true>), dim3(grid), dim3(NTQ), 0, s, A);
            return;
        }
    }
    if (p.MT == 1) hipLaunchKernelGGL((attn_kernel<T, D, 1, E4M3, true>), dim3(grid), dim3(NTQ), 0, s, A);
    else hipLaunchKernelGGL((attn_kernel<T, D, 2, E4M3, true>), dim3(grid), dim3(NTQ), 0, s, A);
}

template <class T, int D>
void launch_attn_d(const AttnParams& A, const AttnPlan& p, bool e4m3, unsigned grid, hipStream_t s) {
    if (e4m3) launch_attn_m<T, D, true>(A, p, grid, s);
    else launch_attn_m<T, D, false>(A, p, grid, s);
}

template <class T>
int launch_attn(AttnParams& A, const AttnPlan& p, bool e4m3, hipStream_t s) {
    const long long x = static_cast<long long>(A.W) * A.c.Hkv;
    const long long grid = (x + 7) / 8 * 8 * A.MB;
    if (grid > (1ll << 31) - 1) return fail(SPEC_ERR_SHAPE, "R * Hq is too large");
    if (A.D == 64) launch_attn_d<T, 64>(A, p, e4m3, static_cast<unsigned>(grid), s);
    else if (A.D == 128) launch_attn_d<T, 128>(A, p, e4m3, static_cast<unsigned>(grid), s);
    else launch_attn_d<T, 256>(A, p, e4m3, static_cast<unsigned>(grid), s);
    const int rc = launched();
    if (rc != SPEC_OK || A.W == 1) return rc;              // one range: nothing crosses
    const int rows = NTQ / (A.D / 4) / A.slices, groups = (A.M16 + rows - 1) / rows;
    const long long join = static_cast<long long>(A.direct ? A.c.B : A.W - 1) * A.c.Hkv * A.MB * groups;
    hipLaunchKernelGGL((join_kernel<T>), dim3(static_cast<unsigned>(join)), dim3(NTQ), 0, s, A);
    return launched();
}

template <bool BIAS>
void launch_adjust(const AdjustParams& A, int dtype, int out_dtype, unsigned grid, hipStream_t s) {
    if (dtype == SPEC_DTYPE_F32)
        hipLaunchKernelGGL((adjust_kernel<InF32, false, BIAS>), dim3(grid), dim3(NTJ), 0, s, A);
    else if (out_dtype == SPEC_DTYPE_BF16)
        hipLaunchKernelGGL((adjust_kernel<InBf16, false, BIAS>), dim3(grid), dim3(NTJ), 0, s, A);
    else
        hipLaunchKernelGGL((adjust_kernel<InBf16, true, BIAS>), dim3(grid), dim3(NTJ), 0, s, A);
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
    return attn_plan(B, R, Hq, Hkv, D, cache_dtype == SPEC_DTYPE_E4M3, page_size, max_pages).bytes;
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
    if (!(fabsf(scale) <= F32_MAX) || !(softcap >= 0.0f && softcap <= F32_MAX) || window < 0 ||
        (softcap > 0.0f && !(fabsf(scale) / softcap <= 1e30f)))
        return fail(SPEC_ERR_VALUE, "scale must be finite, softcap finite and >= 0 (0, or at least 1e-30 |scale|), "
                    "window >= 0 (got %g, %g, %d)", static_cast<double>(scale), static_cast<double>(softcap), window);
    if (!q || !q_stride || !out) return fail(SPEC_ERR_NULL, "q, its strides or out is NULL");
    if (!aligned(q, 16) || !strides_ok(q_stride, 2, A.qs) || !aligned(out, 16))
        return fail(SPEC_ERR_ALIGN, "q and out must be 16-byte aligned and q's strides multiples of 8 elements");
    if (slopes && !aligned(slopes, 4)) return fail(SPEC_ERR_ALIGN, "slopes is not aligned to its element size");
    const bool e4m3 = cache_dtype == SPEC_DTYPE_E4M3;
    const AttnPlan plan = attn_plan(B, R, Hq, Hkv, D, e4m3, page_size, max_pages);
    if (!workspace || workspace_bytes < plan.bytes)
        return fail(SPEC_ERR_WORKSPACE, "workspace needs %zu bytes (got %zu%s)", plan.bytes, workspace_bytes,
                    workspace ? "" : ", NULL");
    if (!aligned(workspace, 256)) return fail(SPEC_ERR_ALIGN, "workspace must be 256-byte aligned");
    A.q = static_cast<const char*>(q);
    A.slopes = slopes;
    A.out = static_cast<char*>(out);
    A.ws = static_cast<float*>(workspace);
    A.scale = scale; A.softcap = softcap; A.window = window;
    A.Hq = Hq; A.G = Hq / Hkv; A.D = D;
    A.M = plan.M; A.MB = plan.MB; A.M16 = plan.M16; A.W = plan.W; A.one = plan.one;
    A.slots_at = static_cast<long long>(plan.slots_at / sizeof(float));
    A.direct = B < plan.W;
    // a sequence has about W / B pieces (one row of 8192 keys, W = 64: 22.5 us with eight
    // slices, 33 with one)
    A.slices = 1;
    while (A.slices < NTQ / (D / 4) && A.slices * B < plan.W) A.slices *= 2;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return dtype == SPEC_DTYPE_BF16 ? launch_attn<Bf16>(A, plan, e4m3, s) : launch_attn<F16>(A, plan, e4m3, s);
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
    if (H < 0 || H > (1 << 29) - 1 || n_bias < 0 || n_bias > 65536 || n_admit < 0)
        return fail(SPEC_ERR_SHAPE, "need 0 <= H < 2^29, 0 <= n_bias <= 65536, n_admit >= 0 (got %d, %d, %d)", H,
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
    // Segments: as few as fit LDS, then as many more as fill the rounds of resident
    // workgroups that these take, unless reading the history once more per segment would
    // cost more than the logits do.
    const int most = n_bias > 0 ? SEG_MAX_BIAS : SEG_MAX;
    const long long least = (V + most - 1) / most;
    const long long rounds = (B * least + ADJ_SLOTS - 1) / ADJ_SLOTS;
    long long nseg = rounds * ADJ_SLOTS / B;
    const long long line = static_cast<long long>(R) * V * static_cast<long long>(es + eo);
    if (H > 0 && nseg > line / (2ll * H)) nseg = line / (2ll * H);
    if (nseg > (V + SEG_MIN - 1) / SEG_MIN) nseg = (V + SEG_MIN - 1) / SEG_MIN;
    if (nseg < least) nseg = least;
    A.seg = static_cast<int>(((V + nseg - 1) / nseg + 63) / 64 * 64);
    A.nseg = (V + A.seg - 1) / A.seg;
    const long long grid = static_cast<long long>(B) * A.nseg;
    if (grid > (1ll << 31) - 1) return fail(SPEC_ERR_SHAPE, "B * V is too large");
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (n_bias > 0) launch_adjust<true>(A, dtype, out_dtype, static_cast<unsigned>(grid), s);
    else launch_adjust<false>(A, dtype, out_dtype, static_cast<unsigned>(grid), s);
    return launched();
}

const char* spec_forward_last_error(void) { return g_err; }

}  // extern "C"
