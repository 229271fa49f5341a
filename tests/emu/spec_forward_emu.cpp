// Host build of the spec_forward library source for the CPU emulation tests.
// TEST INFRASTRUCTURE ONLY: compiled with host clang++ against tests/emu/hip/hip_runtime.h,
// plus the few builtins that only spec_forward.hip uses, by their documented meaning.
#include "hip/hip_runtime.h"

typedef __bf16 emu_bf16x2 __attribute__((ext_vector_type(2)));

extern "C" __bf16 __truncsfbf2(float f) {                  // nearest even; NaN stays NaN
    uint32_t u;
    memcpy(&u, &f, 4);
    uint16_t h;
    if (f != f) h = static_cast<uint16_t>((u >> 16) | 0x40);
    else h = static_cast<uint16_t>((u + 0x7fff + ((u >> 16) & 1)) >> 16);
    __bf16 r;
    memcpy(&r, &h, 2);
    return r;
}

// e4m3 (OCP): 4 exponent bits of bias 7, 3 mantissa bits, no infinities, S.1111.111 = NaN
inline float emu_e4m3_value(unsigned c) {
    const int e = (c >> 3) & 15, m = c & 7;
    if (e == 15 && m == 7) return NAN;
    const float v = e ? ldexpf(1.0f + static_cast<float>(m) / 8.0f, e - 7) : ldexpf(static_cast<float>(m), -9);
    return c & 128 ? -v : v;
}
inline unsigned emu_e4m3_code(float x) {                   // |x| <= 448 or NaN (what the kernels pass)
    if (x != x) return 0x7f;
    const unsigned s = std::signbit(x) ? 128u : 0u;
    const float a = fabsf(x);
    int e;
    frexpf(a, &e);                                         // a = f 2^e, f in [0.5, 1)
    const int q = a < ldexpf(1.0f, -6) ? -9 : e - 4;       // exponent of one step
    const float n = nearbyintf(ldexpf(a, -q));             // ties to even
    const float r = ldexpf(n, q);
    if (r == 0.0f) return s;
    frexpf(r, &e);
    if (r < ldexpf(1.0f, -6)) return s | static_cast<unsigned>(ldexpf(r, 9));
    return s | static_cast<unsigned>((e - 1 + 7) << 3) | (static_cast<unsigned>(ldexpf(r, 4 - e)) & 7);
}
inline int emu_cvt_pk_fp8_f32(float a, float b, int old, bool hi) {
    const unsigned p = emu_e4m3_code(a) | emu_e4m3_code(b) << 8;
    const unsigned o = static_cast<unsigned>(old);
    return static_cast<int>(hi ? (o & 0xffffu) | p << 16 : (o & 0xffff0000u) | p);
}
#define __builtin_amdgcn_cvt_pk_fp8_f32 emu_cvt_pk_fp8_f32
inline emu_bf16x2 emu_cvt_bf16_fp8(int w, float, bool hi) {
    const unsigned p = static_cast<unsigned>(w) >> (hi ? 16 : 0);
    return emu_bf16x2{static_cast<__bf16>(emu_e4m3_value(p & 255)), static_cast<__bf16>(emu_e4m3_value((p >> 8) & 255))};
}
#define __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8 emu_cvt_bf16_fp8

typedef _Float16 emu_f16x2 __attribute__((ext_vector_type(2)));
inline emu_f16x2 emu_cvt_f16_fp8(int w, float, bool hi) {
    const unsigned p = static_cast<unsigned>(w) >> (hi ? 16 : 0);
    return emu_f16x2{static_cast<_Float16>(emu_e4m3_value(p & 255)), static_cast<_Float16>(emu_e4m3_value((p >> 8) & 255))};
}
#define __builtin_amdgcn_cvt_scalef32_pk_f16_fp8 emu_cvt_f16_fp8
#define __builtin_amdgcn_readlane(v, l) __shfl((v), (l), 64)
inline float emu_rcpf(float x) { return 1.0f / x; }
#define __builtin_amdgcn_rcpf emu_rcpf

// 16-byte load with the LDS as destination: lane l's bytes land at the (wave-uniform) address + 16 l
template <class G, class L>
inline void emu_global_load_lds(G src, L dst, unsigned size, unsigned off, unsigned) {
    unsigned char* d = (unsigned char*)(dst) + off + static_cast<size_t>(threadIdx.x & 63u) * size;
    memcpy(d, (const unsigned char*)(src), size);
}
#define __builtin_amdgcn_global_load_lds emu_global_load_lds

// Transposing LDS reads over groups of 16 lanes: of a 4 x 16 matrix of 16-bit values
// whose row r's four 8-byte pieces are at the addresses of lanes 4 r .. 4 r + 3, lane i
// gets column i; likewise 8 x 16 bytes with two pieces a row.
template <class P>
inline const unsigned char* emu_lane_address(P p, unsigned lane) {
    EmuWG* w = emu_wg;
    const unsigned char* a = (const unsigned char*)(p);
    const unsigned me = threadIdx.x;
    memcpy(w->shfl[me], &a, 8);
    emu_wave_sync();
    memcpy(&a, w->shfl[(me & ~63u) + lane], 8);
    return a;
}
typedef short emu_i16x4 __attribute__((ext_vector_type(4)));
typedef int emu_i32x2 __attribute__((ext_vector_type(2)));
template <class P>
inline emu_i16x4 emu_read_tr16(P p) {
    const unsigned lane = threadIdx.x & 63u, i = lane & 15u;
    emu_i16x4 r;
    for (unsigned j = 0; j < 4; ++j) {
        short v;
        memcpy(&v, emu_lane_address(p, (lane & ~15u) + 4 * j + i / 4) + 2 * (i % 4), 2);
        r[j] = v;
        emu_wave_sync();
    }
    return r;
}
#define __builtin_amdgcn_ds_read_tr16_b64_v4i16 emu_read_tr16
template <class P>
inline emu_i32x2 emu_read_tr8(P p) {
    const unsigned lane = threadIdx.x & 63u, i = lane & 15u;
    unsigned char r[8];
    for (unsigned j = 0; j < 8; ++j) {
        r[j] = emu_lane_address(p, (lane & ~15u) + 2 * j + i / 8)[i % 8];
        emu_wave_sync();
    }
    emu_i32x2 o;
    memcpy(&o, r, 8);
    return o;
}
#define __builtin_amdgcn_ds_read_tr8_b64_v2i32 emu_read_tr8

// v_mfma_f32_16x16x32: A(i, k) is element k % 8 of lane i + 16 (k / 8)'s a, B(k, j) of lane
// j + 16 (k / 8)'s b, and D(i, j) register i % 4 of lane j + 16 (i / 4).
typedef float emu_f32x4 __attribute__((ext_vector_type(4)));
template <class V>
inline emu_f32x4 emu_mfma16(V a, V b, emu_f32x4 c, int, int, int) {
    EmuWG* w = emu_wg;
    const unsigned me = threadIdx.x, base = me & ~63u, lane = me & 63u;
    memcpy(w->mfa[me], &a, 16);
    memcpy(w->mfb[me], &b, 16);
    emu_wave_sync();
    emu_f32x4 d = c;
    for (unsigned r = 0; r < 4; ++r) {
        float s = 0.0f;
        for (unsigned k = 0; k < 32; ++k) {
            V x, y;
            memcpy(&x, w->mfa[base + 4 * (lane / 16) + r + 16 * (k / 8)], 16);
            memcpy(&y, w->mfb[base + lane % 16 + 16 * (k / 8)], 16);
            s += static_cast<float>(x[k % 8]) * static_cast<float>(y[k % 8]);
        }
        d[r] += s;
    }
    emu_wave_sync();
    return d;
}
#define __builtin_amdgcn_mfma_f32_16x16x32_bf16 emu_mfma16
#define __builtin_amdgcn_mfma_f32_16x16x32_f16 emu_mfma16

#include "../../token_verification_amd/csrc/spec_forward.hip"

extern "C" unsigned spec_forward_emu_e4m3(float x) { return emu_e4m3_code(x); }
