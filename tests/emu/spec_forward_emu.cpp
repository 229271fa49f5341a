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

#include "../../token_verification_amd/csrc/spec_forward.hip"

extern "C" unsigned spec_forward_emu_e4m3(float x) { return emu_e4m3_code(x); }
