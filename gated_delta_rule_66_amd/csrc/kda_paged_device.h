// Device helpers of the paged cache operators.
#pragma once

#include "kda_mixer_device.h"
#include "kda_paged.h"

namespace kda {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const char* uniform(const char* p) {
    const unsigned long long v = reinterpret_cast<uintptr_t>(p);
    const unsigned lo = (unsigned)uniform((int)(unsigned)v), hi = (unsigned)uniform((int)(unsigned)(v >> 32));
    return reinterpret_cast<const char*>((unsigned long long)hi << 32 | lo);
}

// ---- 8-bit codes --------------------------------------------------------------------
// A row's scale is 2^(byte - 127), so that a code times its scale is exact in
// fp32 and, with at most seven significant bits, in bf16.
// 255 stands for NaN; 0 for 2^-127, which is subnormal.
__device__ __forceinline__ float scale_of(unsigned byte) {
    const unsigned bits = byte == 255u ? 0x7fc00000u : byte == 0u ? 0x00400000u : byte << 23;
    return __uint_as_float(bits);
}
__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
    bf16x2 r;
    r[0] = (bf16)a;
    r[1] = (bf16)b;
    return __builtin_bit_cast(unsigned, r);
}
// Four codes of a dword as bf16: two conversions for e4m3 (which take the
// scale's exponent along), four and two roundings that round nothing for int8.
// A NaN scale makes every e4m3 code its NaN first: what the conversion makes of
// such a scale is not relied on.
template <int KV> struct Codes;
template <> struct Codes<kKvE4m3> {
    float s;
    unsigned nan;
    __device__ __forceinline__ explicit Codes(unsigned byte) {
        nan = byte == 255u ? 0x7f7f7f7fu : 0u;
        s = byte == 255u ? 1.f : scale_of(byte);
    }
    __device__ __forceinline__ void bf(unsigned c, unsigned* o) const {
        c |= nan;
        o[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, false));
        o[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, true));
    }
    __device__ __forceinline__ void f32(unsigned c, float* o) const {
        c |= nan;
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
        o[0] = a[0] * s;
        o[1] = a[1] * s;
        o[2] = b[0] * s;
        o[3] = b[1] * s;
    }
};
template <> struct Codes<kKvI8> {
    float s;
    __device__ __forceinline__ explicit Codes(unsigned byte) { s = scale_of(byte); }
    __device__ __forceinline__ void f32(unsigned c, float* o) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = (float)(int)(signed char)(c >> (8 * i)) * s;
    }
    __device__ __forceinline__ void bf(unsigned c, unsigned* o) const {
        float f[4];
        f32(c, f);
        o[0] = pack_bf16(f[0], f[1]);
        o[1] = pack_bf16(f[2], f[3]);
    }
};

// ---- sequences and pages -------------------------------------------------------------
// first token row and tokens of sequence i; offsets outside the contract are clamped
__device__ __forceinline__ void seq_span(const SeqView& sv, int i, int* first, int* n) {
    if (sv.cu) {
        *first = min(max(sv.cu[i], 0), sv.T);
        *n = max(min(sv.cu[i + 1], sv.T) - *first, 0);
    } else {
        *first = i * sv.T;
        *n = sv.T;
    }
}
// positions of sequence i, at most what its table's row holds; none without pages
__device__ __forceinline__ int seq_positions(const PagedCache& c, int i) {
    return c.pages > 0 ? min(max(c.lens[i], 0), c.blocks << c.lg_page) : 0;
}

// A wave's page numbers along a sequence: lane l holds entry at + l of the
// table's row.  AHEAD: the 64 entries behind are in flight; without, they are
// waited for where they are needed, so that no load is open in the loop (the
// compiler would wait for it, and for all that came after it, in every pass).
template <bool AHEAD> struct PageWalk {
    const int* row;
    int entries;            // entries that hold positions
    int pages;
    int at, here, ahead;
    __device__ __forceinline__ int entry(int i) const {
        return i < entries ? row[i] : -1;
    }
    __device__ __forceinline__ void init(const PagedCache& c, int seq, int positions, int first) {
        row = c.table + (long long)seq * c.table_stride;
        entries = (positions + (1 << c.lg_page) - 1) >> c.lg_page;
        pages = c.pages;
        at = first;
        here = entry(at + (int)(threadIdx.x & 63));
        if constexpr (AHEAD)
            ahead = entry(at + 64 + (int)(threadIdx.x & 63));
        else
            __builtin_amdgcn_s_waitcnt(0x0f70);         // vmcnt(0)
    }
    // page of entry i, i not below those asked before by more than the lanes hold; -1: not there
    __device__ __forceinline__ int page(int i) {
        while (i >= at + 64) {
            at += 64;
            if constexpr (AHEAD) {
                here = ahead;
                ahead = entry(at + 64 + (int)(threadIdx.x & 63));
            } else {
                here = entry(at + (int)(threadIdx.x & 63));
                __builtin_amdgcn_s_waitcnt(0x0f70);
            }
        }
        const int pg = __builtin_amdgcn_readlane(here, i - at);
        return (unsigned)pg < (unsigned)pages ? pg : -1;
    }
};

}  // namespace kda
