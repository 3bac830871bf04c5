// Device parts that the attention kernels share: tiles, roundings, outputs.
#pragma once

#include "kda_paged_device.h"

namespace kda {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// One workgroup's tile of rows and its range of positions.
struct AttnTile {
    int seq, first, n;      // its sequence: first token row, tokens
    int hk, split;
    int r0, rows;           // rows of the sequence: the tile's first, the sequence's number
    int L;                  // positions of the sequence
    int end;                // positions that the tile's last row sees
    int splits;             // non-empty ranges of the tile
    int lo, hi;             // this workgroup's range
    size_t unit;            // its place in the parts
    // false: nothing to do
    __device__ __forceinline__ bool init(const AttnParams& p, int block) {
        hk = block % p.c.Hk;
        const int u = block / p.c.Hk;
        split = u % p.splits;
        const int tile = p.tiles - 1 - u / p.splits;        // a sequence's long tiles first
        int at;
        if (p.sv.cu) {
            int a = 0, b = p.sv.N;      // slot(a) <= tile < slot(b)
            while (b - a > 1) {
                const int mid = (a + b) >> 1;
                if (slot(p, mid) <= tile)
                    a = mid;
                else
                    b = mid;
            }
            seq = uniform(a);
            at = tile - slot(p, seq);
        } else {
            seq = tile / p.tiles_per_seq;
            at = tile - seq * p.tiles_per_seq;
        }
        seq_span(p.sv, seq, &first, &n);
        first = uniform(first);
        n = uniform(n);
        rows = n * p.G;
        if (at < 0 || (long long)at * p.M >= rows) return false;
        r0 = at * p.M;
        L = uniform(seq_positions(p.c, seq));
        end = max(L - n + (min(r0 + p.M, rows) - 1) / p.G + 1, 0);
        splits = end > 0 ? (end - 1) / p.split_len + 1 : 1;
        if (split >= splits) return false;
        lo = split * p.split_len;
        hi = min(end, lo + p.split_len);
        unit = ((size_t)tile * p.c.Hk + hk) * p.splits + split;
        return true;
    }
    static __device__ __forceinline__ int slot(const AttnParams& p, int i) {
        const int c = uniform(min(max(p.sv.cu[i], 0), p.sv.T));
        return (int)((long long)c * p.G / p.M) + i;
    }
    // the last position that row r sees; below zero: none
    __device__ __forceinline__ int limit(int r, int G) const { return r < rows ? L - n + r / G : -1; }
};

// sigmoid gate of one value
template <typename T> __device__ __forceinline__ float gate_of(float o, float z) { return o * sigmoid_of<T>(z); }

// A masked place of V that is not a number or infinite must not reach a row
// through its weight of zero.  Such values are taken out of V (clean), and the
// rows that do see them get them back as what two products of ones count:
// places of +inf or NaN, and of -inf or NaN.
__device__ __forceinline__ bool not_finite(unsigned pair) {
    return (pair & 0x7f80u) == 0x7f80u || (pair & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ unsigned clean_half(unsigned h) { return (h & 0x7f80u) == 0x7f80u ? 0u : h; }
__device__ __forceinline__ unsigned clean(unsigned pair) {
    return clean_half(pair & 0xffffu) | clean_half(pair >> 16) << 16;
}
// bf16 one where the half is NaN or the infinity of this sign
__device__ __forceinline__ unsigned flag_half(unsigned h, unsigned inf) {
    return h == inf || ((h & 0x7f80u) == 0x7f80u && (h & 0x7fu)) ? 0x3f80u : 0u;
}
__device__ __forceinline__ unsigned flag(unsigned pair, unsigned inf) {
    return flag_half(pair & 0xffffu, inf) | flag_half(pair >> 16, inf) << 16;
}
template <class F> __device__ __forceinline__ bf16x8 map_pairs(bf16x8 v, F&& f) {
    u32x4 u = __builtin_bit_cast(u32x4, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = f(u[i]);
    return __builtin_bit_cast(bf16x8, u);
}
__device__ __forceinline__ bf16x8 clean8(bf16x8 v) {
    return map_pairs(v, [](unsigned x) { return clean(x); });
}
__device__ __forceinline__ bf16x8 flag8(bf16x8 v, bool minus) {
    return map_pairs(v, [=](unsigned x) { return flag(x, minus ? 0xff80u : 0x7f80u); });
}
__device__ __forceinline__ float poisoned(float o, float plus, float minus) {
    if (plus > 0.f) o += __uint_as_float(0x7f800000u);
    if (minus > 0.f) o -= __uint_as_float(0x7f800000u);
    return o;
}

// A score's maximum is moved only when a tile passes it by more than this many
// powers of two: weights stay below 2^8, sums below 2^8 times the positions.
constexpr float kLazy = 8.f;

}  // namespace kda
