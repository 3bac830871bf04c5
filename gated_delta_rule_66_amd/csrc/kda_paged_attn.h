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
        const int u = p.by_hk.div(block), v = p.by_splits.div(u);
        hk = block - u * p.c.Hk;
        split = u - v * p.splits;
        int at;
        if (p.by_length) {
            if (!longest_first(p, v, &at)) return false;
        } else {
            const int tile = p.tiles - 1 - v;       // a sequence's long tiles first
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
            } else {
                seq = p.by_tiles.div(tile);
            }
            at = tile - slot(p, seq);
        }
        seq_span(p.sv, seq, &first, &n);
        first = uniform(first);
        n = uniform(n);
        rows = n * p.G;
        if (at < 0 || ((long long)at << p.lg_m) >= rows) return false;
        r0 = at << p.lg_m;
        L = uniform(seq_positions(p.c, seq));
        end = max(L - n + p.by_g.div(min(r0 + p.M, rows) - 1) + 1, 0);
        splits = end > 0 ? p.by_len.div(end - 1) + 1 : 1;
        if (split >= splits) return false;
        lo = split * p.split_len;
        hi = min(end, lo + p.split_len);
        unit = ((size_t)(slot(p, seq) + at) * p.c.Hk + hk) * p.splits + split;
        return true;
    }
    // The v-th tile of the sequences in order of their positions, most first:
    // workgroups then take the long tiles first and the short ones fill the end.
    // Lane i counts the tiles of the sequences before its own, the i-th.
    __device__ __forceinline__ bool longest_first(const AttnParams& p, int v, int* at) {
        const int i = (int)(threadIdx.x & 63);
        int f = 0, m = 0, len = -1;
        if (i < p.sv.N) {
            seq_span(p.sv, i, &f, &m);
            len = seq_positions(p.c, i);
        }
        const int tiles = (m * p.G + p.M - 1) >> p.lg_m;
        int before = 0;
        for (int j = 0; j < p.sv.N; ++j) {
            const int lj = __builtin_amdgcn_readlane(len, j), tj = __builtin_amdgcn_readlane(tiles, j);
            before += lj > len || (lj == len && j < i) ? tj : 0;
        }
        const unsigned long long mine = __ballot(i < p.sv.N && v >= before && v < before + tiles);
        if (!mine) return false;
        seq = uniform(__ffsll(mine) - 1);
        *at = __builtin_amdgcn_readlane(before + tiles, seq) - 1 - v;
        return true;
    }
    // the first tile slot of sequence i
    static __device__ __forceinline__ int slot(const AttnParams& p, int i) {
        if (!p.sv.cu) return i * p.tiles_per_seq;
        const int c = uniform(min(max(p.sv.cu[i], 0), p.sv.T));
        return ((c * p.G) >> p.lg_m) + i;
    }
    // the last position that row r sees; below zero: none
    __device__ __forceinline__ int limit(int r, const AttnParams& p) const { return r < rows ? L - n + p.by_g.div(r) : -1; }
};

// sigmoid gate of one value
template <typename T> __device__ __forceinline__ float gate_of(float o, float z) { return o * sigmoid_of<T>(z); }

// ---- values of V that are not finite ---------------------------------------------------
// A place that a row does not see has weight zero, and zero times NaN or an
// infinity is NaN.  Where some row of a tile does not see all of it (and where a
// weight has two parts), such values are therefore made zero before the product,
// and afterwards added to the rows that do see them (mend_rows).  A second addition
// changes nothing, so the mending may go over positions whose values were left in.
__device__ __forceinline__ bool not_finite(unsigned pair) {
    return (pair & 0x7f80u) == 0x7f80u || (pair & 0x7f800000u) == 0x7f800000u;
}
// some value of a block's pairs: the largest exponents
template <int A, int B> __device__ __forceinline__ bool not_finite(const unsigned (&pairs)[A][B]) {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u16x2 top = {0, 0};
#pragma unroll
    for (int a = 0; a < A; ++a)
#pragma unroll
        for (int b = 0; b < B; ++b)
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, pairs[a][b] & 0x7f807f80u));
    return not_finite(__builtin_bit_cast(unsigned, top));
}
__device__ __forceinline__ unsigned clean(unsigned pair) {
    return ((pair & 0x7f80u) == 0x7f80u ? 0u : pair & 0xffffu) | ((pair & 0x7f800000u) == 0x7f800000u ? 0u : pair & 0xffff0000u);
}
__device__ __forceinline__ bool finite_f(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }

// Four neighbouring channels of V at a position; zeros where it is not there.
template <int KV, int D>
__device__ __forceinline__ void load_v4(const PagedCache& c, int seq, int hk, int pos, int ch, float* f) {
    const int pg = c.table[(long long)seq * c.table_stride + (pos >> c.lg_page)];
    f[0] = f[1] = f[2] = f[3] = 0.f;
    if ((unsigned)pg >= (unsigned)c.pages) return;
    const size_t r = ((size_t)hk << c.lg_page) + (pos & ((1 << c.lg_page) - 1));
    const char* at = c.v + (size_t)pg * c.v_page;
    if constexpr (KV == kKvF32) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(at + (r * D + ch) * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = v[i];
    } else if constexpr (KV == kKvBf16) {
        const bf16x4 v = *reinterpret_cast<const bf16x4*>(at + (r * D + ch) * 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = (float)v[i];
    } else {
        const Codes<KV> d(c.vs[(((size_t)pg * c.Hk) << c.lg_page) + r]);
        d.f32(*reinterpret_cast<const unsigned*>(at + r * D + ch), f);
    }
}
// acc[db][4 j + i]: channel 32 db + 8 j + 4 h + i of the lane's row
template <int KV, int D>
__device__ __forceinline__ void mend_rows(f32x16 (&acc)[D / 32], const AttnParams& p, const AttnTile& t, int from, int lim, int h) {
#pragma unroll 1
    for (int pos = from; pos < t.hi; ++pos)
#pragma unroll
        for (int db = 0; db < D / 32; ++db)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float f[4];
                load_v4<KV, D>(p.c, t.seq, t.hk, pos, 32 * db + 8 * j + 4 * h, f);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (pos <= lim && !finite_f(f[i])) acc[db][4 * j + i] += f[i];
            }
}

// A score's maximum is moved only when a tile passes it by more than this many
// powers of two: weights stay below 2^8, sums below 2^8 times the positions.
constexpr float kLazy = 8.f;

}  // namespace kda
