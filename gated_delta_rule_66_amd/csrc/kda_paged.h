// Host-side declarations of the paged cache operators (writing and reading a
// paged cache of keys and values, attention over it): launch parameters and
// launchers.  The contracts are in include/kda.h.
#pragma once

#include "kda_mixer.h"

namespace kda {

// kda_kv_dtype
enum { kKvF32 = 0, kKvBf16 = 1, kKvE4m3 = 2, kKvI8 = 3 };

// Quotients of 0 <= n < 2^31 by a divisor that the host knows: with
// 2^(s-1) < d <= 2^s and m = floor(2^32 (2^s - d) / d) + 1,
// n / d = (n m / 2^32 + n) >> s, and the sum stays below 2^32.
struct FastDiv {
    unsigned m, s, d;
    void set(unsigned by) {
        d = by;
        for (s = 0; s < 31 && (1u << s) < by; ++s) {}
        m = (unsigned)(((1ull << 32) * ((1ull << s) - by)) / by + 1);
    }
    __host__ __device__ int div(int n) const {
#ifdef __HIP_DEVICE_COMPILE__
        return (int)((__umulhi((unsigned)n, m) + (unsigned)n) >> s);
#else
        return (int)(((((unsigned long long)(unsigned)n * m) >> 32) + (unsigned)n) >> s);
#endif
    }
};

// The cache as the kernels see it.  Sequence i's position j is in row
// j % page of page table[i][j / page]; a page outside [0, pages) is not there.
struct PagedCache {
    char* k;                // [pages][Hk][page][D], pages k_page bytes apart
    char* v;
    unsigned char* ks;      // [pages][Hk][page] scale exponents, 8-bit caches
    unsigned char* vs;
    size_t k_page, v_page;  // bytes
    const int* table;       // [N][blocks], rows table_stride apart
    long long table_stride;
    const int* lens;        // [N]
    int pages, blocks, lg_page, Hk;
};

// tokens [first, first + n) of a sequence are its last n positions
struct CacheIoParams {
    SeqView sv;
    PagedCache c;
    char* k;                // token rows [tokens][Hk][D]
    char* v;
    size_t k_stride, v_stride;  // bytes between token rows
    int M;                  // token rows
    int heads_per_block;
};
hipError_t launch_cache_write(int dtype, int kv, int D, const CacheIoParams& p, int token_blocks, int head_blocks,
                              hipStream_t st);
hipError_t launch_cache_read(int dtype, int kv, int D, const CacheIoParams& p, int token_blocks, int head_blocks,
                             hipStream_t st);

// ---- attention ---------------------------------------------------------------------
// Rows of a sequence: (token t, head g of its group) -> t G + g.  A tile is M
// consecutive rows of one sequence; packed sequences own the tile slots
// floor(cu[i] G / M) + i on (never fewer than they have tiles).
// A tile's positions may be split into `splits` ranges of split_len; a tile of
// more than one non-empty range leaves unnormalised parts that a second launch
// joins.
enum AttnKind { kAttnStep16, kAttnStep32, kAttnChunk, kAttnF32, kAttnChunk256 };
struct AttnParams {
    SeqView sv;
    PagedCache c;
    const char* q;          // [tokens][H][D]
    const char* z;          // gate or null
    char* o;
    size_t q_stride, z_stride;  // bytes between token rows
    int H, G;
    float c_log2;           // scale log2(e)
    int M, lg_m;            // rows a tile
    int tiles, tiles_per_seq;
    int splits, split_len;
    int by_length;          // tiles in order of their sequences' positions (N at most 64)
    FastDiv by_g, by_hk, by_splits, by_tiles, by_len, by_h, by_t;   // G, Hk, splits, tiles_per_seq, split_len, H, T
    float* part;            // [tiles][Hk][splits][M][D]
    float* ml;              // [tiles][Hk][splits][M][2]: running maximum (of q.k) and sum
};
hipError_t launch_attn(AttnKind kind, int kv, int D, const AttnParams& p, hipStream_t st);
hipError_t launch_attn_step(AttnKind kind, int kv, int D, const AttnParams& p, int grid, hipStream_t st);
hipError_t launch_attn_chunk(AttnKind kind, int kv, int D, const AttnParams& p, int grid, hipStream_t st);
hipError_t launch_attn_f32(int kv, int D, const AttnParams& p, int grid, hipStream_t st);
hipError_t launch_attn_join(int dtype, int D, const AttnParams& p, int M_tokens, hipStream_t st);

}  // namespace kda
