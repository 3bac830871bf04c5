// Writing the keys and values of new tokens into a paged cache, as they are or
// in 8 bits, and reading them back.
//
// 8 bits: a row (one token's D values of one head) is held as codes c and the
// exponent of a power of two: x ~ c 2^e, e the smallest with
// max |x| <= L 2^e, L the largest code (e4m3: 448, int8: 127).  Scaling by a
// power of two is exact, so a code is x 2^-e rounded once, and what is read
// back or multiplied later is c 2^e itself: seven significant bits at most, in
// bf16 too.  (A scale of max / L fills int8's range better, by half a bit on
// average, but every product with it is rounded; an e4m3 code has the same
// relative step under either.)
//
// Memory bound.  A block takes 16 consecutive tokens and some heads: a team of
// D / 8 lanes takes one token's row of one head, eight values a lane, so that
// the table is looked up once for all heads, and 16 tokens of a head write 16
// consecutive rows of a page, and 16 neighbouring scale bytes.
// Measured: 8K tokens x 32 heads of 128 from bf16 to e4m3 46 us, 4.4 TB/s (floor 39
// at a large copy's rate); eight prefixes of up to 32K x 8 heads from e4m3 back to
// bf16 146 us, 5.05 TB/s (floor 144); one token of 256 sequences 3.6 us, in a call of 10.5.
// As they are: 8K tokens x 32 heads of 128 written in bf16 57 us (floor 52.5), in fp32
// 105 (105); 8 x 16K tokens x 8 heads read in bf16 211 us (210), in fp32 434 (420).
#include "kda_paged.h"
#include "kda_paged_device.h"

namespace kda {

namespace {

constexpr int kIoTokens = 16;

// The team's token: its sequence, and page and row of its position.
__device__ __forceinline__ bool token_place(const CacheIoParams& p, int t, int* page, int* row) {
    int seq, first, n;
    if (p.sv.cu) {
        if (t < p.sv.cu[0] || t >= p.sv.cu[p.sv.N]) return false;       // no sequence's
        int lo = 0, hi = p.sv.N;        // cu[lo] <= t < cu[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.sv.cu[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        seq = lo;
    } else {
        seq = t / p.sv.T;
    }
    seq_span(p.sv, seq, &first, &n);
    if ((unsigned)(t - first) >= (unsigned)n) return false;     // offsets outside the contract
    const int pos = seq_positions(p.c, seq) - n + (t - first);
    *page = -1;
    *row = 0;
    if (pos >= 0) {
        const int pg = p.c.table[(long long)seq * p.c.table_stride + (pos >> p.c.lg_page)];
        if ((unsigned)pg < (unsigned)p.c.pages) *page = pg;
        *row = pos & ((1 << p.c.lg_page) - 1);
    }
    return true;
}

// maximum over a team of 8 or 16 neighbouring lanes
template <int TEAM> __device__ __forceinline__ unsigned team_max(unsigned v) {
    v = max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, false));      // lane ^ 1
    v = max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, false));      // lane ^ 2
    v = max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, false));     // 7 - lane of eight
    if constexpr (TEAM == 16) v = max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xf, 0xf, false));
    return v;
}

// Codes of a team's row.  most: the largest bits of |x|, so that infinities
// and NaN, whose bits are above every number's, show.
template <int KV> __device__ __forceinline__ u32x2 encode(const float* x, unsigned most, unsigned* byte) {
    // biased exponent of the smallest power of two with most <= L 2^e: L is
    // 1.75 2^8 or 1.984375 2^6, so e is most's own exponent - 8 or - 6, and one
    // more where its fraction is above L's.
    constexpr unsigned frac = KV == kKvE4m3 ? 0x600000u : 0x7e0000u, below = KV == kKvE4m3 ? 8 : 6;
    const int e = max((int)((most + 0x7fffffu - frac) >> 23) - (int)below, 10);
    u32x2 r = {0u, 0u};
    if (most >= 0x7f800000u) {
        *byte = 255u;
        return r;
    }
    *byte = (unsigned)e;
    const float inv = __uint_as_float((unsigned)(254 - e) << 23);       // 2^-(e - 127)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        if constexpr (KV == kKvE4m3) {
            unsigned c = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * w] * inv, x[4 * w + 1] * inv, 0, false);
            c = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * w + 2] * inv, x[4 * w + 3] * inv, c, true);
            r[w] = c;
        } else {
            unsigned c = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) c |= ((unsigned)(int)rintf(x[4 * w + i] * inv) & 255u) << (8 * i);
            r[w] = c;
        }
    }
    return r;
}

// A lane's eight values, held as the compiler's own vectors: HIP's uint4 and
// float4 are structs, and the loops below, which keep a row from one turn to the
// next, kept it in scratch memory (the fp32 read above took 851 us, the bf16 one 277).
template <typename T> struct Eight {
    static constexpr int N = sizeof(T) / 2;
    u32x4 w[N];
    __device__ __forceinline__ void load(const char* p) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const u32x4*>(p)[i];
    }
    __device__ __forceinline__ void store(char* p) const {
#pragma unroll
        for (int i = 0; i < N; ++i) reinterpret_cast<u32x4*>(p)[i] = w[i];
    }
    __device__ __forceinline__ void to_f32(float* x) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (N == 1)
                x[i] = __uint_as_float(i & 1 ? w[0][i / 2] & 0xffff0000u : w[0][i / 2] << 16);
            else
                x[i] = __uint_as_float(w[i / 4][i % 4]);
        }
    }
};

template <typename T, int KV, int D>
__device__ __forceinline__ void write_row(const Eight<T>& x, char* cache, unsigned char* scale, size_t page_bytes,
                                          int Hk, int lg_page, int page, int h, int row, int lane) {
    constexpr int E = KV == kKvF32 ? 4 : KV == kKvBf16 ? 2 : 1, TEAM = D / 8;
    const size_t r = ((size_t)h << lg_page) + row;
    char* to = cache + (size_t)page * page_bytes + (r * D + lane * 8) * E;
    if constexpr (KV <= kKvBf16) {
        x.store(to);
    } else {
        float f[8];
        x.to_f32(f);
        unsigned most = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(f[i]) & 0x7fffffffu);
        most = team_max<TEAM>(most);
        unsigned byte;
        const u32x2 c = encode<KV>(f, most, &byte);
        *reinterpret_cast<u32x2*>(to) = c;
        if (lane == 0) scale[(((size_t)page * Hk) << lg_page) + r] = (unsigned char)byte;
    }
}

template <typename T, int KV, int D> __global__ __launch_bounds__(kIoTokens * D / 8) void kda_cache_write_kernel(CacheIoParams p) {
    constexpr int TEAM = D / 8;
    const int lane = threadIdx.x % TEAM, t = blockIdx.x * kIoTokens + threadIdx.x / TEAM;
    int page, row;
    if (t >= p.M || !token_place(p, t, &page, &row) || page < 0) return;       // whole teams
    const int h0 = blockIdx.y * p.heads_per_block, h1 = min(h0 + p.heads_per_block, p.c.Hk);
    const char* k = p.k + (size_t)t * p.k_stride + lane * 8 * sizeof(T);
    const char* v = p.v + (size_t)t * p.v_stride + lane * 8 * sizeof(T);
    // a head's rows are on their way while those before are written
    Eight<T> nk, nv;
    nk.load(k + (size_t)h0 * D * sizeof(T));
    nv.load(v + (size_t)h0 * D * sizeof(T));
    for (int h = h0; h < h1; ++h) {
        const Eight<T> xk = nk, xv = nv;
        if (h + 1 < h1) {
            nk.load(k + (size_t)(h + 1) * D * sizeof(T));
            nv.load(v + (size_t)(h + 1) * D * sizeof(T));
        }
        write_row<T, KV, D>(xk, p.c.k, p.c.ks, p.c.k_page, p.c.Hk, p.c.lg_page, page, h, row, lane);
        write_row<T, KV, D>(xv, p.c.v, p.c.vs, p.c.v_page, p.c.Hk, p.c.lg_page, page, h, row, lane);
    }
}

// A lane's part of a row of the cache, as it is loaded and as it is read.
template <typename T, int KV, int D> struct Row {
    static constexpr int E = KV == kKvF32 ? 4 : KV == kKvBf16 ? 2 : 1;
    Eight<T> x;             // codes: not used
    u32x2 c;
    unsigned byte;
    __device__ __forceinline__ void load(const char* cache, const unsigned char* scale, size_t page_bytes, int Hk,
                                         int lg_page, int page, int h, int row, int lane) {
        const size_t r = ((size_t)h << lg_page) + row;
        const char* from = cache + (size_t)page * page_bytes + (r * D + lane * 8) * E;
        if constexpr (KV <= kKvBf16) {
            x.load(from);
        } else {
            c = *reinterpret_cast<const u32x2*>(from);
            byte = scale[(((size_t)page * Hk) << lg_page) + r];
        }
    }
    __device__ __forceinline__ void store(T* to) const {
        if constexpr (KV <= kKvBf16) {
            x.store(reinterpret_cast<char*>(to));
        } else {
            const Codes<KV> d(byte);
            if constexpr (sizeof(T) == 2) {
                unsigned o[4];
                d.bf(c[0], o);
                d.bf(c[1], o + 2);
                *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
                float o[8];
                d.f32(c[0], o);
                d.f32(c[1], o + 4);
                st8(to, o);
            }
        }
    }
};

template <typename T, int KV, int D> __global__ __launch_bounds__(kIoTokens * D / 8) void kda_cache_read_kernel(CacheIoParams p) {
    constexpr int TEAM = D / 8;
    const int lane = threadIdx.x % TEAM, t = blockIdx.x * kIoTokens + threadIdx.x / TEAM;
    int page, row;
    if (t >= p.M || !token_place(p, t, &page, &row)) return;
    const int h0 = blockIdx.y * p.heads_per_block, h1 = min(h0 + p.heads_per_block, p.c.Hk);
    T* k = reinterpret_cast<T*>(p.k + (size_t)t * p.k_stride) + lane * 8;
    T* v = reinterpret_cast<T*>(p.v + (size_t)t * p.v_stride) + lane * 8;
    if (page < 0) {
        const float zero[8] = {};
        for (int h = h0; h < h1; ++h) {
            st8(k + (size_t)h * D, zero);
            st8(v + (size_t)h * D, zero);
        }
        return;
    }
    Row<T, KV, D> nk, nv;
    nk.load(p.c.k, p.c.ks, p.c.k_page, p.c.Hk, p.c.lg_page, page, h0, row, lane);
    nv.load(p.c.v, p.c.vs, p.c.v_page, p.c.Hk, p.c.lg_page, page, h0, row, lane);
    for (int h = h0; h < h1; ++h) {
        const Row<T, KV, D> xk = nk, xv = nv;
        if (h + 1 < h1) {
            nk.load(p.c.k, p.c.ks, p.c.k_page, p.c.Hk, p.c.lg_page, page, h + 1, row, lane);
            nv.load(p.c.v, p.c.vs, p.c.v_page, p.c.Hk, p.c.lg_page, page, h + 1, row, lane);
        }
        xk.store(k + (size_t)h * D);
        xv.store(v + (size_t)h * D);
    }
}

template <typename T, int KV, int D>
hipError_t launch_io(bool write, const CacheIoParams& p, dim3 grid, hipStream_t st) {
    if (write)
        kda_cache_write_kernel<T, KV, D><<<grid, kIoTokens * D / 8, 0, st>>>(p);
    else
        kda_cache_read_kernel<T, KV, D><<<grid, kIoTokens * D / 8, 0, st>>>(p);
    return hipGetLastError();
}
template <typename T, int D> hipError_t launch_kv(bool write, int kv, const CacheIoParams& p, dim3 grid, hipStream_t st) {
    if (kv == kKvE4m3) return launch_io<T, kKvE4m3, D>(write, p, grid, st);
    if (kv == kKvI8) return launch_io<T, kKvI8, D>(write, p, grid, st);
    return launch_io<T, sizeof(T) == 2 ? kKvBf16 : kKvF32, D>(write, p, grid, st);
}
hipError_t launch_any(bool write, int dtype, int kv, int D, const CacheIoParams& p, dim3 grid, hipStream_t st) {
    if (dtype) return D == 128 ? launch_kv<bf16, 128>(write, kv, p, grid, st) : launch_kv<bf16, 64>(write, kv, p, grid, st);
    return D == 128 ? launch_kv<float, 128>(write, kv, p, grid, st) : launch_kv<float, 64>(write, kv, p, grid, st);
}

}  // namespace

hipError_t launch_cache_write(int dtype, int kv, int D, const CacheIoParams& p, int token_blocks, int head_blocks,
                              hipStream_t st) {
    return launch_any(true, dtype, kv, D, p, dim3(token_blocks, head_blocks), st);
}
hipError_t launch_cache_read(int dtype, int kv, int D, const CacheIoParams& p, int token_blocks, int head_blocks,
                             hipStream_t st) {
    return launch_any(false, dtype, kv, D, p, dim3(token_blocks, head_blocks), st);
}

}  // namespace kda
