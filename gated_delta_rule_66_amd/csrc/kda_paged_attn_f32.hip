// Attention over a paged cache in full precision: fp32 tokens, the cache fp32
// or in 8 bits.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i.k_j - max_i),  j <= position of i
//
// Bound by its products: 32x32x2 fp32, a sixteenth of the bf16 rate, 64 cycles
// each.  That leaves so much time for loads that nothing of the cache is shared
// through LDS, and a tile can be 32 rows (tokens times the heads that share a
// cache head): a workgroup's four waves take blocks of 32 positions in turn and
// keep maximum, sum and output of their own, joined at the end.  (128 rows, 32 a
// wave, and blocks shared in LDS left ragged batches with too few workgroups: 16
// sequences x 5 heads of 64, 184 us; now 116, 79 TFLOP/s, half of a large library
// product; 8 x 512 over 4K, heads of 64, 106 TFLOP/s.  Eight waves: 142 us; 64 rows a
// workgroup: 132; two accumulators a product: no change.)
//   * S^T = K Q^T, the row in the lane: lane half h holds neighbouring channels
//     of one position, one 16-byte load; their order is free if Q has the same.
//   * O^T = V^T P^T: a result register of S^T, position 8 (e / 4) + 4 h + e % 4,
//     is the operand P^T as it stands.  A lane loads D / 32 neighbouring channels
//     of a position (32 lanes read a whole row); product j makes channels
//     (D / 32) rho + j, rho the accumulator's row.
#include "kda_paged_attn.h"

#include <type_traits>

namespace kda {

namespace {

__device__ __forceinline__ f32x16 mma2(f32x16 acc, float a, float b) {
    return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, acc, 0, 0, 0);
}

// One block of 32 positions as it is loaded, in two halves of one page each.
// Places without a position get what the page, or page 0, holds there.
template <int KV, int D> struct BlockF {
    static constexpr int E = KV == kKvF32 ? 4 : 1, RB = D * E;
    static constexpr int CH = 16 / E;               // channels of K a load
    static constexpr int KL = D / (2 * CH);         // loads of K a lane
    static constexpr int DV = D / 32;               // channels of V a lane
    static constexpr bool CODES = KV >= kKvE4m3;
    u32x4 k[KL];
    typedef typename std::conditional<CODES, typename std::conditional<DV == 4, unsigned, unsigned short>::type,
                                      typename std::conditional<DV == 4, f32x4, float2>::type>::type Vec;
    Vec v[16];
    unsigned ks, vs[4];     // scale bytes: K's row of the lane, V's sixteen rows
    int pg[2];

    __device__ __forceinline__ void find(const PagedCache& c, PageWalk<true>& w, int pos, int end) {
#pragma unroll
        for (int h = 0; h < 2; ++h) pg[h] = pos + 16 * h < end ? w.page((pos + 16 * h) >> c.lg_page) : -1;
    }
    __device__ __forceinline__ int valid() const { return (pg[0] >= 0) | (pg[1] >= 0) << 1; }
    __device__ __forceinline__ static size_t row(const PagedCache& c, int hk, int at) {
        return ((size_t)hk << c.lg_page) + (at & ((1 << c.lg_page) - 1));
    }
    __device__ __forceinline__ void load_k(const PagedCache& c, int hk, int pos, int lane) {
        // the lane's half of the block
        const int half = lane >> 4 & 1;
        const size_t page = (size_t)max(half ? pg[1] : pg[0], 0), r = row(c, hk, pos + 16 * half) + (lane & 15);
        const char* at = c.k + page * c.k_page + r * RB + (lane >> 5) * 16;
#pragma unroll
        for (int i = 0; i < KL; ++i) k[i] = *reinterpret_cast<const u32x4*>(at + 32 * i);
        if constexpr (CODES) ks = (c.ks + ((page * c.Hk) << c.lg_page))[r];
    }
    __device__ __forceinline__ void load_v(const PagedCache& c, int hk, int pos, int lane) {
        const unsigned off = (unsigned)((lane >> 5) * 4 * RB + (lane & 31) * DV * E);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const size_t page = (size_t)max(pg[h], 0), r = row(c, hk, pos + 16 * h);
            const char* at = c.v + page * c.v_page + r * RB;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[8 * h + e] = *reinterpret_cast<const Vec*>(at + (8 * (e >> 2) + (e & 3)) * RB + off);
            if constexpr (CODES) {
                const unsigned char* s = c.vs + ((page * c.Hk) << c.lg_page) + r + 4 * (lane >> 5);
                vs[2 * h] = *reinterpret_cast<const unsigned*>(s);
                vs[2 * h + 1] = *reinterpret_cast<const unsigned*>(s + 8);
            }
        }
    }
    // channels 2 CH i + CH h + 4 w .. of the lane's position
    __device__ __forceinline__ void kvals(int i, int w, float (&o)[4]) const {
        if constexpr (CODES)
            Codes<KV>(ks).f32(k[i][w], o);
        else
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = __uint_as_float(k[i][j]);
    }
    // channels DV (l % 32) .. of operand e's position
    __device__ __forceinline__ void vvals(int e, float (&o)[DV]) const {
        if constexpr (CODES) {
            float f[4];
            Codes<KV>(vs[e >> 2] >> (8 * (e & 3)) & 255u).f32((unsigned)v[e], f);
#pragma unroll
            for (int j = 0; j < DV; ++j) o[j] = f[j];
        } else {
            __builtin_memcpy(o, &v[e], sizeof(o));
        }
    }
};

template <int KV, int D> __global__ __launch_bounds__(256, D == 64 ? 2 : 1) void kda_attn_f32_kernel(AttnParams p) {
    typedef BlockF<KV, D> Block;
    constexpr int R = 32, DV = Block::DV, CH = Block::CH, KL = Block::KL, LD = D + 4;
    __shared__ __align__(16) float lds_o[2][R][LD];
    __shared__ float lds_ml[2][R][2];
    AttnTile t;
    if (!t.init(p, blockIdx.x)) return;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), h = lane >> 5, c32 = lane & 31;
    const int r = t.r0 + c32, tok = p.by_g.div(r), head = t.hk * p.G + r - tok * p.G;
    const int lim = t.limit(r, p), lim_first = t.limit(t.r0, p);
    // Q in the order of Block::kvals, zeros behind the sequence's rows
    f32x4 q[D / 8];
    const char* row = p.q + (size_t)(t.first + tok) * p.q_stride + (size_t)head * D * 4;
#pragma unroll
    for (int i = 0; i < KL; ++i)
#pragma unroll
        for (int w = 0; w < CH / 4; ++w) {
            q[i * (CH / 4) + w] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (r < t.rows) q[i * (CH / 4) + w] = *reinterpret_cast<const f32x4*>(row + (2 * CH * i + CH * h + 4 * w) * 4);
        }
    f32x16 acc[DV];
#pragma unroll
    for (int j = 0; j < DV; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[j][e] = 0.f;
    float m = -INFINITY, l = 0.f;
    const float c = p.c_log2, lazy = kLazy / c;

    int bad_from = -1;      // the wave's first block of V with a value taken out
    int pos = t.lo + 32 * wave;
    if (pos < t.hi) {
        PageWalk<true> walk;
        walk.init(p.c, t.seq, t.L, t.lo >> p.c.lg_page);
        Block b;
        b.find(p.c, walk, pos, t.hi);
        b.load_k(p.c, t.hk, pos, lane);
        b.load_v(p.c, t.hk, pos, lane);
        for (; pos < t.hi; pos += 128) {
            f32x16 s;
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] = 0.f;
#pragma unroll
            for (int i = 0; i < KL; ++i)
#pragma unroll
                for (int w = 0; w < CH / 4; ++w) {
                    float f[4];
                    b.kvals(i, w, f);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s = mma2(s, f[j], q[i * (CH / 4) + w][j]);
                }
            const int valid = b.valid(), next = pos + 128;
            const bool masked = pos + 31 > lim_first || valid != 3;
            if (next < t.hi) {
                b.find(p.c, walk, next, t.hi);
                b.load_k(p.c, t.hk, next, lane);
            }
            if (masked) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (pos + 8 * (e >> 2) + 4 * h + (e & 3) > lim || !(valid >> (e >> 3) & 1)) s[e] = -INFINITY;
            }
            float top = s[0];
#pragma unroll
            for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
            if (__any(top > m + lazy)) {
                const float mn = fmaxf(m, fmaxf(top, __shfl_xor(top, 32)));
                const float a = mn == -INFINITY ? 1.f : fast_exp2((m - mn) * c);
                m = mn;
                l *= a;
#pragma unroll
                for (int j = 0; j < DV; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[j][e] *= a;
            }
            const float mc = m == -INFINITY ? 0.f : m * c;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                s[e] = fast_exp2(fmaf(s[e], c, -mc));
                l += s[e];
            }
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                float f[DV];
                b.vvals(e, f);
                if (masked) {       // what is not finite must not meet a weight of zero
#pragma unroll
                    for (int j = 0; j < DV; ++j) {
                        // (what stands in for a place that is not there is no row's to have back)
                        bad |= !finite_f(f[j]) && (valid >> (e >> 3) & 1);
                        f[j] = finite_f(f[j]) ? f[j] : 0.f;
                    }
                }
#pragma unroll
                for (int j = 0; j < DV; ++j) acc[j] = mma2(acc[j], f[j], s[e]);
            }
            if (masked && bad_from < 0 && __any(bad)) bad_from = pos;
            if (next < t.hi) b.load_v(p.c, t.hk, next, lane);
        }
    }
    if (bad_from >= 0) {
#pragma unroll 1
        for (int i = bad_from; i < t.hi; i += i % 32 == 31 ? 97 : 1)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                // DV channels from a multiple of DV on, within one load of four
                const int ch = DV * (8 * (e >> 2) + 4 * h + (e & 3));
                float f[4];
                load_v4<KV, D>(p.c, t.seq, t.hk, i, ch & ~3, f);
#pragma unroll
                for (int j = 0; j < DV; ++j) {
                    const float x = DV == 4 ? f[j] : (e & 1) ? f[2 + j] : f[j];
                    if (i <= lim && !finite_f(x)) acc[j][e] += x;
                }
            }
    }
    l += __shfl_xor(l, 32);
    // waves 2 and 3 join 0 and 1, then 1 joins 0
#pragma unroll
    for (int half = 2; half > 0; half >>= 1) {
        if (wave >= half && wave < 2 * half) {
            if (h == 0) {
                lds_ml[wave - half][c32][0] = m;
                lds_ml[wave - half][c32][1] = l;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e)
#pragma unroll
                for (int j = 0; j < DV; ++j)
                    lds_o[wave - half][c32][DV * (8 * (e >> 2) + 4 * h + (e & 3)) + j] = acc[j][e];
        }
        __syncthreads();
        if (wave < half) {
            const float mo = lds_ml[wave][c32][0], lo = lds_ml[wave][c32][1], mn = fmaxf(m, mo);
            const float a = m == mn ? 1.f : fast_exp2((m - mn) * c);
            const float b = mo == mn ? 1.f : fast_exp2((mo - mn) * c);
            m = mn;
            l = l * a + lo * b;
#pragma unroll
            for (int e = 0; e < 16; ++e)
#pragma unroll
                for (int j = 0; j < DV; ++j)
                    acc[j][e] = acc[j][e] * a + lds_o[wave][c32][DV * (8 * (e >> 2) + 4 * h + (e & 3)) + j] * b;
        }
        __syncthreads();
    }
    if (wave || r >= t.rows) return;
    const size_t col = (size_t)head * D;
    const bool parts = t.splits > 1;
    float* o = parts ? p.part + (t.unit * R + c32) * D : reinterpret_cast<float*>(p.o) + (size_t)(t.first + tok) * p.H * D + col;
    const float* z = reinterpret_cast<const float*>(p.z + (size_t)(t.first + tok) * p.z_stride) + col;
    if (parts && h == 0) {
        p.ml[(t.unit * R + c32) * 2] = m;
        p.ml[(t.unit * R + c32) * 2 + 1] = l;
    }
#pragma unroll
    for (int e = 0; e < 16; e += 4 / DV) {
        const int d = DV * (8 * (e >> 2) + 4 * h + (e & 3));
        f32x4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = acc[i % DV][e + i / DV];
        if (!parts) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[i] = l == 0.f ? 0.f : y[i] / l;
                if (p.z) y[i] = gate_of<float>(y[i], z[d + i]);
            }
        }
        *reinterpret_cast<f32x4*>(o + d) = y;
    }
}

template <int D> hipError_t launch_f32_kv(int kv, const AttnParams& p, int grid, hipStream_t st) {
    if (kv == kKvE4m3)
        kda_attn_f32_kernel<kKvE4m3, D><<<grid, 256, 0, st>>>(p);
    else if (kv == kKvI8)
        kda_attn_f32_kernel<kKvI8, D><<<grid, 256, 0, st>>>(p);
    else
        kda_attn_f32_kernel<kKvF32, D><<<grid, 256, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_f32(int kv, int D, const AttnParams& p, int grid, hipStream_t st) {
    return D == 128 ? launch_f32_kv<128>(kv, p, grid, st) : launch_f32_kv<64>(kv, p, grid, st);
}

}  // namespace kda
