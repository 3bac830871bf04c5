// Attention over a paged cache in full precision: fp32 tokens, the cache fp32
// or in 8 bits.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i.k_j - max_i),  j <= position of i
//
// Bound by its products: 32x32x2 fp32, a sixteenth of the bf16 rate.  The
// layout is that of the bf16 kernel (the row in the lane, S^T = K Q^T, O^T =
// V^T P^T): a workgroup of four waves takes 128 rows and walks tiles of 32
// positions, which the threads hold in registers while the tile before is
// multiplied.
#include "kda_paged_attn.h"

namespace kda {

namespace {

constexpr int kTileF = 32;

__device__ __forceinline__ f32x16 mma2(f32x16 acc, float a, float b) {
    return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, acc, 0, 0, 0);
}

template <int KV, int D> struct StageF {
    static constexpr int E = KV == kKvF32 ? 4 : 1;
    static constexpr int W = KV == kKvF32 ? 4 : 1;  // dwords of a thread's four values
    static constexpr int PIECES = D / 4;            // threads of a row
    static constexpr int N = kTileF * PIECES / 256; // pieces of a thread
    unsigned w[N][W];
    unsigned s[N];
    __device__ __forceinline__ void load(const PagedCache& c, const char* base, const unsigned char* scale,
                                         size_t page_bytes, PageWalk<true>& walk, int hk, int pos, int end, int tid) {
        constexpr int PER = 256 / PIECES, WPER = 64 / PIECES;       // rows of a load, of a wave's part
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = uniform(pos + i * PER + (tid >> 6) * WPER), page = at < end ? walk.page(at >> c.lg_page) : -1;
            const size_t r = ((size_t)hk << c.lg_page) + (at & ((1 << c.lg_page) - 1));
            const auto rs = make_rsrc_n(base + (size_t)max(page, 0) * page_bytes + r * D * E,
                                        page < 0 ? 0u : (unsigned)(min(end - at, WPER) * D * E));
            if constexpr (KV == kKvF32) {
                const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rs, (tid & 63) * 16, 0, 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) w[i][k] = v[k];
            } else {
                w[i][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, (tid & 63) * 4, 0, 0);
                const auto ss = make_rsrc_n(scale + (((size_t)max(page, 0) * c.Hk) << c.lg_page) + r, page < 0 ? 0u : (unsigned)WPER);
                s[i] = __builtin_amdgcn_raw_buffer_load_b8(ss, (tid & 63) / PIECES, 0, 0);
            }
        }
    }
    template <int LD> __device__ __forceinline__ void store(float* tile, int tid) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = i * (256 / PIECES) + tid / PIECES, d = 4 * (tid % PIECES);
            float f[4];
            if constexpr (KV == kKvF32) {
#pragma unroll
                for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(w[i][k]);
            } else {
                Codes<KV>(s[i]).f32(w[i][0], f);
            }
            *reinterpret_cast<f32x4*>(tile + row * LD + d) = f32x4{f[0], f[1], f[2], f[3]};
        }
    }
};

template <int KV, int D> __global__ __launch_bounds__(256, 1) void kda_attn_f32_kernel(AttnParams p) {
    constexpr int KS = D / 8, DB = D / 32, M = 128, LD = D + 4;
    __shared__ __align__(16) float lds_k[kTileF * LD];
    __shared__ __align__(16) float lds_v[kTileF * LD];
    __shared__ int lds_bad;                         // the first tile of V with a value taken out, or -1
    AttnTile t;
    if (!t.init(p, blockIdx.x)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), h = lane >> 5;
    const int r = t.r0 + 32 * wave + (lane & 31), tok = p.by_g.div(r), head = t.hk * p.G + r - tok * p.G;
    const int lim = t.limit(r, p);
    const int w0 = t.r0 + 32 * wave, lim_first = t.limit(w0, p), t_first = t.limit(t.r0, p);
    const int lim_last = w0 < t.rows ? t.limit(min(w0 + 31, t.rows - 1), p) : -1;
    // operand 4 s + i: channels 8 s + 4 h + i
    f32x4 q[KS];
    const char* row = p.q + (size_t)(t.first + tok) * p.q_stride + (size_t)head * D * 4;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        q[s] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (r < t.rows) q[s] = *reinterpret_cast<const f32x4*>(row + (8 * s + 4 * h) * 4);
    }
    f32x16 acc[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[db][e] = 0.f;
    float m = -INFINITY, l = 0.f;
    const float c = p.c_log2, lazy = kLazy / c;

    PageWalk<true> walk;
    walk.init(p.c, t.seq, t.L, t.lo >> p.c.lg_page);
    StageF<KV, D> sk, sv;
    if (t.lo < t.hi) {
        sk.load(p.c, p.c.k, p.c.ks, p.c.k_page, walk, t.hk, t.lo, t.hi, tid);
        sv.load(p.c, p.c.v, p.c.vs, p.c.v_page, walk, t.hk, t.lo, t.hi, tid);
    }
    if (tid == 0) lds_bad = -1;
    for (int pos = t.lo; pos < t.hi; pos += kTileF) {
        int valid = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = pos + 16 * i;
            valid |= (at < t.hi && walk.page(at >> p.c.lg_page) >= 0) << i;
        }
        sk.template store<LD>(lds_k, tid);
        sv.template store<LD>(lds_v, tid);
        __syncthreads();
        if (pos + kTileF - 1 > t_first || valid != 3) {      // for a row of the tile's
            bool bad = false;
            for (int i = tid; i < kTileF * D; i += 256) {
                float* y = lds_v + i / D * LD + i % D;
                if (!finite_f(*y)) {
                    *y = 0.f;
                    bad = true;
                }
            }
            if (bad && lds_bad < 0) lds_bad = pos;
            __syncthreads();
        }
        if (pos + kTileF < t.hi) {
            sk.load(p.c, p.c.k, p.c.ks, p.c.k_page, walk, t.hk, pos + kTileF, t.hi, tid);
            sv.load(p.c, p.c.v, p.c.vs, p.c.v_page, walk, t.hk, pos + kTileF, t.hi, tid);
        }
        if (pos <= lim_last) {
            f32x16 s;
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const f32x4 kf = *reinterpret_cast<const f32x4*>(lds_k + (lane & 31) * LD + 8 * k + 4 * h);
#pragma unroll
                for (int i = 0; i < 4; ++i) s = mma2(s, kf[i], q[k][i]);
            }
            const bool masked = pos + kTileF - 1 > lim_first || valid != 3;
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
                for (int db = 0; db < DB; ++db)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[db][e] *= a;
            }
            const float mc = m == -INFINITY ? 0.f : m * c;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                s[e] = fast_exp2(fmaf(s[e], c, -mc));
                l += s[e];
            }
            // operand e: positions 8 (e / 4) + 4 h + e % 4
            const float* v = lds_v + 4 * h * LD + (lane & 31);
#pragma unroll
            for (int e = 0; e < 16; ++e)
#pragma unroll
                for (int db = 0; db < DB; ++db) acc[db] = mma2(acc[db], v[(8 * (e >> 2) + (e & 3)) * LD + 32 * db], s[e]);
        }
        __syncthreads();
    }
    if (lds_bad >= 0) mend_rows<KV, D>(acc, p, t, lds_bad, lim, h);
    l += __shfl_xor(l, 32);
    if (r >= t.rows) return;
    if (t.splits > 1) {
        const size_t x = t.unit * M + 32 * wave + (lane & 31);
        float* po = p.part + x * D;
        if (h == 0) {
            p.ml[x * 2] = m;
            p.ml[x * 2 + 1] = l;
        }
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<f32x4*>(po + 32 * db + 8 * j + 4 * h) =
                    f32x4{acc[db][4 * j], acc[db][4 * j + 1], acc[db][4 * j + 2], acc[db][4 * j + 3]};
        return;
    }
    float* o = reinterpret_cast<float*>(p.o) + ((size_t)(t.first + tok) * p.H + head) * D;
    const float* z = reinterpret_cast<const float*>(p.z + (size_t)(t.first + tok) * p.z_stride) + (size_t)head * D;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = 32 * db + 8 * j + 4 * h;
            f32x4 x;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = l == 0.f ? 0.f : acc[db][4 * j + i] / l;
            if (p.z) {
                const f32x4 zz = *reinterpret_cast<const f32x4*>(z + d);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = gate_of<float>(x[i], zz[i]);
            }
            *reinterpret_cast<f32x4*>(o + d) = x;
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
