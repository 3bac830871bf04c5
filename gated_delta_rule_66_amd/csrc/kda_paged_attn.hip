// Attention of chunks of new tokens over a paged cache, bf16.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i.k_j - max_i),  j <= position of i
//
// Bound by its products (4 D flops a pair of row and position).  A workgroup of
// four waves takes 128 rows (tokens times the heads that share a cache head),
// 32 a wave, and walks tiles of 64 positions that all waves share in LDS.
// Products are 32x32x16 with the row in the lane:
//   * S^T = K Q^T: a lane has 32 of a tile's 64 scores of its row, so maximum
//     and sum need no exchange but between two lanes, and that only when the
//     maximum moves;
//   * O^T = V^T P^T: S^T as it sits in the accumulator is the operand P^T if a
//     product's 16 positions are 8 (i / 4) + 4 h + i % 4 (lane half h), which
//     the transposing reads of V deliver as well.
// P is rounded to bf16 for its product (relative 2^-9, as V's own rounding; the
// sum is taken before it), everything else is fp32.
#include "kda_paged_attn.h"

namespace kda {

namespace {

constexpr int kTile = 64;

__device__ __forceinline__ f32x16 mma32(f32x16 acc, bf16x8 a, bf16x8 b) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0);
}

// Rows of a tile in LDS: 16-byte pieces of D bf16, permuted by the row so that
// neither reads of one piece of 16 rows (K) nor transposing reads of two or four
// neighbouring pieces of four rows (V) meet in a bank.
template <int D> __device__ __forceinline__ int k_piece(int row, int piece) {
    return D == 128 ? piece ^ (row & 15) : piece ^ (row >> 1 & 7);
}
template <int D> __device__ __forceinline__ int v_piece(int row, int piece) {
    return D == 128 ? piece ^ ((row & 3) << 2 | (row & 2)) : piece ^ ((row & 3) << 1);
}

// A tile of K or V on its way: what a thread loads of it.
template <int KV, int D> struct Stage {
    static constexpr int E = KV == kKvBf16 ? 2 : 1;
    static constexpr int RB = D * E;                // bytes of a row
    static constexpr int PER = 1024 / RB;           // rows of a wave's load
    static constexpr int N = kTile / (4 * PER);     // loads of a thread
    u32x4 w[N];
    unsigned s[N];
    __device__ __forceinline__ static int row(int i, int wave, int lane) { return (i * 4 + wave) * PER + lane / (64 / PER); }
    __device__ __forceinline__ void load(const PagedCache& c, const char* base, const unsigned char* scale,
                                         size_t page_bytes, PageWalk& walk, int hk, int pos, int end, int wave, int lane) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = pos + (i * 4 + wave) * PER, page = at < end ? walk.page(at >> c.lg_page) : -1;
            const size_t r = ((size_t)hk << c.lg_page) + (at & ((1 << c.lg_page) - 1));
            const auto rs = make_rsrc_n(base + (size_t)max(page, 0) * page_bytes + r * RB,
                                        page < 0 ? 0u : (unsigned)(min(end - at, PER) * RB));
            w[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, lane * 16, 0, 0);
            if constexpr (KV >= kKvE4m3) {
                const auto ss = make_rsrc_n(scale + (((size_t)max(page, 0) * c.Hk) << c.lg_page) + r, page < 0 ? 0u : (unsigned)PER);
                s[i] = __builtin_amdgcn_raw_buffer_load_b8(ss, lane / (64 / PER), 0, 0);
            }
        }
    }
    template <bool V> __device__ __forceinline__ void store(bf16* tile, int wave, int lane) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = row(i, wave, lane), p = lane % (64 / PER);
            u32x4* to = reinterpret_cast<u32x4*>(tile + r * D);
            if constexpr (KV == kKvBf16) {
                to[V ? v_piece<D>(r, p) : k_piece<D>(r, p)] = w[i];
            } else {
                const Codes<KV> d(s[i]);
                unsigned o[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) d.bf(w[i][k], o + 2 * k);
                to[V ? v_piece<D>(r, 2 * p) : k_piece<D>(r, 2 * p)] = u32x4{o[0], o[1], o[2], o[3]};
                to[V ? v_piece<D>(r, 2 * p + 1) : k_piece<D>(r, 2 * p + 1)] = u32x4{o[4], o[5], o[6], o[7]};
            }
        }
    }
};

// K operand: lane: position 32 b + l % 32, channels 16 s + 8 (l / 32) ..
template <int D> __device__ __forceinline__ bf16x8 k_frag(const bf16* tile, int b, int s, int lane) {
    const int r = 32 * b + (lane & 31);
    return *reinterpret_cast<const bf16x8*>(tile + r * D + 8 * k_piece<D>(r, 2 * s + (lane >> 5)));
}
// V operand: lane: channel 32 db + l % 32, positions 16 s + 4 h + i and 16 s + 8 + 4 h + i
template <int D> __device__ __forceinline__ bf16x8 v_frag(const bf16* tile, int db, int s, int lane) {
    const int r = 16 * s + 4 * (lane >> 5) + (lane >> 2 & 3), col = 32 * db + 16 * (lane >> 4 & 1) + 4 * (lane & 3);
    typedef __attribute__((address_space(3))) bf16x4 lds_x4;
    const bf16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_x4*)(tile + r * D + 8 * v_piece<D>(r, col >> 3) + (col & 7)));
    const bf16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
        (lds_x4*)(tile + (r + 8) * D + 8 * v_piece<D>(r + 8, col >> 3) + (col & 7)));
    bf16x8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = a[i];
        f[4 + i] = b[i];
    }
    return f;
}

template <int KV, int D> __global__ __launch_bounds__(256, 2) void kda_attn_chunk_kernel(AttnParams p) {
    constexpr int KS = D / 16, DB = D / 32, M = 128;
    __shared__ __align__(16) bf16 lds_k[2][kTile * D];
    __shared__ __align__(16) bf16 lds_v[2][kTile * D];
    AttnTile t;
    if (!t.init(p, blockIdx.x)) return;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), h = lane >> 5;

    const int r = t.r0 + 32 * wave + (lane & 31), tok = r / p.G, head = t.hk * p.G + r - tok * p.G;
    const int lim = t.limit(r, p.G);
    // the wave's first and last limits
    const int w0 = t.r0 + 32 * wave, lim_first = t.limit(w0, p.G);
    const int lim_last = w0 < t.rows ? t.limit(min(w0 + 31, t.rows - 1), p.G) : -1;
    bf16x8 q[KS];
    const char* row = p.q + (size_t)(t.first + tok) * p.q_stride + (size_t)head * D * 2;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        u32x4 u = {0u, 0u, 0u, 0u};
        if (r < t.rows) u = *reinterpret_cast<const u32x4*>(row + (16 * s + 8 * h) * 2);
        q[s] = __builtin_bit_cast(bf16x8, u);
    }
    f32x16 acc[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[db][e] = 0.f;
    float m = -INFINITY, l = 0.f;
    const float c = p.c_log2, lazy = kLazy / c;

    PageWalk walk;
    walk.init(p.c, t.seq, t.L, t.lo >> p.c.lg_page);
    Stage<KV, D> sk, sv;
    if (t.lo < t.hi) {
        sk.load(p.c, p.c.k, p.c.ks, p.c.k_page, walk, t.hk, t.lo, t.hi, wave, lane);
        sv.load(p.c, p.c.v, p.c.vs, p.c.v_page, walk, t.hk, t.lo, t.hi, wave, lane);
    }
    int buf = 0;
    for (int pos = t.lo; pos < t.hi; pos += kTile, buf ^= 1) {
        sk.template store<false>(lds_k[buf], wave, lane);
        sv.template store<true>(lds_v[buf], wave, lane);
        __syncthreads();
        // which 16 positions have a page
        int valid = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = pos + 16 * i;
            valid |= (at < t.hi && walk.page(at >> p.c.lg_page) >= 0) << i;
        }
        if (pos + kTile < t.hi) {
            sk.load(p.c, p.c.k, p.c.ks, p.c.k_page, walk, t.hk, pos + kTile, t.hi, wave, lane);
            sv.load(p.c, p.c.v, p.c.vs, p.c.v_page, walk, t.hk, pos + kTile, t.hi, wave, lane);
        }
        if (pos > lim_last) continue;       // the wave's rows see nothing of it
        f32x16 s[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int e = 0; e < 16; ++e) s[b][e] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) s[b] = mma32(s[b], k_frag<D>(lds_k[buf], b, k, lane), q[k]);
        }
        const bool masked = pos + kTile - 1 > lim_first || valid != 15;
        if (masked) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int at = 32 * b + 8 * (e >> 2) + 4 * h + (e & 3);
                    if (pos + at > lim || !(valid >> (2 * b + (e >> 3)) & 1)) s[b][e] = -INFINITY;
                }
        }
        float top = s[0][0];
#pragma unroll
        for (int e = 1; e < 16; ++e) top = fmaxf(top, s[0][e]);
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, s[1][e]);
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
        bf16x8 pf[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = fast_exp2(fmaf(s[k >> 1][8 * (k & 1) + i], c, -mc));
                l += x[i];
            }
            pf[k] = frag_from<bf16>(x);
        }
        bool poison = false;
        if (masked) {
            bool bad = false;
            const u32x4* v = reinterpret_cast<const u32x4*>(lds_v[buf]) + lane;
#pragma unroll
            for (int i = 0; i < kTile * D / 512; ++i) {
                const u32x4 x = v[64 * i];
                bad |= not_finite(x[0]) | not_finite(x[1]) | not_finite(x[2]) | not_finite(x[3]);
            }
            poison = __any(bad);
        }
        if (!poison) {
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[db] = mma32(acc[db], v_frag<D>(lds_v[buf], db, k, lane), pf[k]);
        } else {
#pragma unroll 1
            for (int minus = 0; minus < 2; ++minus) {
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    f32x16 n;
#pragma unroll
                    for (int e = 0; e < 16; ++e) n[e] = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float one[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int at = 16 * k + 8 * (i >> 2) + 4 * h + (i & 3);
                            one[i] = pos + at <= lim && (valid >> k & 1) ? 1.f : 0.f;
                        }
                        n = mma32(n, flag8(v_frag<D>(lds_v[buf], db, k, lane), minus), frag_from<bf16>(one));
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[db][e] = poisoned(acc[db][e], minus ? 0.f : n[e], minus ? n[e] : 0.f);
                }
            }
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[db] = mma32(acc[db], clean8(v_frag<D>(lds_v[buf], db, k, lane)), pf[k]);
        }
    }
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
    const float inv = l == 0.f ? 0.f : 1.f / l;
    bf16* o = reinterpret_cast<bf16*>(p.o) + ((size_t)(t.first + tok) * p.H + head) * D;
    const bf16* z = reinterpret_cast<const bf16*>(p.z + (size_t)(t.first + tok) * p.z_stride) + (size_t)head * D;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = 32 * db + 8 * j + 4 * h;
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = acc[db][4 * j + i] * inv;
            if (p.z) {
                const bf16x4 zz = *reinterpret_cast<const bf16x4*>(z + d);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = gate_of<bf16>(x[i], (float)zz[i]);
            }
            st_run<4>(o + d, x);
        }
}

template <int KV, int D> hipError_t launch_chunk_kv(const AttnParams& p, int grid, hipStream_t st) {
    kda_attn_chunk_kernel<KV, D><<<grid, 256, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_chunk(int kv, int D, const AttnParams& p, int grid, hipStream_t st) {
    if (D == 128)
        return kv == kKvE4m3 ? launch_chunk_kv<kKvE4m3, 128>(p, grid, st) : kv == kKvI8 ? launch_chunk_kv<kKvI8, 128>(p, grid, st)
                                                                                        : launch_chunk_kv<kKvBf16, 128>(p, grid, st);
    return kv == kKvE4m3 ? launch_chunk_kv<kKvE4m3, 64>(p, grid, st) : kv == kKvI8 ? launch_chunk_kv<kKvI8, 64>(p, grid, st)
                                                                                   : launch_chunk_kv<kKvBf16, 64>(p, grid, st);
}

hipError_t launch_attn(AttnKind kind, int kv, int D, const AttnParams& p, hipStream_t st) {
    const int grid = p.tiles * p.splits * p.c.Hk;
    if (kind == kAttnF32) return launch_attn_f32(kv, D, p, grid, st);
    if (kind == kAttnChunk) return launch_attn_chunk(kv, D, p, grid, st);
    return launch_attn_step(kind, kv, D, p, grid, st);
}

}  // namespace kda
