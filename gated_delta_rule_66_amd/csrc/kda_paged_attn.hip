// Attention of chunks of new tokens over a paged cache, bf16.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i.k_j - max_i),  j <= position of i
//
// Bound by its products (4 D flops a pair of row and position).  A workgroup of
// W waves takes 128 or 256 rows (tokens times the heads that share a cache
// head), 32 NR a wave, and walks tiles of 64 positions that all waves share in LDS.
// Products are 32x32x16 with the row in the lane:
//   * S^T = K Q^T: a lane has 32 of a tile's 64 scores of its row, so maximum
//     and sum need no exchange but between two lanes, and that only when the
//     maximum moves;
//   * O^T = V^T P^T: S^T as it sits in the accumulator is the operand P^T if a
//     product's 16 positions are 8 (i / 4) + 4 h + i % 4 (lane half h), which
//     the transposing reads of V deliver as well.
// P is rounded to bf16 for its product (relative 2^-8, as V's own rounding; the
// sum is taken before it), everything else is fp32.
//
// Measured: 8K prompt, 32 heads of 128 over 8, bf16, gate: 522 us (1053 TFLOP/s,
// 74 % of a large library product); 4 x 2K tokens over 32K 3.61 ms in bf16 (1181
// TFLOP/s), 3.95 in e4m3, 4.07 in int8; 48 packed sequences over int8, 12 heads of
// 64 over 3: 166 us.  Heads of 128: matrix units are busy half of the time, and the
// card's clock falls as they get busier (2.03 GHz in the prompt, 53 % busy, 1.93 in
// 4 x 2K over 32K in bf16, 59 %, 2.40 where they rest; a tenth fewer cycles a call
// left its time as it was); 8-bit codes add their conversion on the way to LDS.  Heads of 64: the
// exponentials and conversions of the vector units.
// Tried and left out: a higher wave priority during products (bf16 1.5 % faster,
// e4m3 2.5 % slower); heads of 64 with sums from a product with ones (2 % slower)
// or with scores a tile ahead beside them (spills at three waves a SIMD).
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

// 64 lanes' 16 bytes at base + off straight into 1024 bytes of LDS at `to`.
// Written out because the compiler would wait for a builtin's loads before any
// read of LDS, those of the tile before included: the wait is Stage::store's.
// (m0, the LDS address, has to stand one instruction before its use; the
// compiler has no use of its own for it in this kernel.)
__device__ __forceinline__ void load_lds16(const char* base, unsigned off, unsigned to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(to), "v"(off), "s"(base)
                 : "memory");
}
__device__ __forceinline__ unsigned lds_address(const char* p) {
    typedef __attribute__((address_space(3))) const char lds_c;
    return (unsigned)(uintptr_t)(lds_c*)p;
}

// Pages of a tile: of its groups of 16 positions where pages are smaller than
// tiles, else one page.  -1: not there.
struct TilePages {
    int pg[kTile / 16];
    int pos, valid;         // valid: bit i where group i has a page
    __device__ __forceinline__ void find(PageWalk<false>& w, int lg_page, int at, int end) {
        pos = at;
        if (lg_page >= 6) {
            pg[0] = w.page(at >> lg_page);
            valid = pg[0] >= 0 ? 15 : 0;
            return;
        }
        valid = 0;
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i) {
            pg[i] = at + 16 * i < end ? w.page((at + 16 * i) >> lg_page) : -1;
            valid |= (pg[i] >= 0) << i;
        }
    }
};

// A tile of K or V on its way to LDS: four waves' loads of 1024 bytes, each of
// one page.  bf16 rows go straight to their places, the pieces permuted by what
// a lane loads; codes go through registers.  Places without a position (behind
// the last, or on no page) get what the page, or page 0, holds there: such
// scores are masked, and such values of V with them.
template <int KV, int D, bool V, int W> struct Stage {
    static constexpr int E = KV == kKvBf16 ? 2 : 1;
    static constexpr int RB = D * E;                // bytes of a row
    static constexpr int PER = 1024 / RB;           // rows of a wave's load
    static constexpr int N = kTile / (W * PER);     // loads of a wave
    u32x4 w[N];
    unsigned s[N];
    unsigned voff[N];       // a lane's bytes in a load, from the tile's first row (small pages: from the load's)
    __device__ __forceinline__ void init(int wave, int lane, bool small) {
        const int r = wave * PER + lane / (64 / PER), piece = lane % (64 / PER);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            unsigned at = (unsigned)lane * 16;
            if constexpr (KV == kKvBf16)
                at = (unsigned)((lane / (64 / PER)) * RB + 16 * (V ? v_piece<D>(r, piece) : k_piece<D>(r, piece)));
            voff[i] = at + (small ? 0u : (unsigned)((i * W + wave) * PER * RB));
        }
    }
    __device__ __forceinline__ void one(const char* at, int i, char* tile, int wave) {
        if constexpr (KV == kKvBf16)
            load_lds16(uniform(at), voff[i], lds_address(tile) + (unsigned)((i * W + wave) * PER * D * 2));
        else
            w[i] = *reinterpret_cast<const u32x4*>(at + voff[i]);
    }
    __device__ __forceinline__ void load(const PagedCache& c, const TilePages& t, int hk, char* tile, int wave, int lane) {
        const char* base = V ? c.v : c.k;
        const unsigned char* scale = V ? c.vs : c.ks;
        const size_t page_bytes = V ? c.v_page : c.k_page;
        const int mask = (1 << c.lg_page) - 1;
        if (c.lg_page >= 6) {
            const size_t pg = (size_t)max(t.pg[0], 0), r = ((size_t)hk << c.lg_page) + (t.pos & mask);
            const char* at = base + pg * page_bytes + r * RB;
            const unsigned char* sc = scale + ((pg * c.Hk) << c.lg_page) + r;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                one(at, i, tile, wave);
                if constexpr (KV != kKvBf16) s[i] = sc[(i * W + wave) * PER + lane / (64 / PER)];
            }
            return;
        }
        // copies: a choice among the members themselves would put them into memory
        const int p0 = t.pg[0], p1 = t.pg[1], p2 = t.pg[2], p3 = t.pg[3];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r0 = (i * W + wave) * PER;    // of the tile
            const int pg = max(r0 >= 32 ? (r0 >= 48 ? p3 : p2) : (r0 >= 16 ? p1 : p0), 0);
            const size_t r = ((size_t)hk << c.lg_page) + ((t.pos + r0) & mask);
            one(base + (size_t)pg * page_bytes + r * RB, i, tile, wave);
            if constexpr (KV != kKvBf16) s[i] = scale[(((size_t)pg * c.Hk) << c.lg_page) + r + lane / (64 / PER)];
        }
    }
    // what was loaded is in LDS once the workgroup has passed a barrier
    __device__ __forceinline__ void store(char* tile, int wave, int lane) const {
        if constexpr (KV == kKvBf16) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int r = (i * W + wave) * PER + lane / (64 / PER), p = lane % (64 / PER);
                u32x4* to = reinterpret_cast<u32x4*>(tile + r * D * 2);
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

// A lane's byte offsets in the tiles; what changes between the products of a
// tile is added as the reads' own constants.
template <int D> struct Offsets {
    static constexpr int KS = D / 16, RB = 2 * D;
    int k[KS], v[D / 32];
    __device__ __forceinline__ void init(int lane) {
#pragma unroll
        for (int s = 0; s < KS; ++s) k[s] = opaque((lane & 31) * RB + 16 * k_piece<D>(lane & 31, 2 * s + (lane >> 5)));
        const int r = 4 * (lane >> 5) + (lane >> 2 & 3);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const int col = 32 * i + 16 * (lane >> 4 & 1) + 4 * (lane & 3);
            v[i] = opaque(r * RB + 16 * v_piece<D>(r, col >> 3) + 2 * (col & 7));
        }
    }
    // K operand: position 32 b + l % 32, channels 16 s + 8 (l / 32) ..
    __device__ __forceinline__ bf16x8 k_frag(const char* tile, int b, int s) const {
        return *reinterpret_cast<const bf16x8*>(tile + k[s] + 32 * b * RB);
    }
    // V operand: channel 32 db + l % 32, positions 16 s + 4 h + i and 16 s + 8 + 4 h + i
    __device__ __forceinline__ bf16x8 v_frag(const char* tile, int db, int s) const {
        typedef __attribute__((address_space(3))) bf16x4 lds_x4;
        const char* p = tile + v[db] + 16 * s * RB;
        const bf16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_x4*)p);
        const bf16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_x4*)(p + 8 * RB));
        bf16x8 f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = a[i];
            f[4 + i] = b[i];
        }
        return f;
    }
};

// What a wave keeps of its NR times 32 rows.  Scores are a tile ahead: while a
// tile's weights are made and multiplied with V, the matrix units have the next
// tile's scores to go on with.
template <int D, int NR> struct Rows {
    static constexpr int KS = D / 16, DB = D / 32;
    typedef f32x16 Scores[NR][2];
    bf16x8 q[NR][KS];
    f32x16 acc[NR][DB];
    float m[NR], l[NR], mc[NR];
    int lim[NR];            // the last positions that the lane's rows see
    Offsets<D> at;

    __device__ __forceinline__ void scores(Scores& s, const char* tk) {
        bf16x8 kf[2][KS];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e) s[n][b][e] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) kf[b][k] = at.k_frag(tk, b, k);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int n = 0; n < NR; ++n) s[n][b] = mma32(s[n][b], kf[b][k], q[n][k]);
    }
    struct Top {
        float v[NR];
    };
    static __device__ __forceinline__ Top largest(const Scores& s) {
        Top t;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            t.v[n] = s[n][0][0];
#pragma unroll
            for (int e = 1; e < 16; ++e) t.v[n] = fmaxf(t.v[n], s[n][0][e]);
#pragma unroll
            for (int e = 0; e < 16; ++e) t.v[n] = fmaxf(t.v[n], s[n][1][e]);
        }
        return t;
    }
    // Scores of the tile at pos become weights' logarithms: masked where some
    // row of the wave sees only a part of it, and the maximum moved.
    __device__ __forceinline__ void settle(Scores& s, Top top, float c, bool masked, int pos, int valid, int lane) {
        if (masked) {
            const int h = lane >> 5;
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int j = 32 * b + 8 * (e >> 2) + 4 * h + (e & 3);
                        if (pos + j > lim[n] || !(valid >> (2 * b + (e >> 3)) & 1)) s[n][b][e] = -INFINITY;
                    }
            top = largest(s);
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            if (!__any(top.v[n] > m[n] + kLazy / c)) continue;
            const float mn = fmaxf(m[n], fmaxf(top.v[n], __shfl_xor(top.v[n], 32)));
            const float a = mn == -INFINITY ? 1.f : fast_exp2((m[n] - mn) * c);
            m[n] = mn;
            mc[n] = mn == -INFINITY ? 0.f : mn * c;
            l[n] *= a;
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[n][db][e] *= a;
        }
    }
    __device__ __forceinline__ bf16x8 weights(const Scores& s, int n, int k, float c) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = fast_exp2(fmaf(s[n][k >> 1][8 * (k & 1) + i], c, -mc[n]));
            l[n] += x[i];
        }
        return frag_from<bf16>(x);
    }
    // One tile's weights and product with V, 16 positions at a time: the weights
    // of the next beside the products of the present ones.  `made` of the four
    // are made already; `last` is the vector work beside the third's products.
    template <class F>
    __device__ __forceinline__ void product(const Scores& s, bf16x8 (&pf)[NR][4], int made, bf16x8 (&vf)[2][DB],
                                            const char* tv, float c, F&& last) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k < 3) {
#pragma unroll
                for (int db = 0; db < DB; ++db) vf[(k + 1) & 1][db] = at.v_frag(tv, db, k + 1);
            }
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int db = 0; db < DB; ++db) acc[n][db] = mma32(acc[n][db], vf[k & 1][db], pf[n][k]);
            if (k + made < 4) {
#pragma unroll
                for (int n = 0; n < NR; ++n) pf[n][k + made] = weights(s, n, k + made, c);
            }
            if (k == 2) last();
#pragma unroll
            for (int i = 0; i < DB * NR; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                if (k < 3) {
                    __builtin_amdgcn_sched_group_barrier(0x100, NR == 1 ? 2 : 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x402, 28 / DB, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // One tile, and the next one's scores; returns their largest.  The groups
    // order what the compiler otherwise puts apart: LDS reads go out some
    // products ahead, vector work stands between the products.
    // D = 128: products take longer than the vector work (32 cycles each, 4096 a
    // pair of tiles and SIMD), and the next scores' products stand beside the first weights.
    // D = 64: the vector work is longer; the scores come last, in the registers
    // of those before.
    __device__ __forceinline__ Top tile(const Scores& s, Scores& next, const char* tk, const char* tv, float c) {
        bf16x8 vf[2][DB], pf[NR][4];
        Top top;
        if constexpr (D == 128) {
            scores(next, tk);
#pragma unroll
            for (int db = 0; db < DB; ++db) vf[0][db] = at.v_frag(tv, db, 0);
            pf[0][0] = weights(s, 0, 0, c);
            pf[0][1] = weights(s, 0, 1, c);
            __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
            for (int i = 0; i < 2 * KS - 4; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x402, 4, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, DB / 2, 0);
                __builtin_amdgcn_sched_group_barrier(0x402, 4, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            product(s, pf, 2, vf, tv, c, [&]() { top = largest(next); });
        } else {
#pragma unroll
            for (int db = 0; db < DB; ++db) vf[0][db] = at.v_frag(tv, db, 0);
#pragma unroll
            for (int n = 0; n < NR; ++n) pf[n][0] = weights(s, n, 0, c);
            __builtin_amdgcn_sched_barrier(0);
            product(s, pf, 1, vf, tv, c, []() {});
            scores(next, tk);
            top = largest(next);
            __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
            for (int i = 0; i < 2 * KS - 4; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, NR, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
        }
        return top;
    }
};

// W waves of 32 NR rows.
template <int KV, int D, int W, int NR>
__global__ __launch_bounds__(64 * W, D == 128 || NR == 2 ? 2 : 3) void kda_attn_chunk_kernel(AttnParams p) {
    constexpr int KS = D / 16, DB = D / 32, RW = 32 * NR, M = RW * W;
    constexpr int TB = kTile * D * 2;
    __shared__ __align__(16) char lds[4 * TB];      // two tiles of K, two of V
    __shared__ int lds_bad;                         // the first tile of V with a value taken out, or -1
    AttnTile t;
    if (!t.init(p, blockIdx.x)) return;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), h = lane >> 5;

    // The wave's first and last limits.  The last is cut off at the range's end: the
    // scores behind its last tile are those of K that an earlier tile left.
    const int w0 = t.r0 + RW * wave, lim_first = t.limit(w0, p), t_first = t.limit(t.r0, p);
    const int lim_last = w0 < t.rows ? min(t.limit(min(w0 + RW - 1, t.rows - 1), p), t.hi - 1) : -1;
    Rows<D, NR> x;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int r = w0 + 32 * n + (lane & 31), tok = p.by_g.div(r), head = t.hk * p.G + r - tok * p.G;
        x.lim[n] = t.limit(r, p);
        const char* row = p.q + (size_t)(t.first + tok) * p.q_stride + (size_t)head * D * 2;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            u32x4 u = {0u, 0u, 0u, 0u};
            if (r < t.rows) u = *reinterpret_cast<const u32x4*>(row + (16 * s + 8 * h) * 2);
            x.q[n][s] = __builtin_bit_cast(bf16x8, u);
        }
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int e = 0; e < 16; ++e) x.acc[n][db][e] = 0.f;
        x.m[n] = -INFINITY;
        x.l[n] = x.mc[n] = 0.f;
    }
    const float c = p.c_log2;

    PageWalk<false> walk;
    walk.init(p.c, t.seq, t.L, t.lo >> p.c.lg_page);       // waits for its load, and Q's with it
    Stage<KV, D, false, W> sk;
    Stage<KV, D, true, W> sv;
    sk.init(wave, lane, p.c.lg_page < 6);
    sv.init(wave, lane, p.c.lg_page < 6);
    x.at.init(lane);
    if (threadIdx.x == 0) lds_bad = -1;
    typename Rows<D, NR>::Scores sa, sb;
    TilePages next;         // of the tile behind the present one
    int valid = 15;         // of the present one
    if (t.lo < t.hi) {
        next.find(walk, p.c.lg_page, t.lo, t.hi);
        valid = next.valid;
        sk.load(p.c, next, t.hk, lds, wave, lane);
        sv.load(p.c, next, t.hk, lds + 2 * TB, wave, lane);
        sk.store(lds, wave, lane);
        __syncthreads();
        if (t.lo + kTile < t.hi) {
            next.find(walk, p.c.lg_page, t.lo + kTile, t.hi);
            sk.load(p.c, next, t.hk, lds + TB, wave, lane);
        }
        if (t.lo <= lim_last) {
            x.scores(sa, lds);
            x.settle(sa, x.largest(sa), c, t.lo + kTile - 1 > lim_first || valid != 15, t.lo, valid, lane);
        }
    }
    // The tile at pos, whose scores are in s: its V lies at v, the next tile's K
    // at k; the K behind that and the next V go to k_to and v_to.
    auto step = [&](int pos, typename Rows<D, NR>::Scores& s, typename Rows<D, NR>::Scores& n, char* k, char* v, char* k_to, char* v_to) {
        sk.store(k, wave, lane);
        sv.store(v, wave, lane);
        __syncthreads();
        if (pos + kTile - 1 > t_first || valid != 15) {     // some row of the tile's sees only a part
            int bad = 0;            // bits of groups of 16 rows, from the thread's first on
            u32x4* w = reinterpret_cast<u32x4*>(v) + threadIdx.x;
#pragma unroll
            for (int i = 0; i < TB / (1024 * W); ++i) {
                u32x4 y = w[64 * W * i];
                if (not_finite(y[0]) || not_finite(y[1]) || not_finite(y[2]) || not_finite(y[3])) {
                    w[64 * W * i] = u32x4{clean(y[0]), clean(y[1]), clean(y[2]), clean(y[3])};
                    bad |= 1 << (64 * W / (2 * D)) * i;
                }
            }
            // (what stands in for a place that is not there is no row's to have back)
            if (bad && (bad << threadIdx.x / (2 * D) & valid) && lds_bad < 0) lds_bad = pos;
            __syncthreads();
        }
        valid = next.valid;
        if (pos + kTile < t.hi) sv.load(p.c, next, t.hk, v_to, wave, lane);
        if (pos + 2 * kTile < t.hi) {
            next.find(walk, p.c.lg_page, pos + 2 * kTile, t.hi);
            sk.load(p.c, next, t.hk, k_to, wave, lane);
        }
        if (pos > lim_last) return;         // the wave's rows see nothing of it
        const auto top = x.tile(s, n, k, v, c);
        pos += kTile;
        if (pos <= lim_last) x.settle(n, top, c, pos + kTile - 1 > lim_first || valid != 15, pos, valid, lane);
    };
    for (int pos = t.lo; pos < t.hi; pos += 2 * kTile) {
        step(pos, sa, D == 128 ? sb : sa, lds + TB, lds + 2 * TB, lds, lds + 3 * TB);
        if (pos + kTile < t.hi) step(pos + kTile, D == 128 ? sb : sa, sa, lds, lds + 3 * TB, lds + TB, lds + 2 * TB);
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        if (lds_bad >= 0) mend_rows<KV, D>(x.acc[n], p, t, lds_bad, x.lim[n], h);
        const int r = w0 + 32 * n + (lane & 31), tok = p.by_g.div(r), head = t.hk * p.G + r - tok * p.G;
        const float l = x.l[n] + __shfl_xor(x.l[n], 32);
        if (r >= t.rows) continue;
        auto& acc = x.acc[n];
        if (t.splits > 1) {
            const size_t at = t.unit * M + (r - t.r0);
            float* po = p.part + at * D;
            if (h == 0) {
                p.ml[at * 2] = x.m[n];
                p.ml[at * 2 + 1] = l;
            }
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<f32x4*>(po + 32 * db + 8 * j + 4 * h) =
                        f32x4{acc[db][4 * j], acc[db][4 * j + 1], acc[db][4 * j + 2], acc[db][4 * j + 3]};
            continue;
        }
        const float inv = 1.f / l;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[db][e] = l == 0.f ? 0.f : acc[db][e] * inv;
        const size_t out = ((size_t)head * D + 4 * h) * 2;
        if (p.z) {
            const char* z = p.z + (size_t)(t.first + tok) * p.z_stride + out;
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bf16x4 zz = *reinterpret_cast<const bf16x4*>(z + 64 * db + 16 * j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[db][4 * j + i] = gate_of<bf16>(acc[db][4 * j + i], (float)zz[i]);
                }
        }
        char* o = p.o + (size_t)(t.first + tok) * p.H * D * 2 + out;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float y[4] = {acc[db][4 * j], acc[db][4 * j + 1], acc[db][4 * j + 2], acc[db][4 * j + 3]};
                st_run<4>(reinterpret_cast<bf16*>(o + 64 * db + 16 * j), y);
            }
    }
}

template <int KV, int D> hipError_t launch_chunk_kv(AttnKind kind, const AttnParams& p, int grid, hipStream_t st) {
    if (kind != kAttnChunk256)
        kda_attn_chunk_kernel<KV, D, 4, 1><<<grid, 256, 0, st>>>(p);
    else if constexpr (D == 128)
        kda_attn_chunk_kernel<KV, D, 8, 1><<<grid, 512, 0, st>>>(p);
    else
        kda_attn_chunk_kernel<KV, D, 4, 2><<<grid, 256, 0, st>>>(p);
    return hipGetLastError();
}
template <int D> hipError_t launch_chunk_d(AttnKind kind, int kv, const AttnParams& p, int grid, hipStream_t st) {
    if (kv == kKvE4m3) return launch_chunk_kv<kKvE4m3, D>(kind, p, grid, st);
    if (kv == kKvI8) return launch_chunk_kv<kKvI8, D>(kind, p, grid, st);
    return launch_chunk_kv<kKvBf16, D>(kind, p, grid, st);
}

}  // namespace

hipError_t launch_attn_chunk(AttnKind kind, int kv, int D, const AttnParams& p, int grid, hipStream_t st) {
    return D == 128 ? launch_chunk_d<128>(kind, kv, p, grid, st) : launch_chunk_d<64>(kind, kv, p, grid, st);
}

hipError_t launch_attn(AttnKind kind, int kv, int D, const AttnParams& p, hipStream_t st) {
    const int grid = p.tiles * p.splits * p.c.Hk;
    if (kind == kAttnF32) return launch_attn_f32(kv, D, p, grid, st);
    if (kind == kAttnChunk || kind == kAttnChunk256) return launch_attn_chunk(kind, kv, D, p, grid, st);
    return launch_attn_step(kind, kv, D, p, grid, st);
}

}  // namespace kda
