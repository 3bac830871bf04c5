// Attention of few rows (one or a few new tokens a sequence) over a paged cache.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - max)
//
// Bound by reading the cache once.  A tile is 16 NB rows (tokens times the
// heads that share a cache head); a workgroup's four waves take blocks of 32
// positions in turn and keep maximum, sum and output of their own, joined at
// the end.  Nothing of the cache goes through LDS:
//   * S^T = K Q^T with 16x16x32 products: an operand lane holds eight (bf16) or
//     two times eight (8 bits) neighbouring channels of one position, which is
//     one 16-byte load.  The channels' order is free as long as Q has the same.
//   * O^T = V^T P^T: P^T comes out of S^T as it sits in the accumulator if lane
//     group g's eight positions are 4 g + i of either half of the block.  A lane
//     loads D / 16 neighbouring channels of those eight positions (a group of 16
//     lanes reads whole rows), and eight by eight values are transposed between
//     its own registers, one instruction for two values; product j then makes
//     channels (D / 16) rho + j, rho the accumulator's row.
// Up to 16 rows, P goes into its product as two bf16, itself and what its
// rounding left (2^-16 of it stay out): with the products far from being the
// bound, the second costs nothing (256 sequences 743 us, 64 x 4 tokens 228, with
// and without), and outputs are off by their own rounding alone.  The second part
// may be zero or negative, which an infinity in V must not meet: V is looked
// through in every block, by a running maximum of its exponents (the same times
// with and without; comparisons of each value spilled some 140 scalar registers).  With 32 rows the registers for a second part would have to be
// spilled: there P is rounded to bf16.  Everything else is fp32.
//
// Measured: 256 sequences of up to 8K, 32 heads of 128 over 8, one token each: bf16
// 743 us, 5.75 TB/s (a large copy moves 5.1); e4m3 5.4 TB/s, int8 5.0, heads of 64
// 4.9 to 5.6; one sequence of 1M in e4m3 376 us, 5.7 TB/s; 64 x 4 tokens 227 us.
// One sequence of 501 positions: 10.2 us in the kernel, a chain of loads that need
// one another (positions, table, rows, four blocks a wave) in eight workgroups, and
// as long on the host's way into the call.
#include "kda_paged_attn.h"

namespace kda {

namespace {

template <int KV> constexpr int kElem = KV == kKvF32 ? 4 : KV == kKvBf16 ? 2 : 1;

// N bytes at a wave's base and a lane's offset
template <int N> struct Raw {
    unsigned w[N / 4];
    __device__ __forceinline__ void load(const char* base, unsigned off) {
        if constexpr (N == 16) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(base + off);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = v[i];
        } else if constexpr (N == 8) {
            const u32x2 v = *reinterpret_cast<const u32x2*>(base + off);
            w[0] = v[0];
            w[1] = v[1];
        } else {
            w[0] = *reinterpret_cast<const unsigned*>(base + off);
        }
    }
};

// One block of 32 positions as it is loaded, in two halves of one page each.
// Places without a position (behind the last, or on no page) get what the page,
// or page 0, holds there: such scores are masked, and such values of V with them.
template <int KV, int D> struct Block {
    static constexpr int E = kElem<KV>, RB = D * E;
    static constexpr int KL = RB / 64;              // 16-byte loads of a K half (16 positions) a lane
    static constexpr int DV = D / 16;               // channels of V a lane
    static constexpr bool CODES = KV >= kKvE4m3;
    Raw<16> k[2][KL];
    Raw<DV * E> v[8];
    unsigned ks[2], vs[2];                          // scale bytes: K's row of the lane, V's four rows of either half
    int pg[2];
    unsigned koff, voff;

    __device__ __forceinline__ void init(int lane) {
        koff = (unsigned)((lane & 15) * RB + (lane >> 4) * 16);
        voff = (unsigned)((lane >> 4) * 4 * RB + (lane & 15) * DV * E);
    }
    __device__ __forceinline__ void find(const PagedCache& c, PageWalk<true>& w, int pos, int end) {
#pragma unroll
        for (int h = 0; h < 2; ++h) pg[h] = pos + 16 * h < end ? w.page((pos + 16 * h) >> c.lg_page) : -1;
    }
    __device__ __forceinline__ int valid() const { return (pg[0] >= 0) | (pg[1] >= 0) << 1; }
    __device__ __forceinline__ static size_t row(const PagedCache& c, int hk, int at) {
        return ((size_t)hk << c.lg_page) + (at & ((1 << c.lg_page) - 1));
    }
    __device__ __forceinline__ void load_k(const PagedCache& c, int hk, int pos, int lane) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const size_t page = (size_t)max(pg[h], 0), r = row(c, hk, pos + 16 * h);
            const char* at = c.k + page * c.k_page + r * RB;
#pragma unroll
            for (int i = 0; i < KL; ++i) k[h][i].load(at + 64 * i, koff);
            if constexpr (CODES) ks[h] = (c.ks + ((page * c.Hk) << c.lg_page) + r)[lane & 15];
        }
    }
    __device__ __forceinline__ void load_v(const PagedCache& c, int hk, int pos, int lane) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const size_t page = (size_t)max(pg[h], 0), r = row(c, hk, pos + 16 * h);
            const char* at = c.v + page * c.v_page + r * RB;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * h + i].load(at + i * RB, voff);
            if constexpr (CODES)
                vs[h] = *reinterpret_cast<const unsigned*>(c.vs + ((page * c.Hk) << c.lg_page) + r + 4 * (lane >> 4));
        }
    }
    // K operand of product s: channels of Q's operand s
    __device__ __forceinline__ bf16x8 kfrag(int h, int s) const {
        u32x4 u;
        if constexpr (!CODES) {
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = k[h][s].w[i];
        } else {
            const Codes<KV> d(ks[h]);
            unsigned o[4];
            d.bf(k[h][s >> 1].w[2 * (s & 1)], o);
            d.bf(k[h][s >> 1].w[2 * (s & 1) + 1], o + 2);
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = o[i];
        }
        return __builtin_bit_cast(bf16x8, u);
    }
    // Whether some scale of the lane's rows of V is from 2^113 on: no code under a
    // smaller one reaches 2^128, which is infinity in bf16.  (The byte's upper four bits.)
    __device__ __forceinline__ bool large_scales() const {
        const unsigned a = vs[0] & vs[0] << 1, b = vs[1] & vs[1] << 1;
        return ((a & a << 2) | (b & b << 2)) & 0x80808080u;
    }
    // V's eight positions as pairs of bf16: [position][DV / 2]
    __device__ __forceinline__ void vpairs(unsigned (&o)[8][DV / 2]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (!CODES) {
#pragma unroll
                for (int w = 0; w < DV / 2; ++w) o[i][w] = v[i].w[w];
            } else {
                const Codes<KV> d(vs[i >> 2] >> (8 * (i & 3)) & 255u);
#pragma unroll
                for (int w = 0; w < DV / 4; ++w) d.bf(v[i].w[w], &o[i][2 * w]);
            }
        }
    }
};

// first channel of a lane's operand s of Q, the order of Block::kfrag
template <int KV> __device__ __forceinline__ int q_channel(int s, int g) {
    return KV >= kKvE4m3 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
}

template <int KV, int D, int NB> __global__ __launch_bounds__(256, NB == 1 && !(KV == kKvBf16 && D == 128) ? 3 : 2) void kda_attn_step_kernel(AttnParams p) {
    constexpr int R = 16 * NB, DV = D / 16, KS = D / 32, LD = D + 4;
    constexpr bool TWO = NB == 1;       // two blocks of rows have no registers for it
    __shared__ __align__(16) float lds_o[2][R][LD];     // read and written as f32x4
    __shared__ float lds_ml[2][R][2];
    AttnTile t;
    if (!t.init(p, blockIdx.x)) return;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), g = lane >> 4, c16 = lane & 15;

    // Q as an operand, zeros behind the sequence's rows
    bf16x8 q[NB][KS];
    int lim[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int r = t.r0 + 16 * nb + c16;
        lim[nb] = t.limit(r, p);
        const int tok = p.by_g.div(r), head = t.hk * p.G + r - tok * p.G;
        const char* row = p.q + (size_t)(t.first + tok) * p.q_stride + (size_t)head * D * 2;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            u32x4 u = {0u, 0u, 0u, 0u};
            if (r < t.rows) u = *reinterpret_cast<const u32x4*>(row + q_channel<KV>(s, g) * 2);
            q[nb][s] = __builtin_bit_cast(bf16x8, u);
        }
    }
    const int lim_first = t.limit(t.r0, p);

    f32x4 acc[DV][NB];
    float m[NB], l[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        m[nb] = -INFINITY;
        l[nb] = 0.f;
#pragma unroll
        for (int j = 0; j < DV; ++j) acc[j][nb] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const float c = p.c_log2, lazy = kLazy / c;

    int bad_from = -1, bad_to = -1;     // the wave's first and last blocks of V with a value taken out
    int pos = t.lo + 32 * wave;
    if (pos < t.hi) {
        PageWalk<true> walk;
        walk.init(p.c, t.seq, t.L, t.lo >> p.c.lg_page);
        Block<KV, D> b;
        b.init(lane);
        b.find(p.c, walk, pos, t.hi);
        b.load_k(p.c, t.hk, pos, lane);
        b.load_v(p.c, t.hk, pos, lane);
        // (the next V's loads stand in every pass that comes back: a wait for K then leaves them open)
        for (;;) {
            f32x4 s[2][NB];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) s[h][nb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bf16x8 kf = b.kfrag(h, k);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) s[h][nb] = mma(s[h][nb], kf, q[nb][k]);
                }
            const int valid = b.valid();
            // rows of the tile that see less than the block, or pages that are not there
            const bool masked = pos + 31 > lim_first || valid != 3;
            const int next = pos + 128;
            if (next < t.hi) {
                b.find(p.c, walk, next, t.hi);
                b.load_k(p.c, t.hk, next, lane);
            }
            if (masked) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (pos + 16 * h + 4 * g + e > lim[nb] || !(valid >> h & 1)) s[h][nb][e] = -INFINITY;
            }
            // the running maximum moves for the whole wave, and only when a score passes it by enough
            bool up = false;
            float top[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                top[nb] = fmaxf(fmaxf(fmaxf(s[0][nb][0], s[0][nb][1]), fmaxf(s[0][nb][2], s[0][nb][3])),
                                fmaxf(fmaxf(s[1][nb][0], s[1][nb][1]), fmaxf(s[1][nb][2], s[1][nb][3])));
                up |= top[nb] > m[nb] + lazy;
            }
            if (__any(up)) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float x = fmaxf(top[nb], __shfl_xor(top[nb], 16));
                    x = fmaxf(x, __shfl_xor(x, 32));
                    const float mn = fmaxf(m[nb], x);
                    const float a = mn == -INFINITY ? 1.f : fast_exp2((m[nb] - mn) * c);
                    m[nb] = mn;
                    l[nb] *= a;
#pragma unroll
                    for (int j = 0; j < DV; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[j][nb][e] *= a;
                }
            }
            bf16x8 pf[NB], pl[TWO ? NB : 1];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const float mc = m[nb] == -INFINITY ? 0.f : m[nb] * c;
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] = fast_exp2(fmaf(s[i >> 2][nb][i & 3], c, -mc));
                    l[nb] += x[i];
                }
                pf[nb] = frag_from<bf16>(x);
                if constexpr (TWO) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] -= (float)pf[nb][i];
                    pl[nb] = frag_from<bf16>(x);
                }
            }
            unsigned vp[8][DV / 2];
            b.vpairs(vp);
            // A weight's second part may be zero or below zero, so that it must not meet an
            // infinity at all: with two parts these are looked for in every block.
            bool look = masked;
            if constexpr (TWO) look = masked || !Block<KV, D>::CODES || __any(b.large_scales());
            if (look) {
                // (what stands in for a place that is not there is no row's to have back)
                if (valid != 3)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int w = 0; w < DV / 2; ++w) vp[i][w] = valid >> (i >> 2) & 1 ? vp[i][w] : 0u;
                if (__any(not_finite(vp))) {
                    if (bad_from < 0) bad_from = pos;
                    bad_to = pos;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int w = 0; w < DV / 2; ++w) vp[i][w] = clean(vp[i][w]);
                }
            }
#pragma unroll
            for (int j = 0; j < DV; ++j) {
                u32x4 u;
                // halves j & 1 of two positions' dword j / 2
                const unsigned sel = j & 1 ? 0x07060302u : 0x05040100u;
#pragma unroll
                for (int i = 0; i < 4; ++i) u[i] = __builtin_amdgcn_perm(vp[2 * i + 1][j >> 1], vp[2 * i][j >> 1], sel);
                const bf16x8 vf = __builtin_bit_cast(bf16x8, u);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    if constexpr (TWO) acc[j][nb] = mma(acc[j][nb], vf, pl[nb]);
                    acc[j][nb] = mma(acc[j][nb], vf, pf[nb]);
                }
            }
            if (next >= t.hi) break;
            b.load_v(p.c, t.hk, next, lane);
            pos = next;
        }
    }
    if (bad_from >= 0) {
#pragma unroll 1
        for (int i = bad_from; i < min(t.hi, bad_to + 32); i += i % 32 == 31 ? 97 : 1)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < DV; j += 4) {
                    float f[4];
                    load_v4<KV, D>(p.c, t.seq, t.hk, i, DV * (4 * g + e) + j, f);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            if (i <= lim[nb] && !finite_f(f[k])) acc[j + k][nb][e] += f[k];
                }
    }
    // sums over the lane groups' positions
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        l[nb] += __shfl_xor(l[nb], 16);
        l[nb] += __shfl_xor(l[nb], 32);
    }
    // waves 2 and 3 join 0 and 1, then 1 joins 0
#pragma unroll
    for (int half = 2; half > 0; half >>= 1) {
        if (wave >= half && wave < 2 * half) {
            const int to = wave - half;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int r = 16 * nb + c16;
                if (g == 0) {
                    lds_ml[to][r][0] = m[nb];
                    lds_ml[to][r][1] = l[nb];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int j = 0; j < DV; j += 4)
                        *reinterpret_cast<f32x4*>(&lds_o[to][r][DV * (4 * g + e) + j]) =
                            f32x4{acc[j][nb][e], acc[j + 1][nb][e], acc[j + 2][nb][e], acc[j + 3][nb][e]};
            }
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int r = 16 * nb + c16;
                const float mo = lds_ml[wave][r][0], lo = lds_ml[wave][r][1], mn = fmaxf(m[nb], mo);
                const float a = m[nb] == mn ? 1.f : fast_exp2((m[nb] - mn) * c);
                const float b = mo == mn ? 1.f : fast_exp2((mo - mn) * c);
                m[nb] = mn;
                l[nb] = l[nb] * a + lo * b;
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int j = 0; j < DV; j += 4) {
                        const f32x4 o = *reinterpret_cast<const f32x4*>(&lds_o[wave][r][DV * (4 * g + e) + j]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[j + i][nb][e] = acc[j + i][nb][e] * a + o[i] * b;
                    }
            }
        }
        __syncthreads();
    }
    if (wave) return;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int r = t.r0 + 16 * nb + c16;
        if (r >= t.rows) continue;
        if (t.splits > 1) {
            float* po = p.part + (t.unit * R + 16 * nb + c16) * D;
            if (g == 0) {
                p.ml[(t.unit * R + 16 * nb + c16) * 2] = m[nb];
                p.ml[(t.unit * R + 16 * nb + c16) * 2 + 1] = l[nb];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < DV; j += 4)
                    *reinterpret_cast<f32x4*>(po + DV * (4 * g + e) + j) =
                        f32x4{acc[j][nb][e], acc[j + 1][nb][e], acc[j + 2][nb][e], acc[j + 3][nb][e]};
            continue;
        }
        const int tok = p.by_g.div(r), head = t.hk * p.G + r - tok * p.G;
        const float inv = 1.f / l[nb];
        const size_t at = (size_t)head * D;
        bf16* o = reinterpret_cast<bf16*>(p.o) + (size_t)(t.first + tok) * p.H * D + at;
        const bf16* z = reinterpret_cast<const bf16*>(p.z + (size_t)(t.first + tok) * p.z_stride) + at;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x[DV];
#pragma unroll
            for (int j = 0; j < DV; ++j) x[j] = l[nb] == 0.f ? 0.f : acc[j][nb][e] * inv;
            const int d = DV * (4 * g + e);
            if (p.z) {
#pragma unroll
                for (int j = 0; j < DV; ++j) x[j] = gate_of<bf16>(x[j], (float)z[d + j]);
            }
            st_run<DV>(o + d, x);
        }
    }
}

// Joins the ranges of tiles that were split.  D / 4 lanes take a range's row;
// a block of 256 threads takes TEAMS rows (token and head), the ranges of a row
// dealt to the lanes' slots of its team: one row where there are many ranges.
template <typename T, int D, int TEAMS> __global__ __launch_bounds__(256) void kda_attn_join_kernel(AttnParams p, int rows) {
    constexpr int LANES = D / 4, SLOTS = 256 / LANES / TEAMS;
    __shared__ f32x4 lds[SLOTS > 1 ? 256 : 1];
    __shared__ float lds_l[SLOTS > 1 ? SLOTS : 1];
    static_assert(TEAMS == 1 || SLOTS == 1, "a row a block, or a slot a row");
    const int lane = threadIdx.x % LANES, my = TEAMS == 1 ? threadIdx.x / LANES : 0;
    const int id = blockIdx.x * TEAMS + (TEAMS == 1 ? 0 : threadIdx.x / LANES);
    if (id >= rows) return;
    const int tok = p.by_h.div(id), head = id - tok * p.H, hk = p.by_g.div(head), gq = head - hk * p.G;
    int seq, first, n, slot0;
    if (p.sv.cu) {
        if (tok < p.sv.cu[0] || tok >= p.sv.cu[p.sv.N]) return;
        int a = 0, b = p.sv.N;
        while (b - a > 1) {
            const int mid = (a + b) >> 1;
            if (p.sv.cu[mid] <= tok)
                a = mid;
            else
                b = mid;
        }
        seq = a;
        seq_span(p.sv, seq, &first, &n);
        slot0 = ((first * p.G) >> p.lg_m) + seq;
    } else {
        seq = p.by_t.div(tok);
        seq_span(p.sv, seq, &first, &n);
        slot0 = seq * p.tiles_per_seq;
    }
    if ((unsigned)(tok - first) >= (unsigned)n) return;
    const int r = (tok - first) * p.G + gq, at = r >> p.lg_m;
    if (slot0 + at >= p.tiles) return;
    const int L = seq_positions(p.c, seq);
    const int end = max(L - n + p.by_g.div(min((at + 1) << p.lg_m, n * p.G) - 1) + 1, 0);
    const int splits = end > 0 ? p.by_len.div(end - 1) + 1 : 1;
    if (splits <= 1) return;
    const size_t unit = ((size_t)(slot0 + at) * p.c.Hk + hk) * p.splits;
    const size_t row = (unit << p.lg_m) + (r - (at << p.lg_m));     // of range 0; ranges are M rows apart
    const float2* ml = reinterpret_cast<const float2*>(p.ml) + row;
    float top = -INFINITY;
    for (int s = lane; s < splits; s += LANES) top = fmaxf(top, ml[(size_t)s << p.lg_m].x);
#pragma unroll
    for (int m = LANES / 2; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor(top, m));
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
    const float* part = p.part + row * D + 4 * lane;
#pragma unroll 4
    for (int s = my; s < splits; s += SLOTS) {
        const float2 x = ml[(size_t)s << p.lg_m];
        const f32x4 v = *reinterpret_cast<const f32x4*>(part + ((size_t)s << p.lg_m) * D);
        const float w = x.x == top ? 1.f : fast_exp2((x.x - top) * p.c_log2);
        l += w * x.y;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += w * v[i];
    }
    if constexpr (SLOTS > 1) {
        lds[threadIdx.x] = o;
        if (lane == 0) lds_l[my] = l;
        __syncthreads();
        if (my) return;
        for (int s = 1; s < SLOTS; ++s) {
            l += lds_l[s];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] += lds[s * LANES + lane][i];
        }
    }
    const size_t col = (size_t)head * D + 4 * lane;
    const T* z = p.z ? reinterpret_cast<const T*>(p.z + (size_t)tok * p.z_stride) + col : nullptr;
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[i] = l == 0.f ? 0.f : o[i] / l;
        if (z) y[i] = gate_of<T>(y[i], to_f32(z[i]));
    }
    st_run<4>(reinterpret_cast<T*>(p.o) + (size_t)tok * p.H * D + col, y);
}

template <typename T, int D> hipError_t launch_join(const AttnParams& p, int rows, hipStream_t st) {
    constexpr int TEAMS = 1024 / D;
    if (p.splits > 8)
        kda_attn_join_kernel<T, D, 1><<<rows, 256, 0, st>>>(p, rows);
    else
        kda_attn_join_kernel<T, D, TEAMS><<<(rows + TEAMS - 1) / TEAMS, 256, 0, st>>>(p, rows);
    return hipGetLastError();
}

template <int KV, int D> hipError_t launch_step(AttnKind kind, const AttnParams& p, int grid, hipStream_t st) {
    if (kind == kAttnStep16)
        kda_attn_step_kernel<KV, D, 1><<<grid, 256, 0, st>>>(p);
    else
        kda_attn_step_kernel<KV, D, 2><<<grid, 256, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_step(AttnKind kind, int kv, int D, const AttnParams& p, int grid, hipStream_t st) {
    if (D == 128)
        return kv == kKvE4m3 ? launch_step<kKvE4m3, 128>(kind, p, grid, st) : kv == kKvI8 ? launch_step<kKvI8, 128>(kind, p, grid, st)
                                                                                          : launch_step<kKvBf16, 128>(kind, p, grid, st);
    return kv == kKvE4m3 ? launch_step<kKvE4m3, 64>(kind, p, grid, st) : kv == kKvI8 ? launch_step<kKvI8, 64>(kind, p, grid, st)
                                                                                     : launch_step<kKvBf16, 64>(kind, p, grid, st);
}

hipError_t launch_attn_join(int dtype, int D, const AttnParams& p, int M_tokens, hipStream_t st) {
    const int rows = M_tokens * p.H;
    if (dtype) return D == 128 ? launch_join<bf16, 128>(p, rows, st) : launch_join<bf16, 64>(p, rows, st);
    return D == 128 ? launch_join<float, 128>(p, rows, st) : launch_join<float, 64>(p, rows, st);
}

}  // namespace kda
