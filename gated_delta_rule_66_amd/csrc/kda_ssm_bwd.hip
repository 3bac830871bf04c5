// Backward of the selective scan, chunk by chunk, from the state before each
// chunk (S) and the adjoint behind it (E).  With c the chunk's inclusive sums
// of log a, L_ij = e^{c_i - c_j} (i >= j), G = C B^T, w_j = e^{c_63 - c_j} delta_j:
//
//   Q_ij  = (dy_i . x_j) L_ij
//   dx_j  = sum_i G_ij L_ij delta_j dy_i + w_j E^T B_j + D dy_j
//   dC_i  = sum_h [ sum_j Q_ij delta_j B_j + e^{c_i} S dy_i ]
//   dB_j  = sum_h [ sum_i Q_ij delta_j C_i + w_j E x_j ]
//   z_j   = x_j . E^T B_j,   r_i = e^{c_i} dy_i . S^T C_i
//   d log a_t = sum_{i >= t > j} Q_ij G_ij delta_j          (pairs across t)
//             + sum_{i >= t} r_i + sum_{j < t} w_j z_j + e^{c_63} <S, E>
//   d delta_j = sum_i Q_ij G_ij + e^{c_63 - c_j} z_j + A d log a_j
//
// The sum over the heads of a group is taken on Q delta (64 x 64) before the
// products with B and C.  d log a and d delta come from fp32 values of the
// score tiles and from products whose state operand is split exactly, because
// their sums over all tokens are fp32 gradients.  bf16 tokens: dx, dB and dC,
// which leave as bf16, take their fp32 operands (a head's scaled scores, the
// heads' summed score gradients, and the states and adjoints of dB's and dC's
// products) as two bf16 each, exact to 2^-16; one bf16 each would put them at
// 0.0023 of their root mean square instead of the 0.0017 of their own rounding,
// with the gradient kernel at 146 us instead of 157 on 8K x 32 heads.  fp32
// tokens: fp32 products throughout.
#include "kda_ssm_device.h"

namespace kda {

namespace {

constexpr int C = kSsmChunk;

__device__ __forceinline__ f32x4 mma_exact_a(f32x4 acc, const Split3& v, bf16x8 b) {
    acc = mma(acc, v.lo, b);
    acc = mma(acc, v.mid, b);
    return mma(acc, v.hi, b);
}
__device__ __forceinline__ f32x4 mma_exact_a(f32x4 acc, const f32x8& v, f32x8 b) { return mma(acc, v, b); }

// Sums across lanes without LDS: rotations within rows of 16 lanes, and the
// exchange of rows and halves between two registers (v' = a's rows 0, 2 next to
// b's, v'' = rows 1, 3; with a = b = v, v' + v'' adds neighbouring rows).
template <int ROT> __device__ __forceinline__ float row_rotate(float v) {
    return __uint_as_float((unsigned)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x120 + ROT, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum16(float v) {
    v += row_rotate<8>(v);
    v += row_rotate<4>(v);
    v += row_rotate<2>(v);
    return v + row_rotate<1>(v);
}
__device__ __forceinline__ float sum_groups(float v) {
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// the sum over the rows of 16 lanes behind the lane's own (g)
__device__ __forceinline__ float sum_groups_behind(float v, int g) {
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    const float next = (g & 1) ? 0.f : __uint_as_float(r[1]);
    const float pair = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(pair), __float_as_uint(pair), false, false);
    return g < 2 ? next + __uint_as_float(r[1]) : next;
}
__device__ __forceinline__ float sum64(float v) { return sum_groups(sum16(v)); }

// One workgroup (8 waves) per (chunk, group, part of the group's heads), head by
// head.  The group's B, C and scores stay; a head's x, dy and states are loaded
// into registers behind the head before and staged in LDS (states in fp32,
// where they fit; else their fragments come from memory).  Work of the waves:
//   pairs:   the ten lower 16 x 16 tiles, one or two a wave
//   states:  E^T B and S^T C, a 16-column tile of one of them a wave (P = 64)
//            or a tile of each (P = 128); products with exact state operands
//   dB, dC:  16 state rows of both (K = 128) or of one of them (K = 64) a wave,
//            summed over the heads in registers
// A head's rows and states are 80 KB (K = 128, P = 64), which alone take 4 of
// the 10 us a head, and the LDS holds one workgroup a CU; the rest is the three
// phases' LDS reads (0.6 MB a head) between barriers.  8K x 32 heads: 157 us
// (347 MB read, 56 MB written).  With one bf16 an operand 146 us; that with all
// waves loading the next head at once 166 us, and with four waves and states
// from memory 314.  K = 64, P = 128, 6 heads packed: 68 us.
template <typename T, int K, int P>
__global__ __launch_bounds__(512) void kda_ssm_bwd_kernel(SsmBwdParams p) {
    constexpr int TH = 512;
    constexpr int EPP = 16 / sizeof(T);
    constexpr int LDK = K + tr_pad<T>(K), LDP = P + tr_pad<T>(P), LDM = C + 16 / sizeof(T);
    constexpr bool STAGED = sizeof(T) == 2 && K * P <= 8192;
    constexpr int LDS_ = P + 4;             // fp32 state rows
    constexpr int TU = P / 64, TK = K / 64; // state and dB/dC tasks a wave
    constexpr int PX = C * P / EPP / TH, PS = STAGED ? K * P / 4 / TH : 1;
    static_assert(C * P / EPP % TH == 0 && (K * P / 4) % TH == 0, "whole pieces");
    typedef typename FragOf<T>::type Frag;
    __shared__ T sB[C * LDK], sC[C * LDK], sX[C * LDP], sDY[C * LDP], sM[C * LDM];
    __shared__ T sML[sizeof(T) == 2 ? C * LDM : 1];     // sM's lower halves
    __shared__ __align__(16) float sS[STAGED ? K * LDS_ : 1], sE[STAGED ? K * LDS_ : 1];
    // what the step sizes' gradients need of a head, for two heads in turn: the
    // last wave works on it beside the next head's pairs (fp32 at K = P = 128
    // has no LDS for two, and does it at the head's end)
    constexpr int NB = sizeof(T) == 4 && K * P > 8192 ? 1 : 2;
    __shared__ __align__(16) float s_gate_[NB][kGates][C];
    __shared__ float s_row_[NB][10][16], s_colf_[NB][10][16], s_cols_[NB][10][16], s_z_[NB][P / 16][C],
        s_r_[NB][P / 16][C], s_se_[NB][8], s_dd_[NB][8];

    const SsmParams& f = p.f;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, r16 = lane & 15;
    const int flat = xcd_swizzle(blockIdx.x, gridDim.x);
    const int part = flat % p.parts, grp = (flat / p.parts) % f.G, ci = flat / (p.parts * f.G);
    const int hpg = f.H / f.G;
    const int ha = grp * hpg + min(part * p.heads_per, hpg), hb = grp * hpg + min((part + 1) * p.heads_per, hpg);
    constexpr int KP = K * P;
    if (ci >= total_chunks(f)) {
        // chunks that a packed call's bound counts and its lengths do not have
        for (int h = ha + tid; h < hb; h += TH)
            for (int m = 0; m < 3; ++m) p.sums[((size_t)ci * 3 + m) * f.H + h] = 0.f;
        return;
    }
    ChunkWalk at;
    at.init(f, ci);
    const int t0 = at.t0(), len = at.len();
    auto start_of = [&](int h) { return p.start + ((size_t)ci * f.H + h) * KP; };
    auto dend_of = [&](int h) { return p.dend + ((size_t)ci * f.H + h) * KP; };

    // ---- a head's rows, states and gates: loads, then LDS
    uint4 rx[PX], rg[PX], rs[PS], re[PS], rgate;
    T rdt = (T)0.f;
    auto fetch = [&](int h) {
        const int td = opaque(tid);
        const auto xr = row_rsrc<T>(reinterpret_cast<const T*>(f.x) + h * P, f.x_stride, t0, len, P);
        const auto gr = row_rsrc<T>(reinterpret_cast<const T*>(p.d_y) + h * P, (size_t)f.H * P, t0, len, P);
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            const int q = td + TH * i, row = q / (P / EPP), col = (q % (P / EPP)) * EPP;
            rx[i] = buf_load16(xr, (unsigned)(row * (int)f.x_stride + col) * sizeof(T));
            rg[i] = buf_load16(gr, (unsigned)(row * f.H * P + col) * sizeof(T));
        }
        if constexpr (STAGED) {
            const auto sr = make_rsrc_n(start_of(h), KP * 4), er = make_rsrc_n(dend_of(h), KP * 4);
#pragma unroll
            for (int i = 0; i < PS; ++i) {
                rs[i] = buf_load16(sr, 16u * (unsigned)(td + TH * i));
                re[i] = buf_load16(er, 16u * (unsigned)(td + TH * i));
            }
        }
        const auto ar = make_rsrc_n(f.gates + ((size_t)ci * f.H + h) * (kGates * C), kGates * C * 4);
        rgate = buf_load16(ar, 16u * (unsigned)td);
        const auto dr = row_rsrc<T>(reinterpret_cast<const T*>(f.dt) + h, f.dt_stride, t0, len, 1);
        buf_load1(rdt, dr, (unsigned)(opaque(lane) * (int)f.dt_stride) * sizeof(T), 0);
    };
    float se = 0.f;         // the thread's share of <S, E>
    auto stage = [&](float* gate) {
        const int td = opaque(tid);
        se = 0.f;
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            const int q = td + TH * i, row = q / (P / EPP), col = (q % (P / EPP)) * EPP;
            *reinterpret_cast<uint4*>(sX + row * LDP + col) = rx[i];
            *reinterpret_cast<uint4*>(sDY + row * LDP + col) = rg[i];
        }
        if constexpr (STAGED) {
#pragma unroll
            for (int i = 0; i < PS; ++i) {
                const int q = td + TH * i, row = q / (P / 4), col = (q % (P / 4)) * 4;
                *reinterpret_cast<uint4*>(sS + row * LDS_ + col) = rs[i];
                *reinterpret_cast<uint4*>(sE + row * LDS_ + col) = re[i];
                se = fmaf(__uint_as_float(rs[i].x), __uint_as_float(re[i].x), se);
                se = fmaf(__uint_as_float(rs[i].y), __uint_as_float(re[i].y), se);
                se = fmaf(__uint_as_float(rs[i].z), __uint_as_float(re[i].z), se);
                se = fmaf(__uint_as_float(rs[i].w), __uint_as_float(re[i].w), se);
            }
        }
        if (td < kGates * C / 4) *reinterpret_cast<uint4*>(gate + 4 * td) = rgate;
    };
    if (ha < hb) fetch(ha);

    // ---- B and C of the chunk, and the score tiles the wave keeps
    {
        const auto br = row_rsrc<T>(reinterpret_cast<const T*>(f.B) + grp * K, f.b_stride, t0, len, K);
        const auto cr = row_rsrc<T>(reinterpret_cast<const T*>(f.C) + grp * K, f.c_stride, t0, len, K);
        for (int q = tid; q < C * K / EPP; q += TH) {
            const int row = q / (K / EPP), col = (q % (K / EPP)) * EPP;
            *reinterpret_cast<uint4*>(sB + row * LDK + col) = buf_load16(br, (unsigned)(row * (int)f.b_stride + col) * sizeof(T));
            *reinterpret_cast<uint4*>(sC + row * LDK + col) = buf_load16(cr, (unsigned)(row * (int)f.c_stride + col) * sizeof(T));
        }
        for (int q = tid; q < C * LDM; q += TH) {
            sM[q] = (T)0.f;
            if constexpr (sizeof(T) == 2) sML[q] = (T)0.f;
        }
    }
    __syncthreads();
    // tile k of wave w is lower tile q = (w + 4) % 8 + 8 k: rows 16 ti + 4 g + e, column 16 tj + r16
    f32x4 Gt[2], dG[2];
    int ti[2], tj[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int q = ((w + 4) & 7) + 8 * k;
        ti[k] = q < 1 ? 0 : q < 3 ? 1 : q < 6 ? 2 : 3;
        tj[k] = q - ti[k] * (ti[k] + 1) / 2;
        Gt[k] = dG[k] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (q < 10)
#pragma unroll
            for (int m = 0; m < K / 32; ++m)
                Gt[k] = mma(Gt[k], ld_frag<T>(sC + (16 * ti[k] + r16) * LDK + 32 * m + 8 * g),
                            ld_frag<T>(sB + (16 * tj[k] + r16) * LDK + 32 * m + 8 * g));
    }
    // gradients of B and C, transposed: task k is state rows 16 nrow + 4 g + e
    // of dC (K = 128: k = 0; K = 64: waves 0..3) or dB, tokens 16 t + r16
    const int nrow = K == 128 ? w : (w & 3);
    f32x4 acc[TK][4];
#pragma unroll
    for (int k = 0; k < TK; ++k)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[k][t] = f32x4{0.f, 0.f, 0.f, 0.f};

    // ---- step sizes and decays of head h, in one wave
    auto step_sizes = [&](int h, int nb, T head_dt) {
        auto& s_gate = s_gate_[nb];
        auto& s_row = s_row_[nb];
        auto& s_colf = s_colf_[nb];
        auto& s_cols = s_cols_[nb];
        auto& s_z = s_z_[nb];
        auto& s_r = s_r_[nb];
        auto& s_se = s_se_[nb];
        auto& s_dd = s_dd_[nb];
        const int t = lane >> 4, q = lane & 15;
        // Pairs across token t (i >= t > j) without pairs that cancel, whose
        // rounding would stay: of tiles in t's row of tiles the rows from t on,
        // of those in its column of tiles the columns before t, all of the tiles
        // behind and before it; t's own tile has them summed (s_row).
        const int own = t * (t + 1) / 2 + t;
        double left = 0.0, under = 0.0;
        float cf = s_colf[own][q];
        for (int b = 0; b < t; ++b) left += (double)s_row[t * (t + 1) / 2 + b][q];
        for (int a = t + 1; a < 4; ++a) {
            cf += s_colf[a * (a + 1) / 2 + t][q];
            under += (double)s_cols[a * (a + 1) / 2 + t][q];
        }
        // tiles (2, 0), (3, 0) pass token tile 1; (3, 0), (3, 1) pass tile 2
        const double past = t == 1 ? (double)s_row[3][q] + (double)s_row[6][q]
                            : t == 2 ? (double)s_row[6][q] + (double)s_row[7][q] : 0.0;
        float zz = 0.f, rr = 0.f, sev = 0.f, ddv = 0.f;
#pragma unroll
        for (int k = 0; k < P / 16; ++k) {
            zz += s_z[k][lane];
            rr += s_r[k][lane];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            sev += s_se[k];
            ddv += s_dd[k];
        }
        const float c = s_gate[kGateC][lane], rest = s_gate[kGateRest][lane], delta = s_gate[kGateDelta][lane];
        const float cT = s_gate[kGateC][C - 1], restT = s_gate[kGateRest][C - 1];
        rr *= exp2_pair(c, rest);
        const double pr = row_prefix(left), pu = row_prefix(under);
        const double pairs = (double)s_row[own][q] + row_last(pr) - pr + left + pu - under + row_last(row_prefix(past));
        const double through = (double)rr, pre = wave_prefix(through);  // summed over i >= t
        const double suffix = pairs + last_lane(pre) - pre + through;
        const double wz = (double)s_gate[kGateW][lane] * (double)zz;
        const double before = wave_prefix(wz) - wz;                     // summed over j < t
        const double dla = suffix + before + (double)exp2_pair(cT, restT) * (double)sev;
        const bool in = lane < len;
        const float raw = to_f32(head_dt) + (f.dt_bias ? f.dt_bias[h] : 0.f);
        const float sig = f.softplus ? 1.f / (1.f + expf(-raw)) : 1.f;
        const float out = fast_exp2((cT - c) + (restT - rest));
        const float dd_raw = (float)(((double)cf + (double)out * (double)zz + (double)f.A[h] * dla) * (double)sig);
        if (in) reinterpret_cast<T*>(p.ddt)[(size_t)(t0 + lane) * f.H + h] = from_f32<T>(dd_raw);
        const double sa = last_lane(wave_prefix(in ? dla * (double)delta : 0.0));
        const double sb = last_lane(wave_prefix(in ? (double)dd_raw : 0.0));
        if (lane == 0) {
            float* o = p.sums + (size_t)ci * 3 * f.H + h;
            o[0] = (float)sa;
            o[f.H] = (float)sb;
            o[2 * f.H] = ddv;
        }
    };
    T my_dt = (T)0.f;

    for (int h = ha; h < hb; ++h) {
        const float *start = start_of(h), *dend = dend_of(h);
        const int nb = NB == 2 ? (h - ha) & 1 : 0;
        auto& s_gate = s_gate_[nb];
        auto& s_row = s_row_[nb];
        auto& s_colf = s_colf_[nb];
        auto& s_cols = s_cols_[nb];
        auto& s_z = s_z_[nb];
        auto& s_r = s_r_[nb];
        auto& s_se = s_se_[nb];
        auto& s_dd = s_dd_[nb];
        const T last_dt = my_dt;
        my_dt = rdt;
        stage(&s_gate[0][0]);
        __syncthreads();
        // the next head's loads: half the waves issue theirs before their pairs,
        // half behind (all at once queue, and hold up the waves with two tiles)
        if (h + 1 < hb && w < 4) fetch(h + 1);
        if (NB == 2 && w == 7 && h > ha) step_sizes(h - 1, nb ^ 1, last_dt);
        // ---- pairs of tokens
        float dd = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int q = ((w + 4) & 7) + 8 * k;
            if (q >= 10) continue;
            f32x4 dm{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < P / 32; ++m)
                dm = mma(dm, ld_frag<T>(sDY + (16 * ti[k] + r16) * LDP + 32 * m + 8 * g),
                         ld_frag<T>(sX + (16 * tj[k] + r16) * LDP + 32 * m + 8 * g));
            const int j = 16 * tj[k] + r16, i0 = 16 * ti[k] + 4 * g;
            const float cj = s_gate[kGateC][j], cjl = s_gate[kGateRest][j], dj = s_gate[kGateDelta][j];
            float mv[4], pairs[4], colf = 0.f, cols = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + e;
                const bool in = j <= i, below = j < i;
                const float l = fast_exp2(in ? (s_gate[kGateC][i] - cj) + (s_gate[kGateRest][i] - cjl) : 0.f);
                const float ql = in ? dm[e] * l : 0.f;
                const float pr = in ? ql * Gt[k][e] : 0.f;
                mv[e] = in ? Gt[k][e] * l * dj : 0.f;
                dG[k][e] += ql * dj;
                pairs[e] = below ? pr * dj : 0.f;
                colf += pr;
                cols += pairs[e];
                if (i == j) dd += dm[e];
            }
            if (ti[k] == tj[k]) {
                // on the diagonal a token's own rows would hold pairs behind it:
                // the rows from token 4 g + e on, of the columns before it
                pairs[2] += pairs[3];
                pairs[1] += pairs[2];
                pairs[0] += pairs[1];
                const float behind = sum_groups_behind(pairs[0], g);
#pragma unroll
                for (int e = 0; e < 4; ++e) pairs[e] = r16 < 4 * g + e ? pairs[e] + behind : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float row = sum16(pairs[e]);
                if (r16 == 0) s_row[q][4 * g + e] = row;
            }
            st_near4(sM + j * LDM + i0, sML + j * LDM + i0, mv);
            colf = sum_groups(colf);
            cols = sum_groups(cols);
            if (g == 0) {
                s_colf[q][r16] = colf;
                s_cols[q][r16] = cols;
            }
        }
        dd = sum64(dd);
        if (lane == 0) s_dd[w] = dd;
        if (h + 1 < hb && w >= 4) fetch(h + 1);
        // ---- what passes through the states: U = E^T B or Y = S^T C, columns
        // col + 4 g + e of token 16 t + r16
        f32x4 dx[4];
#pragma unroll
        for (int k = 0; k < TU; ++k) {
            const bool is_y = P == 64 ? w >= 4 : k == 1;
            const int ct = P == 64 ? (w & 3) : w, col = 16 * ct;
            const T* rows = is_y ? sC : sB;
            f32x4 U[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) U[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < K / 32; ++m) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int n = 32 * m + 8 * g + i;
                    if constexpr (STAGED) {
                        v[i] = (is_y ? sS : sE)[n * LDS_ + col + r16];
                    } else {
                        const float* st = is_y ? start : dend;
                        v[i] = st[(size_t)n * P + col + r16];
                        if (!is_y) se = fmaf(v[i], start[(size_t)n * P + col + r16], se);
                    }
                }
                const auto vf = Exact<T>::of(v);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    U[t] = mma_exact_a(U[t], vf, ld_frag<T>(rows + (16 * t + r16) * LDK + 32 * m + 8 * g));
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f32x4 gv = ld4_as_f32<T>(sDY + (16 * t + r16) * LDP + col + 4 * g);
                const f32x4 o = is_y ? gv : ld4_as_f32<T>(sX + (16 * t + r16) * LDP + col + 4 * g);
                float z = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) z = fmaf(U[t][e], o[e], z);
                z = sum_groups(z);
                if (g == 0) (is_y ? s_r : s_z)[ct][16 * t + r16] = z;
                if (!is_y) {
                    dx[t] = U[t] * s_gate[kGateW][16 * t + r16];
                    if (f.Dskip) dx[t] += gv * f.Dskip[h];
                }
            }
        }
        se = sum64(se);
        if (lane == 0) s_se[w] = se;
        __syncthreads();
        // ---- dx: the chunk's own tokens
        if (P == 128 || w < 4) {
            const int col = 16 * w;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Frag gf = ld_frag_tokens(sDY, LDP, 32 * s, col, lane);
#pragma unroll
                for (int t = 0; t < 2 + 2 * s; ++t) {
                    const int at = (16 * t + r16) * LDM + 32 * s + 4 * g;
                    if constexpr (sizeof(T) == 2) dx[t] = mma(dx[t], gf, ld_frag_perm<T>(sML + at));
                    dx[t] = mma(dx[t], gf, ld_frag_perm<T>(sM + at));
                }
            }
            const auto xr = row_rsrc<T>(reinterpret_cast<const T*>(p.dx) + h * P + col, p.dx_stride, t0, len, 16);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float o[4] = {dx[t][0], dx[t][1], dx[t][2], dx[t][3]};
                buf_store4(xr, (unsigned)((16 * t + r16) * (int)p.dx_stride + 4 * g) * sizeof(T), 0, o, (const T*)nullptr);
            }
        }
        // ---- dB and dC through the states
#pragma unroll
        for (int k = 0; k < TK; ++k) {
            const bool is_c = K == 128 ? k == 0 : w < 4;
            const float* st = is_c ? start : dend;
            const T* tok = is_c ? sDY : sX;
            typename Near<T>::type sf[P / 32];
#pragma unroll
            for (int m = 0; m < P / 32; ++m) {
                float v[8];
                if constexpr (STAGED)
                    ld8f((is_c ? sS : sE) + (16 * nrow + r16) * LDS_ + 32 * m + 8 * g, v);
                else
                    ld8f(st + (size_t)(16 * nrow + r16) * P + 32 * m + 8 * g, v);
                sf[m] = Near<T>::of(v);
            }
            f32x4 v[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) v[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < P / 32; ++m) {
                Frag f[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) f[t] = ld_frag<T>(tok + (16 * t + r16) * LDP + 32 * m + 8 * g);
                mma_near(v, sf[m], f);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int j = 16 * t + r16;
                acc[k][t] += v[t] * (is_c ? exp2_pair(s_gate[kGateC][j], s_gate[kGateRest][j]) : s_gate[kGateW][j]);
            }
        }
        if (NB == 1 && w == 7) step_sizes(h, 0, my_dt);
        __syncthreads();
    }
    if (NB == 2 && w == 7 && hb > ha) step_sizes(hb - 1, (hb - 1 - ha) & 1, my_dt);
    // ---- the heads' summed score gradients, times C and B
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (((w + 4) & 7) + 8 * k < 10) {
            float v[4] = {dG[k][0], dG[k][1], dG[k][2], dG[k][3]};
            const int o = (16 * tj[k] + r16) * LDM + 16 * ti[k] + 4 * g;
            st_near4(sM + o, sML + o, v);
        }
    }
    __syncthreads();
    const size_t tokens = f.sv.cu ? (size_t)f.sv.T : (size_t)f.sv.N * f.sv.T;
#pragma unroll
    for (int k = 0; k < TK; ++k) {
        const bool is_c = K == 128 ? k == 0 : w < 4;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const Frag rf = ld_frag_tokens(is_c ? sB : sC, LDK, 32 * s, 16 * nrow, lane);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                // dB_j: rows i of the slab at or behind j's tile; dC_i: rows j up to i's tile
                if (is_c ? t < 2 * s : t >= 2 + 2 * s) continue;
                auto part = [&](const T* tile) {
                    const Frag f = is_c ? ld_frag_tokens(tile, LDM, 32 * s, 16 * t, lane)
                                        : ld_frag_perm<T>(tile + (16 * t + r16) * LDM + 32 * s + 4 * g);
                    acc[k][t] = mma(acc[k][t], rf, f);
                };
                if constexpr (sizeof(T) == 2) part(sML);
                part(sM);
            }
        }
        const int row = grp * K + 16 * nrow + 4 * g;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int j = 16 * t + r16;
            if (j >= len) continue;
            float v[4] = {acc[k][t][0], acc[k][t][1], acc[k][t][2], acc[k][t][3]};
            if (p.parts == 1) {
                T* o = is_c ? reinterpret_cast<T*>(p.dC) + (size_t)(t0 + j) * p.dc_stride
                            : reinterpret_cast<T*>(p.dB) + (size_t)(t0 + j) * p.db_stride;
                st_run<4>(o + row, v);
            } else {
                st_run<4>((is_c ? p.dC_part : p.dB_part) + ((size_t)part * tokens + t0 + j) * f.G * K + row, v);
            }
        }
    }
}

// dB and dC: the parts added in order, rounded once.  Four values a thread.
// Rows of a packed call behind its last sequence are left as they are.
template <typename T>
__global__ __launch_bounds__(256) void kda_ssm_bwd_join_kernel(SsmBwdParams p, long long tokens) {
    const int width4 = p.f.G * p.f.K / 4;
    const long long at = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long row = at / width4;
    if (row >= tokens) return;
    if (p.f.sv.cu && row >= p.f.sv.cu[p.f.sv.N]) return;
    const int c = (int)(at - row * width4) * 4;
    const size_t o = (size_t)row * p.f.G * p.f.K + c, step = (size_t)tokens * p.f.G * p.f.K;
    f32x4 b{0.f, 0.f, 0.f, 0.f}, d = b;
    for (int k = 0; k < p.parts; ++k) {
        b += *reinterpret_cast<const f32x4*>(p.dB_part + o + k * step);
        d += *reinterpret_cast<const f32x4*>(p.dC_part + o + k * step);
    }
    float vb[4] = {b[0], b[1], b[2], b[3]}, vd[4] = {d[0], d[1], d[2], d[3]};
    st_run<4>(reinterpret_cast<T*>(p.dB) + (size_t)row * p.db_stride + c, vb);
    st_run<4>(reinterpret_cast<T*>(p.dC) + (size_t)row * p.dc_stride + c, vd);
}

// sums [rows][3][H] added over the rows (fixed order, fp64)
__global__ __launch_bounds__(256) void kda_ssm_bwd_sums_kernel(const float* sums, int rows, int H, float* dA,
                                                               float* dbias, float* dD) {
    __shared__ double red[256];
    const int h = blockIdx.x, m = blockIdx.y;
    float* out = m == 0 ? dA : m == 1 ? dbias : dD;
    if (!out) return;
    double v = 0.0;
    for (int r = threadIdx.x; r < rows; r += 256) v += (double)sums[((size_t)r * 3 + m) * H + h];
    red[threadIdx.x] = v;
    __syncthreads();
    for (int d = 128; d > 0; d >>= 1) {
        if ((int)threadIdx.x < d) red[threadIdx.x] += red[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) out[h] = (float)red[0];
}

template <typename T>
hipError_t bwd_launch(const SsmBwdParams& p, hipStream_t st) {
    const dim3 grid((unsigned)((long long)p.f.chunks * p.f.G * p.parts));
    if (p.f.K == 128 && p.f.P == 128) hipLaunchKernelGGL((kda_ssm_bwd_kernel<T, 128, 128>), grid, dim3(512), 0, st, p);
    else if (p.f.K == 128) hipLaunchKernelGGL((kda_ssm_bwd_kernel<T, 128, 64>), grid, dim3(512), 0, st, p);
    else if (p.f.P == 128) hipLaunchKernelGGL((kda_ssm_bwd_kernel<T, 64, 128>), grid, dim3(512), 0, st, p);
    else hipLaunchKernelGGL((kda_ssm_bwd_kernel<T, 64, 64>), grid, dim3(512), 0, st, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ssm_bwd(int dtype, const SsmBwdParams& p, hipStream_t st) {
    return dtype == 1 ? bwd_launch<bf16>(p, st) : bwd_launch<float>(p, st);
}

hipError_t launch_ssm_bwd_join(int dtype, const SsmBwdParams& p, long long tokens, hipStream_t st) {
    const long long n = tokens * (p.f.G * p.f.K / 4);
    if (n <= 0) return hipSuccess;
    const dim3 grid((unsigned)((n + 255) / 256));
    if (dtype == 1) hipLaunchKernelGGL(kda_ssm_bwd_join_kernel<bf16>, grid, dim3(256), 0, st, p, tokens);
    else hipLaunchKernelGGL(kda_ssm_bwd_join_kernel<float>, grid, dim3(256), 0, st, p, tokens);
    return hipGetLastError();
}

hipError_t launch_ssm_bwd_sums(const float* sums, int rows, int H, float* dA, float* dbias, float* dD, hipStream_t st) {
    hipLaunchKernelGGL(kda_ssm_bwd_sums_kernel, dim3((unsigned)H, 3), dim3(256), 0, st, sums, rows, H, dA, dbias, dD);
    return hipGetLastError();
}

}  // namespace kda
