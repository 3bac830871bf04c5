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
// their sums over all tokens are fp32 gradients.
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

// sum over the 16 lanes of a row group
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) v += __shfl_xor(v, m);
    return v;
}
// sum over the four lane groups
__device__ __forceinline__ float sum_groups(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

template <typename T, int K, int P>
__global__ __launch_bounds__(256) void kda_ssm_bwd_kernel(SsmBwdParams p) {
    constexpr int PAD = 16 / sizeof(T);
    constexpr int EPP = 16 / sizeof(T);
    constexpr int LDK = K + PAD, LDP = P + PAD, LDM = C + PAD;
    constexpr int PT = P / 64;          // column tiles a wave
    constexpr int NT = K / 64;          // state row tiles a wave
    typedef typename FragOf<T>::type Frag;
    __shared__ T sB[C * LDK], sC[C * LDK], sX[C * LDP], sDY[C * LDP], sM[C * LDM];
    __shared__ __align__(16) float s_c[C], s_cl[C], s_delta[C], s_ec[C], s_w[C], s_out[C], s_sig[C];
    __shared__ float s_row[10][16], s_colf[10][16], s_cols[10][16], s_z[4][C], s_r[4][C], s_se[4], s_dd[4];
    __shared__ float s_decay;

    const SsmParams& f = p.f;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, r16 = lane & 15;
    const int flat = xcd_swizzle(blockIdx.x, gridDim.x);
    const int part = flat % p.parts, grp = (flat / p.parts) % f.G, ci = flat / (p.parts * f.G);
    const int hpg = f.H / f.G;
    const int ha = grp * hpg + min(part * p.heads_per, hpg), hb = grp * hpg + min((part + 1) * p.heads_per, hpg);
    const size_t kp = (size_t)K * P;
    if (ci >= total_chunks(f)) {
        // chunks that a packed call's bound counts and its lengths do not have
        for (int h = ha + tid; h < hb; h += 256)
            for (int m = 0; m < 3; ++m) p.sums[((size_t)ci * 3 + m) * f.H + h] = 0.f;
        return;
    }
    ChunkWalk at;
    at.init(f, ci);
    const int t0 = at.t0(), len = at.len();

    // ---- B and C of the chunk, and the score tiles the wave keeps
    {
        const T* bp = reinterpret_cast<const T*>(f.B) + (size_t)t0 * f.b_stride + grp * K;
        const T* cp = reinterpret_cast<const T*>(f.C) + (size_t)t0 * f.c_stride + grp * K;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        for (int q = tid; q < C * K / EPP; q += 256) {
            const int row = q / (K / EPP), col = (q % (K / EPP)) * EPP;
            *reinterpret_cast<uint4*>(sB + row * LDK + col) =
                row < len ? *reinterpret_cast<const uint4*>(bp + (size_t)row * f.b_stride + col) : zero;
            *reinterpret_cast<uint4*>(sC + row * LDK + col) =
                row < len ? *reinterpret_cast<const uint4*>(cp + (size_t)row * f.c_stride + col) : zero;
        }
        for (int q = tid; q < C * LDM; q += 256) sM[q] = (T)0.f;
    }
    __syncthreads();
    // tile k of wave w is lower tile q = w + 4 k: rows 16 ti + 4 g + e, column 16 tj + r16
    f32x4 Gt[3], dG[3];
    int ti[3], tj[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int q = w + 4 * k;
        ti[k] = q < 1 ? 0 : q < 3 ? 1 : q < 6 ? 2 : 3;
        tj[k] = q - ti[k] * (ti[k] + 1) / 2;
        Gt[k] = dG[k] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (q < 10)
#pragma unroll
            for (int m = 0; m < K / 32; ++m)
                Gt[k] = mma(Gt[k], ld_frag<T>(sC + (16 * ti[k] + r16) * LDK + 32 * m + 8 * g),
                            ld_frag<T>(sB + (16 * tj[k] + r16) * LDK + 32 * m + 8 * g));
    }
    // gradients of B and C, transposed: state rows 16 (NT w + n) + 4 g + e, token 16 t + r16
    f32x4 dBt[NT][4], dCt[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < 4; ++t) dBt[n][t] = dCt[n][t] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (int h = ha; h < hb; ++h) {
        const float* start = at.first() ? (f.s0 ? f.s0 + ((size_t)at.seq * f.H + h) * kp : nullptr)
                                        : p.start + ((size_t)ci * f.H + h) * kp;
        const float* dend = at.last() ? (f.sT ? f.sT + ((size_t)at.seq * f.H + h) * kp : nullptr)
                                      : p.dend + ((size_t)ci * f.H + h) * kp;
        __syncthreads();
        {
            const T* xp = reinterpret_cast<const T*>(f.x) + (size_t)t0 * f.x_stride + h * P;
            const T* gp = reinterpret_cast<const T*>(p.d_y) + ((size_t)t0 * f.H + h) * P;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            for (int q = tid; q < C * P / EPP; q += 256) {
                const int row = q / (P / EPP), col = (q % (P / EPP)) * EPP;
                *reinterpret_cast<uint4*>(sX + row * LDP + col) =
                    row < len ? *reinterpret_cast<const uint4*>(xp + (size_t)row * f.x_stride + col) : zero;
                *reinterpret_cast<uint4*>(sDY + row * LDP + col) =
                    row < len ? *reinterpret_cast<const uint4*>(gp + (size_t)row * f.H * P + col) : zero;
            }
        }
        if (w == 0) {
            float delta = 0.f, sig = 0.f;
            if (lane < len) {
                const float raw = to_f32(reinterpret_cast<const T*>(f.dt)[(size_t)(t0 + lane) * f.dt_stride + h]) +
                                  (f.dt_bias ? f.dt_bias[h] : 0.f);
                delta = delta_of(raw, f.softplus);
                sig = f.softplus ? 1.f / (1.f + expf(-raw)) : 1.f;
            }
            const double c = wave_prefix((double)delta * (double)f.A[h] * 1.4426950408889634);
            const double ct = last_lane(c);
            const float ch = (float)c;
            s_c[lane] = ch;
            s_cl[lane] = (float)(c - (double)ch);
            s_delta[lane] = delta;
            s_ec[lane] = exp2_of(c);
            const float out = exp2_of(ct - c);
            s_out[lane] = out;
            s_w[lane] = out * delta;
            s_sig[lane] = sig;
            if (lane == 0) s_decay = exp2_of(ct);
        }
        __syncthreads();
        // ---- pairs of tokens
        float dd = 0.f;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int q = w + 4 * k;
            if (q >= 10) continue;
            f32x4 dm{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < P / 32; ++m)
                dm = mma(dm, ld_frag<T>(sDY + (16 * ti[k] + r16) * LDP + 32 * m + 8 * g),
                         ld_frag<T>(sX + (16 * tj[k] + r16) * LDP + 32 * m + 8 * g));
            const int j = 16 * tj[k] + r16, i0 = 16 * ti[k] + 4 * g;
            const float cj = s_c[j], cjl = s_cl[j], dj = s_delta[j];
            float mv[4], colf = 0.f, cols = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + e;
                const bool in = j <= i, below = j < i;
                const float l = fast_exp2(in ? (s_c[i] - cj) + (s_cl[i] - cjl) : 0.f);
                const float ql = in ? dm[e] * l : 0.f;
                const float pr = in ? ql * Gt[k][e] : 0.f;
                mv[e] = in ? Gt[k][e] * l * dj : 0.f;
                dG[k][e] += ql * dj;
                const float prs = below ? pr * dj : 0.f;
                colf += pr;
                cols += prs;
                const float row = sum16(prs);
                if (r16 == 0) s_row[q][4 * g + e] = row;
                if (i == j) dd += dm[e];
            }
            st_run<4>(sM + j * LDM + i0, mv);
            colf = sum_groups(colf);
            cols = sum_groups(cols);
            if (g == 0) {
                s_colf[q][r16] = colf;
                s_cols[q][r16] = cols;
            }
        }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) dd += __shfl_xor(dd, m);
        if (lane == 0) s_dd[w] = dd;
        // ---- what passes through the states: U = E^T B and Y = S^T C, columns
        // 16 (PT w + n) + 4 g + e of token 16 t + r16
        f32x4 dx[PT][4];
        float se = 0.f;
        float z[4] = {0.f, 0.f, 0.f, 0.f}, r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = 0; n < PT; ++n) {
            const int col = 16 * (PT * w + n);
            f32x4 U[4], Y[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) U[t] = Y[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < K / 32; ++m) {
                float ev[8], sv[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const size_t o = (size_t)(32 * m + 16 * (i >> 2) + 4 * g + (i & 3)) * P + col + r16;
                    ev[i] = dend ? dend[o] : 0.f;
                    sv[i] = start ? start[o] : 0.f;
                    se = fmaf(ev[i], sv[i], se);
                }
                const auto ef = Exact<T>::of(ev);
                const auto sf = Exact<T>::of(sv);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    U[t] = mma_exact_a(U[t], ef, ld_frag_perm<T>(sB + (16 * t + r16) * LDK + 32 * m + 4 * g));
                    Y[t] = mma_exact_a(Y[t], sf, ld_frag_perm<T>(sC + (16 * t + r16) * LDK + 32 * m + 4 * g));
                }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f32x4 xv = ld4_as_f32<T>(sX + (16 * t + r16) * LDP + col + 4 * g);
                const f32x4 gv = ld4_as_f32<T>(sDY + (16 * t + r16) * LDP + col + 4 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    z[t] = fmaf(U[t][e], xv[e], z[t]);
                    r[t] = fmaf(Y[t][e], gv[e], r[t]);
                }
                dx[n][t] = U[t] * s_w[16 * t + r16];
                if (f.Dskip) dx[n][t] += gv * f.Dskip[h];
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            z[t] = sum_groups(z[t]);
            r[t] = sum_groups(r[t]);
            if (g == 0) {
                s_z[w][16 * t + r16] = z[t];
                s_r[w][16 * t + r16] = r[t];
            }
        }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) se += __shfl_xor(se, m);
        if (lane == 0) s_se[w] = se;
        __syncthreads();
        // ---- dx: the chunk's own tokens
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int n = 0; n < PT; ++n) {
                const Frag gf = ld_frag_tokens(sDY, LDP, 32 * s, 16 * (PT * w + n), lane);
#pragma unroll
                for (int t = 0; t < 2 + 2 * s; ++t)
                    dx[n][t] = mma(dx[n][t], gf, ld_frag_perm<T>(sM + (16 * t + r16) * LDM + 32 * s + 4 * g));
            }
        }
        {
            T* xp = reinterpret_cast<T*>(p.dx) + (size_t)t0 * p.dx_stride + h * P;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int j = 16 * t + r16;
                if (j < len)
#pragma unroll
                    for (int n = 0; n < PT; ++n) {
                        float o[4] = {dx[n][t][0], dx[n][t][1], dx[n][t][2], dx[n][t][3]};
                        st_run<4>(xp + (size_t)j * p.dx_stride + 16 * (PT * w + n) + 4 * g, o);
                    }
            }
        }
        // ---- dB and dC through the states
        auto through = [&](const float* state, const T* tok, const float* scale, f32x4(&acc)[NT][4]) {
            if (!state) return;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                Frag sf[P / 32];
#pragma unroll
                for (int m = 0; m < P / 32; ++m) {
                    float v[8];
                    ld8f(state + (size_t)(16 * (NT * w + n) + r16) * P + 32 * m + 8 * g, v);
                    sf[m] = frag_from<T>(v);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    f32x4 v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int m = 0; m < P / 32; ++m)
                        v = mma(v, sf[m], ld_frag<T>(tok + (16 * t + r16) * LDP + 32 * m + 8 * g));
                    acc[n][t] += v * scale[16 * t + r16];
                }
            }
        };
        through(start, sDY, s_ec, dCt);
        through(dend, sX, s_w, dBt);
        // ---- step sizes and decays
        if (w == 0) {
            const int t = lane >> 4, q = lane & 15;
            float row = 0.f, cf = 0.f, cs = 0.f;
            for (int b = 0; b <= t; ++b) row += s_row[t * (t + 1) / 2 + b][q];
            for (int a = t; a < 4; ++a) {
                cf += s_colf[a * (a + 1) / 2 + t][q];
                cs += s_cols[a * (a + 1) / 2 + t][q];
            }
            const float zz = s_z[0][lane] + s_z[1][lane] + s_z[2][lane] + s_z[3][lane];
            const float rr = (s_r[0][lane] + s_r[1][lane] + s_r[2][lane] + s_r[3][lane]) * s_ec[lane];
            const double after = (double)row - (double)cs + (double)rr;     // summed over i >= t
            const double pre = wave_prefix(after);
            const double suffix = last_lane(pre) - pre + after;
            const double wz = (double)s_w[lane] * (double)zz;
            const double before = wave_prefix(wz) - wz;               // summed over j < t
            const double thru = (double)s_decay * ((double)s_se[0] + s_se[1] + s_se[2] + s_se[3]);
            const double dla = suffix + before + thru;
            const float dd_raw =
                (float)(((double)cf + (double)s_out[lane] * (double)zz + (double)f.A[h] * dla) * (double)s_sig[lane]);
            const bool in = lane < len;
            if (in) reinterpret_cast<T*>(p.ddt)[(size_t)(t0 + lane) * f.H + h] = from_f32<T>(dd_raw);
            double a = in ? dla * (double)s_delta[lane] : 0.0, b = in ? (double)dd_raw : 0.0;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                a += __shfl_xor(a, m);
                b += __shfl_xor(b, m);
            }
            if (lane == 0) {
                float* out = p.sums + (size_t)ci * 3 * f.H + h;
                out[0] = (float)a;
                out[f.H] = (float)b;
                out[2 * f.H] = s_dd[0] + s_dd[1] + s_dd[2] + s_dd[3];
            }
        }
    }
    // ---- the heads' summed score gradients, times C and B
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (w + 4 * k < 10) {
            float v[4] = {dG[k][0], dG[k][1], dG[k][2], dG[k][3]};
            st_run<4>(sM + (16 * tj[k] + r16) * LDM + 16 * ti[k] + 4 * g, v);
        }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const Frag cf = ld_frag_tokens(sC, LDK, 32 * s, 16 * (NT * w + n), lane);
            const Frag bf = ld_frag_tokens(sB, LDK, 32 * s, 16 * (NT * w + n), lane);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                // dB_j: rows i of the slab at or behind j's tile; dC_i: rows j up to i's tile
                if (t < 2 + 2 * s)
                    dBt[n][t] = mma(dBt[n][t], cf, ld_frag_perm<T>(sM + (16 * t + r16) * LDM + 32 * s + 4 * g));
                if (t >= 2 * s) dCt[n][t] = mma(dCt[n][t], bf, ld_frag_tokens(sM, LDM, 32 * s, 16 * t, lane));
            }
        }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int j = 16 * t + r16;
        if (j >= len) continue;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = grp * K + 16 * (NT * w + n) + 4 * g;
            float vb[4] = {dBt[n][t][0], dBt[n][t][1], dBt[n][t][2], dBt[n][t][3]};
            float vc[4] = {dCt[n][t][0], dCt[n][t][1], dCt[n][t][2], dCt[n][t][3]};
            if (p.parts == 1) {
                st_run<4>(reinterpret_cast<T*>(p.dB) + (size_t)(t0 + j) * p.db_stride + row, vb);
                st_run<4>(reinterpret_cast<T*>(p.dC) + (size_t)(t0 + j) * p.dc_stride + row, vc);
            } else {
                const size_t tokens = f.sv.cu ? (size_t)f.sv.T : (size_t)f.sv.N * f.sv.T;
                const size_t o = ((size_t)part * tokens + t0 + j) * f.G * K + row;
                st_run<4>(p.dB_part + o, vb);
                st_run<4>(p.dC_part + o, vc);
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
    if (p.f.K == 128 && p.f.P == 128) hipLaunchKernelGGL((kda_ssm_bwd_kernel<T, 128, 128>), grid, dim3(256), 0, st, p);
    else if (p.f.K == 128) hipLaunchKernelGGL((kda_ssm_bwd_kernel<T, 128, 64>), grid, dim3(256), 0, st, p);
    else if (p.f.P == 128) hipLaunchKernelGGL((kda_ssm_bwd_kernel<T, 64, 128>), grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL((kda_ssm_bwd_kernel<T, 64, 64>), grid, dim3(256), 0, st, p);
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
