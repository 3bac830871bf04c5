// Selective scan with a scalar decay a head: chunked prefill, its state-only
// passes, and the one-token step.
//
//   S_t = a_t S_{t-1} + delta_t B_t x_t^T,   y_t = S_t^T C_t + D x_t,
//   a_t = exp(delta_t A)
//
// Chunk form (64 tokens, start state S, c_t the inclusive sum of log a):
//
//   y_i = sum_{j <= i} (C_i . B_j) e^{c_i - c_j} delta_j x_j + e^{c_i} S^T C_i + D x_i
//   S'  = e^{c_63} S + sum_j e^{c_63 - c_j} delta_j B_j x_j^T
//
// All exponents are differences of a decreasing sum, taken before the
// exponential, so nothing overflows where A delta <= 0.
#include "kda_ssm_device.h"

namespace kda {

namespace {

constexpr int C = kSsmChunk;

// One workgroup (4 waves) per (segment, 64 NT columns of x: one or two heads)
// walks the segment's chunks with the state in registers: wave w owns columns
// [16 NT w, 16 NT (w + 1)) of all K state rows, as accumulator tiles that serve
// as operands as they are.  B, C and x of a chunk are staged in LDS (the next
// chunk's loads in flight meanwhile); the scores C B^T are computed once for
// the workgroup's heads, scaled and masked per head, and passed through LDS.
//   OUT:  y, and the final state where a sequence ends
//   else: each segment's local state and decay
template <typename T, int K, int P, int NT, bool OUT>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void kda_ssm_chunk_kernel(SsmParams p) {
    constexpr int COLS = 64 * NT;
    constexpr int NH = COLS / P;                // heads of the workgroup
    constexpr int PAD = 16 / sizeof(T);
    constexpr int LDK = K + PAD, LDX = COLS + PAD, LDG = C + PAD;
    constexpr int NTK = K / 16;                 // state row tiles
    constexpr int EPP = 16 / sizeof(T);         // elements of a 16-byte piece
    constexpr int PK = C * K / EPP / 256, PX = C * COLS / EPP / 256;
    constexpr int KP = K * P;
    __shared__ T sB[C * LDK];
    __shared__ T sX[C * LDX];
    __shared__ T sC[OUT ? C * LDK : 1];
    __shared__ T sG[OUT ? NH * C * LDG : 1];
    // per head, for this chunk and the next: c (as hi + lo), delta, e^{c}, the
    // state's token weights
    __shared__ __align__(16) float s_c[2][NH][C], s_cl[2][NH][C], s_delta[2][NH][C], s_ec[2][NH][C], s_w[2][NH][C];
    __shared__ float s_decay[2][NH];
    typedef typename FragOf<T>::type Frag;

    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, r16 = lane & 15;
    const int units = p.H / NH;
    const int flat = xcd_swizzle(blockIdx.x, gridDim.x);
    const int seg = p.seg0 + flat / units, h0 = (flat % units) * NH;
    const int col0 = w * 16 * NT;
    const int hl = col0 / P, pc = col0 % P, h = h0 + hl;
    const int grp = h0 / (p.H / p.G);
    const int all = total_chunks(p);
    const int begin = min(seg * p.cps, all), end = min(begin + p.cps, all);
    const bool rev = !OUT && p.reverse;
    const bool summary = !OUT;
    const int own = (4 * g) * P + pc + r16;     // the lane's first state element
    float* seg_slot = p.seg_state ? p.seg_state + ((size_t)seg * p.H + h) * KP : nullptr;

    f32x4 S[NTK][NT];
#pragma unroll
    for (int m = 0; m < NTK; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) S[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto load_state = [&](const float* src) {   // src: [K][P] of head h, or null
        if (src) {
#pragma unroll
            for (int m = 0; m < NTK; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[m][n][e] = src[own + (16 * m + e) * P + 16 * n];
        } else {
#pragma unroll
            for (int m = 0; m < NTK; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) S[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    };
    auto store_state = [&](float* dst) {
#pragma unroll
        for (int m = 0; m < NTK; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) dst[own + (16 * m + e) * P + 16 * n] = S[m][n][e];
    };
    if (begin >= end) {
        if (summary) store_state(seg_slot);
        if (summary && pc == 0 && lane == 0) p.seg_decay[(size_t)seg * p.H + h] = 1.f;
        return;
    }
    ChunkWalk walk;
    if (summary && !p.reverse) {
        // nobody reads this segment's end if the next one opens a sequence
        walk.init(p, end - 1);
        if (walk.last()) {
            if (pc == 0 && lane == 0) p.seg_decay[(size_t)seg * p.H + h] = -1.f;
            return;
        }
    }
    // the start state: none for a summary, else what the segments before left
    if (!summary && seg_slot) load_state(seg_slot);

    if constexpr (OUT) {
        // the score tiles above the diagonal that products read with their
        // neighbours: zero once, never written again
        for (int k = tid; k < NH * C * LDG; k += 256) sG[k] = (T)0.f;
    }

    walk.init(p, rev ? end - 1 : begin);
    // pieces of a chunk: the thread's rows and columns never change, so each
    // load is a chunk's resource and a fixed offset
    unsigned ob[PK], oc[OUT ? PK : 1], ox[PX];
#pragma unroll
    for (int i = 0; i < PK; ++i) {
        const int q = tid + 256 * i, row = q / (K / EPP), col = (q % (K / EPP)) * EPP;
        ob[i] = (unsigned)((row * p.b_stride + col) * sizeof(T));
        if constexpr (OUT) oc[i] = (unsigned)((row * p.c_stride + col) * sizeof(T));
    }
#pragma unroll
    for (int i = 0; i < PX; ++i) {
        const int q = tid + 256 * i, row = q / (COLS / EPP), col = (q % (COLS / EPP)) * EPP;
        ox[i] = (unsigned)((row * p.x_stride + col) * sizeof(T));
    }
    const T* xbase = reinterpret_cast<const T*>(p.x) + h0 * P;
    const T* bbase = reinterpret_cast<const T*>(p.B) + grp * K;
    const T* cbase = reinterpret_cast<const T*>(p.C) + grp * K;
    // the waves with fewer score tiles (3, then 2) prepare the heads' decays
    const int ph = 3 - w;
    const bool preps = ph < NH;
    const int hp = h0 + (preps ? ph : 0);
    const float bias = p.dt_bias ? p.dt_bias[hp] : 0.f;
    const double rate = (double)p.A[hp] * 1.4426950408889634;
    uint4 rb[PK], rx[PX], rc[OUT ? PK : 1];
    float rdt = 0.f;
    int rlen = 0;
    auto fetch = [&](const ChunkWalk& at) {
        const int t0 = at.t0(), len = at.len();
        const auto xr = row_rsrc<T>(xbase, p.x_stride, t0, len, COLS);
        const auto br = row_rsrc<T>(bbase, p.b_stride, t0, len, K);
#pragma unroll
        for (int i = 0; i < PK; ++i) rb[i] = buf_load16(br, ob[i]);
        if constexpr (OUT) {
            const auto cr = row_rsrc<T>(cbase, p.c_stride, t0, len, K);
#pragma unroll
            for (int i = 0; i < PK; ++i) rc[i] = buf_load16(cr, oc[i]);
        }
#pragma unroll
        for (int i = 0; i < PX; ++i) rx[i] = buf_load16(xr, ox[i]);
        rlen = len;
        if (preps && lane < len)
            rdt = to_f32(reinterpret_cast<const T*>(p.dt)[(size_t)(t0 + lane) * p.dt_stride + hp]);
    };
    // decays and step sizes of the chunk last fetched, into buffer b
    auto prepare = [&](int b) {
        if (!preps) return;
        const float delta = lane < rlen ? delta_of(rdt + bias, p.softplus) : 0.f;
        const double c = wave_prefix((double)delta * rate);
        const double ct = last_lane(c);
        const float ch = (float)c;
        s_c[b][ph][lane] = ch;
        s_cl[b][ph][lane] = (float)(c - (double)ch);
        s_delta[b][ph][lane] = delta;
        const float ec = exp2_of(c);
        s_ec[b][ph][lane] = ec;
        // the recurrence's token weights; the adjoint's are e^{c}
        s_w[b][ph][lane] = rev ? (lane < rlen ? ec : 0.f) : exp2_of(ct - c) * delta;
        if (lane == 63) s_decay[b][ph] = ec;
    };
    auto stage = [&]() {
#pragma unroll
        for (int i = 0; i < PK; ++i) {
            const int q = tid + 256 * i, row = q / (K / EPP), col = (q % (K / EPP)) * EPP;
            *reinterpret_cast<uint4*>(sB + row * LDK + col) = rb[i];
            if constexpr (OUT) *reinterpret_cast<uint4*>(sC + row * LDK + col) = rc[i];
        }
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            const int q = tid + 256 * i, row = q / (COLS / EPP), col = (q % (COLS / EPP)) * EPP;
            *reinterpret_cast<uint4*>(sX + row * LDX + col) = rx[i];
        }
    };
    fetch(walk);
    prepare(begin & 1);
    float seg_dec = 1.f;

    for (int it = begin; it < end; ++it) {
        const int b = it & 1;
        const int t0 = walk.t0(), len = walk.len(), seq = walk.seq;
        const bool opens = rev ? walk.last() : walk.first();
        const bool closes = rev ? walk.first() : walk.last();
        if (opens) {
            load_state(p.s0 ? p.s0 + ((size_t)seq * p.H + h) * KP : nullptr);
            seg_dec = -1.f;
        }
        stage();
        __syncthreads();
        // the next chunk's loads run behind this chunk's products
        if (it + 1 < end) {
            if (rev)
                walk.prev();
            else
                walk.next();
            fetch(walk);
        }
        f32x4 Y[OUT ? 4 : 1][NT];
        if constexpr (OUT) {
            // ---- scores, transposed: a lane gets four tokens j of one row i
            for (int q = w; q < 10; q += 4) {
                const int ti = q < 1 ? 0 : q < 3 ? 1 : q < 6 ? 2 : 3;
                const int tj = q - ti * (ti + 1) / 2;
                f32x4 acc{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int m = 0; m < K / 32; ++m)
                    acc = mma(acc, ld_frag<T>(sB + (16 * tj + r16) * LDK + 32 * m + 8 * g),
                              ld_frag<T>(sC + (16 * ti + r16) * LDK + 32 * m + 8 * g));
                const int i = 16 * ti + r16, j0 = 16 * tj + 4 * g;
#pragma unroll
                for (int k = 0; k < NH; ++k) {
                    const f32x4 cj = *reinterpret_cast<const f32x4*>(&s_c[b][k][j0]);
                    const f32x4 dj = *reinterpret_cast<const f32x4*>(&s_delta[b][k][j0]);
                    const float ci = s_c[b][k][i];
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float d = ci - cj[e];
                        if constexpr (sizeof(T) == 4) d += s_cl[b][k][i] - s_cl[b][k][j0 + e];
                        v[e] = j0 + e <= i ? acc[e] * fast_exp2(d) * dj[e] : 0.f;
                    }
                    st_run<4>(sG + (k * C + i) * LDG + j0, v);
                }
            }
            // ---- what the start state gives, transposed: a lane holds four
            // columns of one token
#pragma unroll
            for (int ti = 0; ti < 4; ++ti)
#pragma unroll
                for (int n = 0; n < NT; ++n) Y[ti][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < K / 32; ++m) {
                Frag sf[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) sf[n] = frag_from_tiles<T>(S[2 * m][n], S[2 * m + 1][n]);
#pragma unroll
                for (int ti = 0; ti < 4; ++ti) {
                    const Frag cf = ld_frag_perm<T>(sC + (16 * ti + r16) * LDK + 32 * m + 4 * g);
#pragma unroll
                    for (int n = 0; n < NT; ++n) Y[ti][n] = mma(Y[ti][n], sf[n], cf);
                }
            }
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) {
                const float e = s_ec[b][hl][16 * ti + r16];
#pragma unroll
                for (int n = 0; n < NT; ++n) Y[ti][n] *= e;
            }
            __syncthreads();
        }
        // ---- the chunk's own tokens: outputs and the state update
        const float decay = s_decay[b][hl];
        seg_dec = seg_dec < 0.f ? seg_dec : seg_dec * decay;
#pragma unroll
        for (int m = 0; m < NTK; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) S[m][n] *= decay;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            Frag xf[NT];
            typename Exact<T>::type xw[NT];
            const f32x4 wa = *reinterpret_cast<const f32x4*>(&s_w[b][hl][32 * s + 4 * g]);
            const f32x4 wb = *reinterpret_cast<const f32x4*>(&s_w[b][hl][32 * s + 16 + 4 * g]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                xf[n] = ld_frag_tokens(sX, LDX, 32 * s, col0 + 16 * n, lane);
                float v[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = (float)xf[n][i] * wa[i];
                    v[4 + i] = (float)xf[n][4 + i] * wb[i];
                }
                xw[n] = Exact<T>::of(v);
            }
            if constexpr (OUT) {
#pragma unroll
                for (int ti = 2 * s; ti < 4; ++ti) {
                    const Frag gf = ld_frag_perm<T>(sG + (hl * C + 16 * ti + r16) * LDG + 32 * s + 4 * g);
#pragma unroll
                    for (int n = 0; n < NT; ++n) Y[ti][n] = mma(Y[ti][n], xf[n], gf);
                }
            }
#pragma unroll
            for (int m = 0; m < NTK; ++m) {
                const Frag bf = ld_frag_tokens(sB, LDK, 32 * s, 16 * m, lane);
#pragma unroll
                for (int n = 0; n < NT; ++n) S[m][n] = mma_exact(S[m][n], bf, xw[n]);
            }
        }
        if constexpr (OUT) {
            const auto yr = row_rsrc<T>(reinterpret_cast<const T*>(p.y) + h * P + pc, (size_t)p.H * P, t0, len, 16 * NT);
            const float dskip = p.Dskip ? p.Dskip[h] : 0.f;
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) {
                const int i = 16 * ti + r16;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    f32x4 v = Y[ti][n];
                    if (p.Dskip) v += ld4_as_f32<T>(sX + i * LDX + col0 + 16 * n + 4 * g) * dskip;
                    float o[4] = {v[0], v[1], v[2], v[3]};
                    buf_store4(yr, (unsigned)((i * p.H * P + 4 * g) * sizeof(T)), 16 * n * sizeof(T), o, (const T*)nullptr);
                }
            }
        }
        if (it + 1 < end) prepare(b ^ 1);
        if (closes && p.sT && !summary) store_state(p.sT + ((size_t)seq * p.H + h) * KP);
        __syncthreads();
    }
    if (summary) {
        store_state(seg_slot);
        if (pc == 0 && lane == 0) p.seg_decay[(size_t)seg * p.H + h] = seg_dec;
    }
}

// Segment start states from the segments' local states and decays, written
// over the local states: start_{j+1} = decay_j start_j + local_j (local_j
// alone where a sequence starts in segment j).  A thread owns four state
// values of a head and keeps eight segments' loads in flight.
__global__ __launch_bounds__(256) void kda_ssm_combine_kernel(SsmParams p, float* d_s0) {
    const size_t kp4 = (size_t)p.K * p.P / 4;
    const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= (size_t)p.H * kp4) return;
    const int h = (int)(at / kp4);
    float4* L = reinterpret_cast<float4*>(p.seg_state) + at;
    const size_t step = (size_t)p.H * kp4;
    // segments that hold chunks (a packed call may have fewer than its bound)
    const int all = total_chunks(p), n_seg = min(p.n_seg, (all + p.cps - 1) / p.cps);
    // the last segment's local state is of use only to d_s0
    const int used = d_s0 ? n_seg : n_seg - 1;
    ChunkWalk walk;
    if (d_s0 && n_seg > 0) walk.init(p, n_seg - 1);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 8;
    for (int j = 0; j < n_seg; j += U) {
        float4 l[U];
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u < used) {
                const int k = p.reverse ? n_seg - 1 - (j + u) : j + u;
                l[u] = L[(size_t)k * step];
                d[u] = p.seg_decay[(size_t)k * p.H + h];
            }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j + u < n_seg) {
                const int k = p.reverse ? n_seg - 1 - (j + u) : j + u;
                // a sequence that starts (in reverse: ends) in this segment
                // takes its own start state, which an empty one passes on
                L[(size_t)k * step] = s;
                if (j + u < used) {
                    if (d[u] < 0.f)
                        s = l[u];
                    else
                        s = make_float4(fmaf(d[u], s.x, l[u].x), fmaf(d[u], s.y, l[u].y), fmaf(d[u], s.z, l[u].z),
                                        fmaf(d[u], s.w, l[u].w));
                }
                if (d_s0) {
                    if (walk.first()) reinterpret_cast<float4*>(d_s0)[(size_t)walk.seq * step + at] = s;
                    walk.prev();
                }
            }
        }
    }
}

__global__ __launch_bounds__(256) void kda_ssm_prep_kernel(SeqView sv, int* chunk_off, int max_chunks) {
    __shared__ int buf[256];
    __shared__ int carry;
    const int tid = threadIdx.x;
    if (tid == 0) {
        carry = 0;
        chunk_off[0] = 0;
    }
    __syncthreads();
    for (int base = 0; base < sv.N; base += 256) {
        const int i = base + tid;
        int c = 0;
        if (i < sv.N) {
            const int s0 = min(max(sv.cu[i], 0), sv.T);
            const int len = max(min(sv.cu[i + 1], sv.T) - s0, 0);
            c = max(1, (len + C - 1) / C);
        }
        buf[tid] = c;
        __syncthreads();
        for (int d = 1; d < 256; d <<= 1) {
            const int add = tid >= d ? buf[tid - d] : 0;
            __syncthreads();
            buf[tid] += add;
            __syncthreads();
        }
        // offsets that overlap could count more chunks than the bound: capped,
        // so that every chunk index stays inside the buffers
        if (i < sv.N) chunk_off[i + 1] = min(carry + buf[tid], max_chunks);
        __syncthreads();
        if (tid == 0) carry = min(carry + buf[255], max_chunks);
        __syncthreads();
    }
}

// One token of N sequences.  A workgroup takes COLB columns of one (n, head):
// its state slice is read, decayed, written and dotted with C in one pass
// (memory bound: 8 bytes a state value).
template <typename T, int K, int COLB>
__global__ __launch_bounds__(256) void kda_ssm_step_kernel(int H, int G, int P, int softplus, const T* x,
                                                           size_t x_stride, const T* dt, size_t dt_stride, const float* A, const T* B,
                                                           size_t b_stride, const T* Cm, size_t c_stride,
                                                           const float* Dskip, const float* dt_bias, float* state,
                                                           T* y) {
    constexpr int CQ = COLB / 4;            // column quads
    constexpr int RG = 256 / CQ;            // row groups
    constexpr int NR = K / RG > 0 ? K / RG : 1;
    __shared__ float4 red[4][CQ];
    const int blocks = P / COLB;
    const int cb = blockIdx.x % blocks, nhh = blockIdx.x / blocks;
    const int n = nhh / H, h = nhh - n * H, grp = h / (H / G);
    const int tid = threadIdx.x, cq = tid % CQ, rg = tid / CQ, lane = tid & 63;
    float* st = state + ((size_t)nhh * K) * P + cb * COLB + 4 * cq;
    float4 s[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) s[i] = *reinterpret_cast<const float4*>(st + (size_t)(rg + RG * i) * P);
    float b[NR], c[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        b[i] = to_f32(B[(size_t)n * b_stride + grp * K + rg + RG * i]);
        c[i] = to_f32(Cm[(size_t)n * c_stride + grp * K + rg + RG * i]);
    }
    const T* xp = x + (size_t)n * x_stride + (size_t)h * P + cb * COLB + 4 * cq;
    float4 xv = make_float4(to_f32(xp[0]), to_f32(xp[1]), to_f32(xp[2]), to_f32(xp[3]));
    const float delta = delta_of(to_f32(dt[(size_t)n * dt_stride + h]) + (dt_bias ? dt_bias[h] : 0.f), softplus);
    const float a = expf(delta * A[h]);
    const float4 xd = make_float4(delta * xv.x, delta * xv.y, delta * xv.z, delta * xv.w);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        s[i].x = fmaf(a, s[i].x, b[i] * xd.x);
        s[i].y = fmaf(a, s[i].y, b[i] * xd.y);
        s[i].z = fmaf(a, s[i].z, b[i] * xd.z);
        s[i].w = fmaf(a, s[i].w, b[i] * xd.w);
        *reinterpret_cast<float4*>(st + (size_t)(rg + RG * i) * P) = s[i];
        acc.x = fmaf(c[i], s[i].x, acc.x);
        acc.y = fmaf(c[i], s[i].y, acc.y);
        acc.z = fmaf(c[i], s[i].z, acc.z);
        acc.w = fmaf(c[i], s[i].w, acc.w);
    }
#pragma unroll
    for (int m = CQ; m < 64; m <<= 1) {
        acc.x += __shfl_xor(acc.x, m);
        acc.y += __shfl_xor(acc.y, m);
        acc.z += __shfl_xor(acc.z, m);
        acc.w += __shfl_xor(acc.w, m);
    }
    if (lane < CQ) red[tid >> 6][cq] = acc;
    __syncthreads();
    if (tid < CQ) {
        const float4 r0 = red[0][tid], r1 = red[1][tid], r2 = red[2][tid], r3 = red[3][tid];
        const float d = Dskip ? Dskip[h] : 0.f;
        float o[4] = {r0.x + r1.x + r2.x + r3.x, r0.y + r1.y + r2.y + r3.y, r0.z + r1.z + r2.z + r3.z,
                      r0.w + r1.w + r2.w + r3.w};
        if (Dskip) {
            o[0] = fmaf(d, xv.x, o[0]);
            o[1] = fmaf(d, xv.y, o[1]);
            o[2] = fmaf(d, xv.z, o[2]);
            o[3] = fmaf(d, xv.w, o[3]);
        }
        T* yp = y + (size_t)nhh * P + cb * COLB + 4 * tid;
#pragma unroll
        for (int i = 0; i < 4; ++i) yp[i] = from_f32<T>(o[i]);
    }
}

template <typename T, int K, int COLB>
hipError_t step_launch(int N, int H, int G, int P, int softplus, const void* x, size_t xs, const void* dt,
                       size_t ds, const float* A, const void* B, size_t bs, const void* Cm, size_t cs, const float* D,
                       const float* bias, float* state, void* y, hipStream_t st) {
    const long long blocks = (long long)N * H * (P / COLB);
    hipLaunchKernelGGL((kda_ssm_step_kernel<T, K, COLB>), dim3((unsigned)blocks), dim3(256), 0, st, H, G, P, softplus,
                       reinterpret_cast<const T*>(x), xs, reinterpret_cast<const T*>(dt), ds, A,
                       reinterpret_cast<const T*>(B), bs, reinterpret_cast<const T*>(Cm), cs, D, bias, state,
                       reinterpret_cast<T*>(y));
    return hipGetLastError();
}

template <typename T, int K, int P, int NT>
hipError_t chunks_launch(bool out, const SsmParams& p, int segs, hipStream_t st) {
    const dim3 grid((unsigned)((long long)segs * (p.H / (64 * NT / P))));
    if (out) hipLaunchKernelGGL((kda_ssm_chunk_kernel<T, K, P, NT, true>), grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL((kda_ssm_chunk_kernel<T, K, P, NT, false>), grid, dim3(256), 0, st, p);
    return hipGetLastError();
}
template <typename T, int K>
hipError_t chunks_pick(bool out, int nt, const SsmParams& p, int segs, hipStream_t st) {
    if (p.P == 128) return chunks_launch<T, K, 128, 2>(out, p, segs, st);
    return nt == 2 ? chunks_launch<T, K, 64, 2>(out, p, segs, st) : chunks_launch<T, K, 64, 1>(out, p, segs, st);
}

}  // namespace

hipError_t launch_ssm_prep(const SeqView& sv, int* chunk_off, int max_chunks, hipStream_t st) {
    hipLaunchKernelGGL(kda_ssm_prep_kernel, dim3(1), dim3(256), 0, st, sv, chunk_off, max_chunks);
    return hipGetLastError();
}

hipError_t launch_ssm_chunks(int dtype, bool out, int nt, const SsmParams& p, int segs, hipStream_t st) {
    if (segs <= 0) return hipSuccess;
    if (dtype == 1) return p.K == 128 ? chunks_pick<bf16, 128>(out, nt, p, segs, st) : chunks_pick<bf16, 64>(out, nt, p, segs, st);
    return p.K == 128 ? chunks_pick<float, 128>(out, nt, p, segs, st) : chunks_pick<float, 64>(out, nt, p, segs, st);
}

hipError_t launch_ssm_combine(const SsmParams& p, float* d_s0, hipStream_t st) {
    const size_t n = (size_t)p.H * p.K * p.P / 4;
    hipLaunchKernelGGL(kda_ssm_combine_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, p, d_s0);
    return hipGetLastError();
}

hipError_t launch_ssm_step(int dtype, int N, int H, int G, int K, int P, int softplus, const void* x, size_t xs,
                           const void* dt, size_t ds, const float* A, const void* B, size_t bs, const void* Cm, size_t cs,
                           const float* D, const float* bias, float* state, void* y, hipStream_t st) {
#define KDA_STEP(T, KK) step_launch<T, KK, 64>(N, H, G, P, softplus, x, xs, dt, ds, A, B, bs, Cm, cs, D, bias, state, y, st)
    if (dtype == 1) return K == 128 ? KDA_STEP(bf16, 128) : KDA_STEP(bf16, 64);
    return K == 128 ? KDA_STEP(float, 128) : KDA_STEP(float, 64);
#undef KDA_STEP
}

}  // namespace kda
