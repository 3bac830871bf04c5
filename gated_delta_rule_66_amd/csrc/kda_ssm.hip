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

// The gates of every chunk and head (kda_ssm_device.h): a wave a head, a lane a
// token, eight heads a block, whose step sizes share cache lines.  Memory
// bound: 20 bytes written a token and head (8K x 32 heads 6 us, 8 x 32K x 32
// heads 57 us, 168 MB).
template <typename T>
__global__ __launch_bounds__(256) void kda_ssm_gates_kernel(SsmParams p) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int hb = (p.H + 7) / 8;
    const int chunk = blockIdx.x / hb, first = (blockIdx.x - chunk * hb) * 8;
    if (chunk >= total_chunks(p)) return;
    ChunkWalk at;
    at.init(p, chunk);
    const int t0 = at.t0(), len = at.len();
    for (int h = first + w; h < min(first + 8, p.H); h += 4) {
        float delta = 0.f;
        if (lane < len)
            delta = delta_of(to_f32(reinterpret_cast<const T*>(p.dt)[(size_t)(t0 + lane) * p.dt_stride + h]) +
                                 (p.dt_bias ? p.dt_bias[h] : 0.f),
                             p.softplus);
        const double c = wave_prefix((double)delta * (double)p.A[h] * 1.4426950408889634);
        const float ch = (float)c;
        float* out = p.gates + ((size_t)chunk * p.H + h) * (kGates * C) + lane;
        out[kGateC * C] = ch;
        out[kGateDelta * C] = delta;
        out[kGateNear * C] = exp2_of(row_last(c) - c) * delta;
        out[kGateW * C] = exp2_of(last_lane(c) - c) * delta;
        out[kGateRest * C] = (float)(c - (double)ch);
    }
}

// One workgroup per (segment, COLS columns of x: one or two heads) walks the
// segment's chunks with the state in registers: wave w owns columns
// [16 NT w, 16 NT (w + 1)) of all K state rows, as accumulator tiles that serve
// as operands as they are.  B, C and x of a chunk are staged in LDS (the next
// chunk's loads in flight meanwhile); the scores C B^T are computed once for
// the workgroup's heads, scaled and masked per head, and passed through LDS.
//   output:  y, and the final state where a sequence ends
//   summary: each segment's local state and decay
//   states:  the state before each chunk, and the final state
// blockIdx.y picks one of two recurrences (the backward runs the states and,
// with C for B, dy for x and the chunks in reverse, their adjoints).
// Final states over the initial ones: a sequence that came in from the segment
// before may have its initial state still read there, so its final state goes to
// this segment's slot (whose start state is in registers), and from there on by
// kda_ssm_final_kernel.  A segment has one such sequence at most.
//
// The state is exact to fp32: delta x e^{..} is split into three bf16 for its
// product with B, half of the output pass's and all of the summary's matrix
// work.  bf16 tokens: y, which is rounded to bf16, takes the scaled scores (sG,
// sGL) and the start state as two bf16 each, exact to 2^-16, and so is off by its
// own rounding alone, 0.0017 of its root mean square.  One bf16 each would make
// it 0.0019, and the output pass 42 us instead of 48 on 8K x 32 heads, 1045
// instead of 1180 on 8 x 32K x 32 heads.
// Everything else is fp32, the decays' exponents two floats (kGateC, kGateRest).
// fp32 tokens: fp32 products throughout.
// What bounds it: nothing alone.  By count, a chunk of two heads (K = 128,
// P = 64) takes a CU 3100 cycles of matrix instructions in the output pass, 2900
// of LDS accesses and about 3800 of vector operations; it takes 10500 with two
// workgroups a CU.  The summary: 1500 cycles of matrix instructions and 1600 of
// vector operations out of 5400; without its loads 424 us instead of 485.  Tried
// on 8 x 32K x 32 heads with one bf16 each (1117 us; loads, stores, scores or
// update products left out one at a time saved 12 to 15 %): one workgroup a CU
// 1477 us, and more than two do not fit; eight waves of 16 columns as long as
// four of 32 in all passes (more operands read from LDS); scores kept in
// registers by each wave 1357 us; y stored from registers, 32 bytes a token, 1093
// instead of 1072.  With two bf16: the lower halves by dot products with -1 1367
// us instead of 1328, by matrix products with -I 1320 instead of 1298.
// Measured, K = 128, P = 64: output 8K x 32 heads 48 us, 8 x 32K x 32 heads
// 1180 us (1.42 GB read, 1.08 GB written); summary 22 and 445 us; 2 x 8K x 16
// heads of 128: output 80, summary 36 us.
template <typename T, int K, int P, int COLS, SsmPass PASS>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void kda_ssm_chunk_kernel(SsmPair a) {
    constexpr bool OUT = PASS == kSsmOutput, summary = PASS == kSsmSummary;
    const SsmParams& p = a.p[PASS == kSsmOutput ? 0 : blockIdx.y];
    constexpr int TH = 256, NW = TH / 64;
    constexpr int NT = COLS / 16 / NW;          // column tiles a wave
    constexpr int NH = COLS / P;                // heads of the workgroup
    constexpr int PAD = 16 / sizeof(T);
    // scores: the six lower slabs of 16 rows x 32 tokens, each a fragment in the
    // order of its lanes (rows of 64 bytes instead: four lanes a bank, 49 us
    // instead of 47 on 8K x 32 heads)
    constexpr int SLAB = 512, NG = NH * 6 * SLAB;
    constexpr int LDB = K + tr_pad<T>(K), LDX = COLS + tr_pad<T>(COLS), LDK = K + PAD;
    constexpr int NTK = K / 16;                 // state row tiles
    constexpr int EPP = 16 / sizeof(T);         // elements of a 16-byte piece
    constexpr int PK = C * K / EPP / TH, PX = C * COLS / EPP / TH;
    constexpr int KP = K * P;
    __shared__ T sB[C * LDB];
    __shared__ T sX[C * LDX];
    __shared__ T sC[OUT ? C * LDK : 1];
    __shared__ T sG[OUT ? NG : 1], sGL[OUT && sizeof(T) == 2 ? NG : 1];     // upper and lower halves
    __shared__ __align__(16) float s_gate[NH][kGates][C];
    typedef typename FragOf<T>::type Frag;

    // the wave's index as a scalar: resources and addresses built on it stay scalar
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, r16 = lane & 15;
    const int units = p.H / NH;
    const int flat = xcd_swizzle(blockIdx.x, gridDim.x);
    const int seg = p.seg0 + flat / units, h0 = (flat % units) * NH;
    const int col0 = w * 16 * NT;
    const int hl = col0 / P, pc = col0 % P, h = h0 + hl;
    const int grp = h0 / (p.H / p.G);
    const int all = total_chunks(p);
    const int begin = min(seg * p.cps, all), end = min(begin + p.cps, all);
    const bool rev = !OUT && p.reverse;
    const int own = (4 * g) * P + pc + r16;     // the lane's first state element
    float* seg_slot = p.seg_state ? p.seg_state + ((size_t)seg * p.H + h) * KP : nullptr;

    f32x4 S[NTK][NT];
#pragma unroll
    for (int m = 0; m < NTK; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) S[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    // states go by one lane offset and scalar offsets: per-element addresses
    // would be kept in registers across the chunk loop
    auto load_state = [&](const float* src) {   // src: [K][P] of head h, or null
        if (src) {
            const auto r = make_rsrc_n(src, KP * sizeof(float));
#pragma unroll
            for (int m = 0; m < NTK; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        S[m][n][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                            r, own * 4, ((16 * m + e) * P + 16 * n) * 4, 0));
            // waited for here: a wait where S is next used would also stand on
            // the way without these loads, and hold up the chunk loads there
#pragma unroll
            for (int m = 0; m < NTK; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) asm volatile("" : "+v"(S[m][n]));
        } else {
#pragma unroll
            for (int m = 0; m < NTK; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) S[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    };
    auto store_state = [&](float* dst) {
        const auto r = make_rsrc_n(dst, KP * sizeof(float));
#pragma unroll
        for (int m = 0; m < NTK; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[m][n][e]), r, own * 4,
                                                          ((16 * m + e) * P + 16 * n) * 4, 0);
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
        for (int k = tid; k < NG; k += TH) {
            sG[k] = (T)0.f;
            if constexpr (sizeof(T) == 2) sGL[k] = (T)0.f;
        }
    }

    walk.init(p, rev ? end - 1 : begin);
    const T* xbase = reinterpret_cast<const T*>(p.x) + h0 * P;
    const T* bbase = reinterpret_cast<const T*>(p.B) + grp * K;
    const T* cbase = reinterpret_cast<const T*>(p.C) + grp * K;
    const bool skips = OUT && p.Dskip;
    const float dskip = skips ? p.Dskip[h] : 0.f;
    uint4 rb[PK], rx[PX], rc[OUT ? PK : 1];
    uint4 rg;
    constexpr int PG = NH * kGates * C / 4;     // 16-byte pieces of a chunk's gates
    auto fetch = [&](const ChunkWalk& at, int chunk) {
        const int t0 = at.t0(), len = at.len();
        const auto xr = row_rsrc<T>(xbase, p.x_stride, t0, len, COLS);
        const auto br = row_rsrc<T>(bbase, p.b_stride, t0, len, K);
        const int td = opaque(tid);
#pragma unroll
        for (int i = 0; i < PK; ++i) {
            const int q = td + TH * i, row = q / (K / EPP), col = (q % (K / EPP)) * EPP;
            rb[i] = buf_load16(br, (unsigned)(row * (int)p.b_stride + col) * sizeof(T));
        }
        if constexpr (OUT) {
            const auto cr = row_rsrc<T>(cbase, p.c_stride, t0, len, K);
#pragma unroll
            for (int i = 0; i < PK; ++i) {
                const int q = td + TH * i, row = q / (K / EPP), col = (q % (K / EPP)) * EPP;
                rc[i] = buf_load16(cr, (unsigned)(row * (int)p.c_stride + col) * sizeof(T));
            }
        }
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            const int q = td + TH * i, row = q / (COLS / EPP), col = (q % (COLS / EPP)) * EPP;
            rx[i] = buf_load16(xr, (unsigned)(row * (int)p.x_stride + col) * sizeof(T));
        }
        // the heads' gates lie together; threads behind them read zeros
        const auto gr = make_rsrc_n(p.gates + ((size_t)chunk * p.H + h0) * (kGates * C), PG * 16);
        rg = buf_load16(gr, 16u * (unsigned)td);
    };
    auto stage = [&]() {
        const int td = opaque(tid);
#pragma unroll
        for (int i = 0; i < PK; ++i) {
            const int q = td + TH * i, row = q / (K / EPP), col = (q % (K / EPP)) * EPP;
            *reinterpret_cast<uint4*>(sB + row * LDB + col) = rb[i];
            if constexpr (OUT) st_slots(sC + row * LDK, col, rc[i]);
        }
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            const int q = td + TH * i, row = q / (COLS / EPP), col = (q % (COLS / EPP)) * EPP;
            *reinterpret_cast<uint4*>(sX + row * LDX + col) = rx[i];
        }
        if (td < PG) *reinterpret_cast<uint4*>(&s_gate[0][0][0] + 4 * td) = rg;
    };
    auto store_y = [&](int t0, int len) {
        const int td = opaque(tid);
        const auto yr = row_rsrc<T>(reinterpret_cast<const T*>(p.y) + h0 * P, (size_t)p.H * P, t0, len, COLS);
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            const int q = td + TH * i, row = q / (COLS / EPP), col = (q % (COLS / EPP)) * EPP;
            buf_store16(yr, (unsigned)(row * p.H * P + col) * sizeof(T), 0,
                        *reinterpret_cast<const uint4*>(sX + row * LDX + col));
        }
    };
    fetch(walk, rev ? end - 1 : begin);
    float seg_dec = 1.f;
    int y_t0 = 0, y_len = 0;
    bool came_in = OUT && p.in_place;       // the sequence opened in a segment before

    for (int it = begin; it < end; ++it) {
        const int t0 = walk.t0(), len = walk.len(), seq = walk.seq;
        const bool opens = rev ? walk.last() : walk.first();
        const bool closes = rev ? walk.first() : walk.last();
        if (opens) {
            load_state(p.s0 ? p.s0 + ((size_t)seq * p.H + h) * KP : nullptr);
            seg_dec = -1.f;
            came_in = false;
        }
        // y of the chunk before leaves from the pieces that stage() writes next
        if (OUT && it > begin) store_y(y_t0, y_len);
        y_t0 = t0;
        y_len = len;
        stage();
        if (PASS == kSsmStates)
            store_state(p.states + ((size_t)(rev ? begin + end - 1 - it : it) * p.H + h) * KP);
        __syncthreads();
        // the next chunk's loads run behind this chunk's products
        if (it + 1 < end) {
            if (rev)
                walk.prev();
            else
                walk.next();
            fetch(walk, rev ? begin + end - 2 - it : it + 1);
        }
        f32x4 Y[OUT ? 4 : 1][NT];
        if constexpr (OUT) {
            // LDS addresses are worked out again in each phase (opaque): kept in
            // registers across the loop they spill
            const int ln = opaque(lane), g = ln >> 4, r16 = ln & 15;
            // ---- scores, transposed: a lane gets four tokens j of one row i.
            // On the diagonal each pair takes its own decay; below it the decay is
            // the product of j's to the end of its tile and i's from there on,
            // both at most 1, so one exponential a lane does.
            auto b_frag = [&](int tj, int m) { return ld_frag_perm<T>(sB + (16 * tj + r16) * LDB + 32 * m + 4 * g); };
            auto c_frag = [&](int ti, int m) { return ld_frag<T>(sC + (16 * ti + r16) * LDK + 32 * m + 8 * g); };
            auto put = [&](int k, int ti, int tj, const float* v) {
                const int o = (k * 6 + ti + (tj & 2)) * SLAB + 8 * ln + 4 * (tj & 1);
                st_near4(sG + o, sGL + o, v);
            };
            auto below = [&](int ti, int tj, f32x4 acc) {
                const int i = 16 * ti + r16, last = 16 * tj + 15;
#pragma unroll
                for (int k = 0; k < NH; ++k) {
                    const float f = fast_exp2((s_gate[k][kGateC][i] - s_gate[k][kGateC][last]) +
                                              (s_gate[k][kGateRest][i] - s_gate[k][kGateRest][last]));
                    const f32x4 dj = *reinterpret_cast<const f32x4*>(&s_gate[k][kGateNear][16 * tj + 4 * g]);
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = acc[e] * dj[e] * f;
                    put(k, ti, tj, v);
                }
            };
            auto diagonal = [&](int t, f32x4 acc) {
                const int i = 16 * t + r16, j0 = 16 * t + 4 * g;
#pragma unroll
                for (int k = 0; k < NH; ++k) {
                    const f32x4 cj = *reinterpret_cast<const f32x4*>(&s_gate[k][kGateC][j0]);
                    const f32x4 rj = *reinterpret_cast<const f32x4*>(&s_gate[k][kGateRest][j0]);
                    const f32x4 dj = *reinterpret_cast<const f32x4*>(&s_gate[k][kGateDelta][j0]);
                    const float ci = s_gate[k][kGateC][i], ri = s_gate[k][kGateRest][i];
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = j0 + e <= i ? acc[e] * fast_exp2((ci - cj[e]) + (ri - rj[e])) * dj[e] : 0.f;
                    put(k, t, t, v);
                }
            };
            // waves 0 to 2 take up to three tiles down from (w, w), which share
            // B's rows; wave 3 takes (3, 3) and (3, 0), which share C's
            f32x4 a0{0.f, 0.f, 0.f, 0.f}, a1 = a0, a2 = a0;
            if (w < 3) {
#pragma unroll
                for (int m = 0; m < K / 32; ++m) {
                    const Frag bf = b_frag(w, m);
                    a0 = mma(a0, bf, c_frag(w, m));
                    a1 = mma(a1, bf, c_frag(w + 1, m));
                    if (w < 2) a2 = mma(a2, bf, c_frag(w + 2, m));
                }
            } else {
#pragma unroll
                for (int m = 0; m < K / 32; ++m) {
                    const Frag cf = c_frag(3, m);
                    a0 = mma(a0, b_frag(3, m), cf);
                    a1 = mma(a1, b_frag(0, m), cf);
                }
            }
            diagonal(w, a0);
            below(w < 3 ? w + 1 : 3, w < 3 ? w : 0, a1);
            if (w < 2) below(w + 2, w, a2);
            {
            const int ln = opaque(lane), g = ln >> 4, r16 = ln & 15;
            // ---- what the start state gives, transposed: a lane holds four
            // columns of one token
#pragma unroll
            for (int m = 0; m < K / 32; ++m) {
                typename Near<T>::type sf[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const f32x4 a = S[2 * m][n], b = S[2 * m + 1][n];
                    const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
                    sf[n] = Near<T>::of(v);
                }
#pragma unroll
                for (int ti = 0; ti < 4; ++ti) {
                    if (m == 0)
#pragma unroll
                        for (int n = 0; n < NT; ++n) Y[ti][n] = f32x4{0.f, 0.f, 0.f, 0.f};
                    mma_near(Y[ti], sf, ld_frag<T>(sC + (16 * ti + r16) * LDK + 32 * m + 8 * g));
                }
            }
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) {
                const float e = exp2_pair(s_gate[hl][kGateC][16 * ti + r16], s_gate[hl][kGateRest][16 * ti + r16]);
#pragma unroll
                for (int n = 0; n < NT; ++n) Y[ti][n] *= e;
            }
            }
            __syncthreads();
        }
        // ---- the chunk's own tokens: outputs and the state update
        const int ln = opaque(lane), g = ln >> 4, r16 = ln & 15;
        const float decay = exp2_pair(s_gate[hl][kGateC][C - 1], s_gate[hl][kGateRest][C - 1]);
        seg_dec = seg_dec < 0.f ? seg_dec : seg_dec * decay;
#pragma unroll
        for (int m = 0; m < NTK; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) S[m][n] *= decay;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            Frag xf[NT];
            typename Exact<T>::type xw[NT];
            f32x4 wa = *reinterpret_cast<const f32x4*>(&s_gate[hl][kGateW][32 * s + 4 * g]);
            f32x4 wb = *reinterpret_cast<const f32x4*>(&s_gate[hl][kGateW][32 * s + 16 + 4 * g]);
            if (rev) {
                // the adjoint's token weights: the decay from the chunk's start
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 32 * s + 4 * g + e;
                    wa[e] = exp2_pair(s_gate[hl][kGateC][j], s_gate[hl][kGateRest][j]);
                    wb[e] = exp2_pair(s_gate[hl][kGateC][j + 16], s_gate[hl][kGateRest][j + 16]);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                xf[n] = ld_frag_tokens(sX, LDX, 32 * s, col0 + 16 * n, ln);
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
                    const int o = (hl * 6 + ti + 2 * s) * SLAB + 8 * ln;
                    if constexpr (sizeof(T) == 2) {
                        const Frag gl = ld_frag<T>(sGL + o);
#pragma unroll
                        for (int n = 0; n < NT; ++n) Y[ti][n] = mma(Y[ti][n], xf[n], gl);
                    }
                    const Frag gf = ld_frag<T>(sG + o);
#pragma unroll
                    for (int n = 0; n < NT; ++n) Y[ti][n] = mma(Y[ti][n], xf[n], gf);
                }
            }
#pragma unroll
            for (int m = 0; m < NTK; m += 2) {
                // independent products between two of one tile
                const Frag b0 = ld_frag_tokens(sB, LDB, 32 * s, 16 * m, ln);
                const Frag b1 = ld_frag_tokens(sB, LDB, 32 * s, 16 * m + 16, ln);
                if constexpr (sizeof(T) == 2) {
#pragma unroll
                    for (int part = 0; part < 3; ++part)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const bf16x8 v = part == 0 ? xw[n].lo : part == 1 ? xw[n].mid : xw[n].hi;
                            S[m][n] = mma(S[m][n], b0, v);
                            S[m + 1][n] = mma(S[m + 1][n], b1, v);
                        }
                } else {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        S[m][n] = mma(S[m][n], b0, xw[n]);
                        S[m + 1][n] = mma(S[m + 1][n], b1, xw[n]);
                    }
                }
            }
        }
        if constexpr (OUT) {
            // y, with D x in fp32 (of a short or fast decaying sequence the
            // largest part), takes the place of x, whose columns only this wave
            // reads
#pragma unroll
            for (int ti = 0; ti < 4; ++ti)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    T* at = sX + (16 * ti + r16) * LDX + col0 + 16 * n + 4 * g;
                    f32x4 v = Y[ti][n];
                    if (skips) v += ld4_as_f32<T>(at) * dskip;
                    float o[4] = {v[0], v[1], v[2], v[3]};
                    st_run<4>(at, o);
                }
        }
        if (closes && p.sT && !summary) store_state(came_in ? seg_slot : p.sT + ((size_t)seq * p.H + h) * KP);
        __syncthreads();
    }
    if constexpr (OUT) store_y(y_t0, y_len);
    if (summary) {
        store_state(seg_slot);
        if (pc == 0 && lane == 0) p.seg_decay[(size_t)seg * p.H + h] = seg_dec;
    }
}

// Segment start states from the segments' local states and decays, written
// over the local states: start_{j+1} = decay_j start_j + local_j (local_j
// alone where a sequence starts in segment j).  A thread owns four state values
// of a head and has 32 segments' loads in flight, so a call of up to 33
// segments waits for memory once (8K x 32 heads, 64 MiB: 12 us; two values a
// thread 14 us, one 31 us).
__global__ __launch_bounds__(256) void kda_ssm_combine_kernel(SsmPair a) {
    const SsmParams& p = a.p[blockIdx.y];
    const unsigned kp = (unsigned)(p.K * p.P);              // a multiple of a block's 1024
    const unsigned h = blockIdx.x / (kp / 1024);
    f32x4* L = reinterpret_cast<f32x4*>(p.seg_state) + (size_t)blockIdx.x * 256 + threadIdx.x;
    const size_t step = (size_t)p.H * kp / 4;
    // segments that hold chunks (a packed call may have fewer than its bound)
    const int all = total_chunks(p), n_seg = min(p.n_seg, (all + p.cps - 1) / p.cps);
    f32x4 s{0.f, 0.f, 0.f, 0.f};
    constexpr int U = 32;
    for (int j = 0; j < n_seg; j += U) {
        f32x4 l[U];
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u < n_seg - 1) {
                const int k = p.reverse ? n_seg - 1 - (j + u) : j + u;
                l[u] = L[(size_t)k * step];
                d[u] = p.seg_decay[(size_t)k * p.H + h];
            }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j + u < n_seg) {
                const int k = p.reverse ? n_seg - 1 - (j + u) : j + u;
                L[(size_t)k * step] = s;
                if (j + u < n_seg - 1) s = d[u] < 0.f ? l[u] : d[u] * s + l[u];
            }
        }
    }
}

// The final states that the output pass of an in-place call left in the slots
// of the segments in which their sequences end.  Four values a thread.
__global__ __launch_bounds__(256) void kda_ssm_final_kernel(SsmParams p) {
    const unsigned blocks = (unsigned)(p.K * p.P) / 1024 * (unsigned)p.H;      // a segment
    const int seg = 1 + (int)(blockIdx.x / blocks), all = total_chunks(p);
    const int begin = min(seg * p.cps, all), end = min(begin + p.cps, all);
    if (begin >= end) return;
    ChunkWalk walk;
    walk.init(p, begin);
    if (walk.first() || begin + (walk.nk - walk.k) > end) return;
    const size_t at = (size_t)(blockIdx.x % blocks) * 256 + threadIdx.x, state = (size_t)blocks * 256;
    reinterpret_cast<f32x4*>(p.sT)[(size_t)walk.seq * state + at] =
        reinterpret_cast<const f32x4*>(p.seg_state)[(size_t)seg * state + at];
}

// The chunk offsets of a packed call: a prefix sum over the sequences' chunks.
// One block: 4 us, which the host cannot take over without the lengths.
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
// (memory bound: 8 bytes a state value).  256 sequences x 32 heads, K = 128,
// P = 64 (539 MB): 77 us, 7.0 TB/s, part of the state from the cache behind the
// L2s; one sequence 3.9 us.
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

template <typename T, int K, int P, int COLS>
hipError_t chunks_launch(SsmPass pass, const SsmPair& a, int n, int segs, hipStream_t st) {
    const dim3 grid((unsigned)((long long)segs * (a.p[0].H / (COLS / P))), (unsigned)n), block(256);
    if (pass == kSsmOutput) hipLaunchKernelGGL((kda_ssm_chunk_kernel<T, K, P, COLS, kSsmOutput>), grid, block, 0, st, a);
    else if (pass == kSsmSummary) hipLaunchKernelGGL((kda_ssm_chunk_kernel<T, K, P, COLS, kSsmSummary>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((kda_ssm_chunk_kernel<T, K, P, COLS, kSsmStates>), grid, block, 0, st, a);
    return hipGetLastError();
}
template <typename T, int K>
hipError_t chunks_pick(SsmPass pass, int cols, const SsmPair& a, int n, int segs, hipStream_t st) {
    if (a.p[0].P == 128) return chunks_launch<T, K, 128, 128>(pass, a, n, segs, st);
    return cols == 128 ? chunks_launch<T, K, 64, 128>(pass, a, n, segs, st) : chunks_launch<T, K, 64, 64>(pass, a, n, segs, st);
}

}  // namespace

hipError_t launch_ssm_prep(const SeqView& sv, int* chunk_off, int max_chunks, hipStream_t st) {
    hipLaunchKernelGGL(kda_ssm_prep_kernel, dim3(1), dim3(256), 0, st, sv, chunk_off, max_chunks);
    return hipGetLastError();
}

size_t ssm_gate_bytes(int chunks, int H) { return (size_t)chunks * H * kGates * C * sizeof(float); }

hipError_t launch_ssm_gates(int dtype, const SsmParams& p, hipStream_t st) {
    const dim3 grid((unsigned)((long long)p.chunks * ((p.H + 7) / 8)));
    if (dtype == 1) hipLaunchKernelGGL(kda_ssm_gates_kernel<bf16>, grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL(kda_ssm_gates_kernel<float>, grid, dim3(256), 0, st, p);
    return hipGetLastError();
}

hipError_t launch_ssm_chunks(int dtype, SsmPass pass, int cols, const SsmPair& a, int n, int segs, hipStream_t st) {
    if (segs <= 0) return hipSuccess;
    if (dtype == 1)
        return a.p[0].K == 128 ? chunks_pick<bf16, 128>(pass, cols, a, n, segs, st) : chunks_pick<bf16, 64>(pass, cols, a, n, segs, st);
    return a.p[0].K == 128 ? chunks_pick<float, 128>(pass, cols, a, n, segs, st) : chunks_pick<float, 64>(pass, cols, a, n, segs, st);
}

hipError_t launch_ssm_combine(const SsmPair& a, int n, hipStream_t st) {
    const size_t values = (size_t)a.p[0].H * a.p[0].K * a.p[0].P;
    hipLaunchKernelGGL(kda_ssm_combine_kernel, dim3((unsigned)(values / 1024), (unsigned)n), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_ssm_final(const SsmParams& p, hipStream_t st) {
    if (p.n_seg < 2) return hipSuccess;
    const unsigned blocks = (unsigned)((size_t)(p.n_seg - 1) * p.H * p.K * p.P / 1024);
    hipLaunchKernelGGL(kda_ssm_final_kernel, dim3(blocks), dim3(256), 0, st, p);
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
