// Short causal depthwise convolution over the token axis (width W = 2, 3, 4),
// with bias and SiLU: forward, backward and the one-token step.
//
//   c_t = bias + sum_w weight[:, w] x_{t-W+1+w},   y_t = act(c_t)
//
// Memory bound: 2 W + 6 flops a value against 4 bytes moved (bf16).  A thread
// owns 16 bytes of channels and a tile of consecutive tokens, the last W - 1
// rows in registers, so every row is read once and W - 1 halo rows more per
// tile; four rows are loaded while the four before them are worked on.  No LDS:
// neighbouring tokens of a channel meet in one thread.
// Forward, 8192 x 12288 bf16 (403 MB): 87 us, 4.6 TB/s.
#include "kda_mixer.h"
#include "kda_mixer_device.h"

#include <type_traits>

namespace kda {

namespace {

constexpr int kRowsAhead = 4;    // token rows loaded together, one group ahead

// The runs of one sequence each that make up a tile [a, b) of token rows.
// Offsets are clamped to [0, T], so that any cu keeps every access in bounds;
// rows behind the last sequence belong to no run.
struct Runs {
    SeqView sv;
    int seq, a, b;
    int s0, s1;     // the current run's sequence
    int end;        // the current run: [a, end)

    __device__ __forceinline__ void init_regular(const SeqView& v, int tile, int tiles_per_seq, int tt) {
        sv = v;
        seq = tile / tiles_per_seq;
        s0 = 0;
        s1 = v.T;
        a = (tile - seq * tiles_per_seq) * tt;
        b = end = min(a + tt, v.T);
    }
    __device__ __forceinline__ void init_packed(const SeqView& v, int tile, int tt) {
        sv = v;
        a = tile * tt;
        b = min(a + tt, v.T);
        // the last sequence that starts at or before a
        int lo = 0, hi = v.N;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (v.cu[mid] <= a)
                lo = mid;
            else
                hi = mid;
        }
        seq = lo;
        s1 = a;
        end = a;
    }
    // the next run; false when the tile is done.  Packed only.
    __device__ __forceinline__ bool next() {
        a = end;
        for (; a < b && seq < sv.N; ++seq) {
            s0 = max(sv.cu[seq], 0);
            s1 = min(sv.cu[seq + 1], sv.T);
            if (s1 > a && s0 <= a) {
                end = min(b, s1);
                return true;
            }
        }
        return false;
    }
};

__device__ __forceinline__ void seq_bounds(const SeqView& sv, int i, int& s0, int& len) {
    if (sv.cu) {
        s0 = max(sv.cu[i], 0);
        len = max(min(sv.cu[i + 1], sv.T) - s0, 0);
    } else {
        s0 = 0;
        len = sv.T;
    }
}

// first row of the token axis that a run's row indices are relative to
__device__ __forceinline__ size_t base_row(const SeqView& sv, int seq) {
    return sv.cu ? 0 : (size_t)seq * sv.T;
}

template <typename T, int V, int W>
__device__ __forceinline__ void load_params(const ConvParams& p, int c, float (&wt)[W][V], float (&bs)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int w = 0; w < W; ++w) wt[w][i] = p.weight[(size_t)(c + i) * W + w];
        bs[i] = p.bias ? p.bias[c + i] : 0.f;
    }
}

// the W - 1 rows before row a of a sequence that starts at s0
template <typename T, int V, int W>
__device__ __forceinline__ void load_halo(const ConvParams& p, const T* x, int seq, int s0, int a, int c,
                                          Vec<T, V> (&win)[W - 1]) {
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        const int t = a - (W - 1) + r;
        if (t >= s0)
            win[r].load(x + (size_t)t * p.x_stride + c);
        else if (p.s0)
            win[r].load(reinterpret_cast<const T*>(p.s0) + ((size_t)seq * (W - 1) + (t - s0 + W - 1)) * p.D + c);
        else
            win[r].zero();
    }
}

// Sequences without tokens: their state passes through.  Threads over
// (sequence, channels), `step` sequences apart.
template <typename T, int V>
__device__ __forceinline__ void pass_empty(const SeqView& sv, int W, int D, const void* from, void* to, int first,
                                           int step, int c) {
    for (int i = first; i < sv.N; i += step) {
        int s0, len;
        seq_bounds(sv, i, s0, len);
        if (len > 0) continue;
        for (int r = 0; r < W - 1; ++r) {
            const size_t at = ((size_t)i * (W - 1) + r) * D + c;
            Vec<T, V> v;
            if (from)
                v.load(reinterpret_cast<const T*>(from) + at);
            else
                v.zero();
            v.store(reinterpret_cast<T*>(to) + at);
        }
    }
}

template <typename T, int V, int W>
__global__ __launch_bounds__(256) void kda_conv_fwd_kernel(ConvParams p) {
    const int cx = 1 << p.cx_log2;
    const int c = (blockIdx.y * cx + (threadIdx.x & (cx - 1))) * V;
    const int ty = threadIdx.x >> p.cx_log2, tys = 256 >> p.cx_log2;
    if (c >= p.D) return;
    const int tile_blocks = (p.tiles + tys - 1) / tys;
    if ((int)blockIdx.x >= tile_blocks) {
        pass_empty<T, V>(p.sv, W, p.D, p.s0, p.sT, ((int)blockIdx.x - tile_blocks) * tys + ty,
                         ((int)gridDim.x - tile_blocks) * tys, c);
        return;
    }
    const int tile = blockIdx.x * tys + ty;
    if (tile >= p.tiles) return;
    float wt[W][V], bs[V];
    load_params<T, V, W>(p, c, wt, bs);
    Runs run;
    const bool packed = p.sv.cu != nullptr;
    if (packed) {
        run.init_packed(p.sv, tile, p.tile_tokens);
        if (!run.next()) return;
    } else {
        run.init_regular(p.sv, tile, p.tiles_per_seq, p.tile_tokens);
    }
    for (;;) {
        const size_t base = base_row(p.sv, run.seq);
        const T* x = reinterpret_cast<const T*>(p.x) + base * p.x_stride;
        T* y = reinterpret_cast<T*>(p.y) + base * p.D;
        Vec<T, V> win[W - 1];
        load_halo<T, V, W>(p, x, run.seq, run.s0, run.a, c, win);
        auto row_out = [&](int at, const Vec<T, V>& row) {
            Vec<T, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float acc = fmaf(wt[W - 1][i], row.f(i), bs[i]);
#pragma unroll
                for (int w = 0; w < W - 1; ++w) acc = fmaf(wt[w][i], win[w].f(i), acc);
                o.set(i, act_of<T>(acc, p.act));
            }
            o.store(y + (size_t)at * p.D + c);
#pragma unroll
            for (int w = 0; w + 1 < W - 1; ++w) win[w] = win[w + 1];
            win[W - 2] = row;
        };
        auto fetch = [&](int at, Vec<T, V>(&rows)[kRowsAhead]) {
#pragma unroll
            for (int u = 0; u < kRowsAhead; ++u) rows[u].load(x + (size_t)(at + u) * p.x_stride + c);
        };
        int t = run.a;
        Vec<T, V> now[kRowsAhead], next[kRowsAhead];
        if (t + kRowsAhead <= run.end) fetch(t, next);
        while (t + kRowsAhead <= run.end) {
#pragma unroll
            for (int u = 0; u < kRowsAhead; ++u) now[u] = next[u];
            if (t + 2 * kRowsAhead <= run.end) fetch(t + kRowsAhead, next);
#pragma unroll
            for (int u = 0; u < kRowsAhead; ++u) row_out(t + u, now[u]);
            t += kRowsAhead;
        }
        for (; t < run.end; ++t) {
            Vec<T, V> row;
            row.load(x + (size_t)t * p.x_stride + c);
            row_out(t, row);
        }
        if (p.sT && run.end == run.s1) {
#pragma unroll
            for (int r = 0; r < W - 1; ++r)
                win[r].store(reinterpret_cast<T*>(p.sT) + ((size_t)run.seq * (W - 1) + r) * p.D + c);
        }
        if (!packed) return;
        ++run.seq;
        if (!run.next()) return;
    }
}

// Backward.  With q_t = d_y_t act'(c_t) (c recomputed from x):
//   dx_t        = sum_j weight[:, W-1-j] q_{t+j}  (+ d_final of row t)
//   dweight[w]  = sum_t q_t x_{t-W+1+w},   dbias = sum_t q_t
// A tile computes q for its rows and the W - 1 rows behind it (of the same
// sequence).  The parameter sums stay in registers over a thread's tiles, are
// added across the block's tile rows in LDS (fixed order) and leave as one
// partial row per block, summed by kda_sum_rows_kernel.
// About 35 vector operations a value, the activation's exponential and
// reciprocal at a quarter of the rate, against 6 bytes (bf16): loads and
// arithmetic both count.  18K packed tokens x 2304 bf16 (249 MB): 69 us,
// 3.6 TB/s, and 5 us for the row sums.  Eight bytes a thread: of 16, the weights
// and sums alone would be 80 registers.  Four rows at a time: with eight, or
// with a tile's edge rows loaded together, the kernel spills (115, 100 us).
template <typename T, int V, int W>
__global__ __launch_bounds__(256, 3) void kda_conv_bwd_kernel(ConvParams p) {
    const int cx = 1 << p.cx_log2;
    const int lane_c = threadIdx.x & (cx - 1);
    const int c = (blockIdx.y * cx + lane_c) * V;
    const int ty = threadIdx.x >> p.cx_log2, tys = 256 >> p.cx_log2;
    const bool live = c < p.D;
    float dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) dw[w][i] = 0.f;
    }
    const bool packed = p.sv.cu != nullptr;
    const int slots = gridDim.x * tys;
    float wt[W][V], bs[V];
    if (live) load_params<T, V, W>(p, c, wt, bs);
    if (live && p.d_s0) pass_empty<T, V>(p.sv, W, p.D, p.d_sT, p.d_s0, blockIdx.x * tys + ty, slots, c);
    for (int tile = blockIdx.x * tys + ty; live && tile < p.tiles; tile += slots) {
        Runs run;
        bool more = true;
        if (packed) {
            run.init_packed(p.sv, tile, p.tile_tokens);
            more = run.next();
        } else {
            run.init_regular(p.sv, tile, p.tiles_per_seq, p.tile_tokens);
        }
        while (more) {
            const size_t base = base_row(p.sv, run.seq);
            const T* x = reinterpret_cast<const T*>(p.x) + base * p.x_stride;
            const T* dy = reinterpret_cast<const T*>(p.d_y) + base * p.D;
            T* dx = reinterpret_cast<T*>(p.dx) + base * p.D;
            const T* dsT = p.d_sT ? reinterpret_cast<const T*>(p.d_sT) + (size_t)run.seq * (W - 1) * p.D : nullptr;
            Vec<T, V> win[W - 1];
            load_halo<T, V, W>(p, x, run.seq, run.s0, run.a, c, win);
            // q of rows s - W + 1 .. s - 1 as row s is reached; rows before
            // the run's first count for the state's gradient only where the
            // run opens the sequence, and are zero there
            float q[W][V];
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) q[j][i] = 0.f;
            const bool opens = run.a == run.s0;
            // One row: q of row s (0 behind the sequence), its share of the
            // parameter sums if it is the run's, and the gradient of row
            // s - W + 1.  MAIN: row s and that row are both the run's, and that
            // row is no row of the final state (it is W - 1 before a row that
            // exists), so nothing needs asking.
            auto step = [&](auto main, int s, const Vec<T, V>& xr, const Vec<T, V>& gr) {
                constexpr bool MAIN = decltype(main)::value;
#pragma unroll
                for (int j = 0; j + 1 < W; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) q[j][i] = q[j + 1][i];
                if (MAIN || s < run.s1) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float acc = fmaf(wt[W - 1][i], xr.f(i), bs[i]);
#pragma unroll
                        for (int w = 0; w < W - 1; ++w) acc = fmaf(wt[w][i], win[w].f(i), acc);
                        const float g = gr.f(i) * dact_of<T>(acc, p.act);
                        q[W - 1][i] = g;
                        if (MAIN || s < run.end) {
                            db[i] += g;
#pragma unroll
                            for (int w = 0; w < W - 1; ++w) dw[w][i] = fmaf(g, win[w].f(i), dw[w][i]);
                            dw[W - 1][i] = fmaf(g, xr.f(i), dw[W - 1][i]);
                        }
                    }
#pragma unroll
                    for (int w = 0; w + 1 < W - 1; ++w) win[w] = win[w + 1];
                    win[W - 2] = xr;
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) q[W - 1][i] = 0.f;
                }
                const int t = s - (W - 1);
                const bool in_run = MAIN || (t >= run.a && t < run.end);
                if (!in_run && !(t < run.s0 && opens && p.d_s0)) return;
                Vec<T, V> f, o;
                if constexpr (!MAIN) {
                    const int fin = t - (run.s1 - (W - 1));      // row of the final state
                    if (dsT && fin >= 0)
                        f.load(dsT + (size_t)fin * p.D + c);
                    else
                        f.zero();
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float g = MAIN ? 0.f : f.f(i);
#pragma unroll
                    for (int j = 0; j < W; ++j) g = fmaf(wt[W - 1 - j][i], q[j][i], g);
                    o.set(i, g);
                }
                if (in_run)
                    o.store(dx + (size_t)t * p.D + c);
                else
                    o.store(reinterpret_cast<T*>(p.d_s0) + ((size_t)run.seq * (W - 1) + (t - run.s0 + W - 1)) * p.D + c);
            };
            auto edge = [&](int s) {
                Vec<T, V> xr, gr;
                if (s < run.s1) {
                    xr.load(x + (size_t)s * p.x_stride + c);
                    gr.load(dy + (size_t)s * p.D + c);
                }
                step(std::false_type{}, s, xr, gr);
            };
            auto fetch = [&](int at, Vec<T, V>(&xs)[kRowsAhead], Vec<T, V>(&gs)[kRowsAhead]) {
#pragma unroll
                for (int u = 0; u < kRowsAhead; ++u) {
                    xs[u].load(x + (size_t)(at + u) * p.x_stride + c);
                    gs[u].load(dy + (size_t)(at + u) * p.D + c);
                }
            };
            int s = run.a;
            for (; s < run.a + W - 1; ++s) edge(s);
            Vec<T, V> xn[kRowsAhead], gn[kRowsAhead], xs[kRowsAhead], gs[kRowsAhead];
            if (s + kRowsAhead <= run.end) fetch(s, xn, gn);
            while (s + kRowsAhead <= run.end) {
#pragma unroll
                for (int u = 0; u < kRowsAhead; ++u) {
                    xs[u] = xn[u];
                    gs[u] = gn[u];
                }
                if (s + 2 * kRowsAhead <= run.end) fetch(s + kRowsAhead, xn, gn);
#pragma unroll
                for (int u = 0; u < kRowsAhead; ++u) step(std::true_type{}, s + u, xs[u], gs[u]);
                s += kRowsAhead;
            }
            for (; s < run.end + W - 1; ++s) edge(s);
            more = false;
            if (packed) {
                ++run.seq;
                more = run.next();
            }
        }
    }
    // block sums over the tile rows, one value at a time through LDS
    __shared__ float red[256 * V];
    for (int m = 0; m <= W; ++m) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float v = db[i];
#pragma unroll
            for (int w = 0; w < W; ++w) v = m == w ? dw[w][i] : v;
            red[threadIdx.x * V + i] = v;
        }
        __syncthreads();
        // threads over the block's cx * V channels
        for (int k = threadIdx.x; k < cx * V; k += 256) {
            const int d = blockIdx.y * cx * V + k;
            if (d >= p.D) continue;
            float sum = 0.f;
            for (int r = 0; r < tys; ++r) sum += red[r * cx * V + k];
            p.part[((size_t)blockIdx.x * (W + 1) + m) * p.D + d] = sum;
        }
    }
}

// part [rows][M][D] summed over the rows in a fixed order: 32 columns x 8 row
// groups a block, the groups joined in LDS.
__global__ __launch_bounds__(256) void kda_sum_rows_kernel(const float* part, int rows, int M, int D, float* out0,
                                                           int M0, float* out1) {
    __shared__ float red[8][33];
    const int col = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int d = blockIdx.x * 32 + col, m = blockIdx.y;
    float s = 0.f;
    if (d < D) {
        const float* p = part + (size_t)m * D + d;
        const size_t step = (size_t)M * D;
#pragma unroll 8
        for (int r = grp; r < rows; r += 8) s += p[r * step];
    }
    red[grp][col] = s;
    __syncthreads();
    if (grp == 0 && d < D) {
        for (int k = 1; k < 8; ++k) s += red[k][col];
        if (m < M0) {
            if (out0) out0[(size_t)d * M0 + m] = s;
        } else if (out1) {
            out1[d] = s;
        }
    }
}

// One token a sequence: the state's rows move up in place.  256 x 2304 bf16
// (9.5 MB): 7.8 us, one round trip to memory and the launch.
template <typename T, int V, int W>
__global__ __launch_bounds__(256) void kda_conv_step_kernel(int N, int D, int act, const T* x, size_t x_stride,
                                                            const float* weight, const float* bias, T* state, T* y) {
    const int per = D / V;
    const long long at = (long long)blockIdx.x * 256 + threadIdx.x;
    if (at >= (long long)N * per) return;
    const int n = (int)(at / per), c = (int)(at - (long long)n * per) * V;
    T* st = state + (size_t)n * (W - 1) * D + c;
    Vec<T, V> win[W], o;
#pragma unroll
    for (int r = 0; r < W - 1; ++r) win[r].load(st + (size_t)r * D);
    win[W - 1].load(x + (size_t)n * x_stride + c);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float acc = bias ? bias[c + i] : 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) acc = fmaf(weight[(size_t)(c + i) * W + w], win[w].f(i), acc);
        o.set(i, act_of<T>(acc, act));
    }
    o.store(y + (size_t)n * D + c);
#pragma unroll
    for (int r = 0; r < W - 1; ++r) win[r + 1].store(st + (size_t)r * D);
}

template <typename T, int V>
hipError_t conv_fwd_v(const ConvParams& p, dim3 grid, hipStream_t st) {
    if (p.W == 2) hipLaunchKernelGGL((kda_conv_fwd_kernel<T, V, 2>), grid, dim3(256), 0, st, p);
    else if (p.W == 3) hipLaunchKernelGGL((kda_conv_fwd_kernel<T, V, 3>), grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL((kda_conv_fwd_kernel<T, V, 4>), grid, dim3(256), 0, st, p);
    return hipGetLastError();
}
template <typename T, int V>
hipError_t conv_bwd_v(const ConvParams& p, dim3 grid, hipStream_t st) {
    if (p.W == 2) hipLaunchKernelGGL((kda_conv_bwd_kernel<T, V, 2>), grid, dim3(256), 0, st, p);
    else if (p.W == 3) hipLaunchKernelGGL((kda_conv_bwd_kernel<T, V, 3>), grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL((kda_conv_bwd_kernel<T, V, 4>), grid, dim3(256), 0, st, p);
    return hipGetLastError();
}
template <typename T, int V>
hipError_t conv_step_v(int N, int D, int W, int act, const void* x, size_t xs, const float* w, const float* b, void* s,
                       void* y, hipStream_t st) {
    const long long n = (long long)N * (D / V);
    const dim3 grid((unsigned)((n + 255) / 256));
    const T* xp = reinterpret_cast<const T*>(x);
    T *sp = reinterpret_cast<T*>(s), *yp = reinterpret_cast<T*>(y);
    if (W == 2) hipLaunchKernelGGL((kda_conv_step_kernel<T, V, 2>), grid, dim3(256), 0, st, N, D, act, xp, xs, w, b, sp, yp);
    else if (W == 3) hipLaunchKernelGGL((kda_conv_step_kernel<T, V, 3>), grid, dim3(256), 0, st, N, D, act, xp, xs, w, b, sp, yp);
    else hipLaunchKernelGGL((kda_conv_step_kernel<T, V, 4>), grid, dim3(256), 0, st, N, D, act, xp, xs, w, b, sp, yp);
    return hipGetLastError();
}

unsigned channel_blocks(const ConvParams& p, int V) {
    const int per = V << p.cx_log2;
    return (unsigned)((p.D + per - 1) / per);
}

}  // namespace

hipError_t launch_conv_fwd(int dtype, bool vec, const ConvParams& p, int tile_blocks, hipStream_t st) {
    const int V = vec ? (dtype == 1 ? 8 : 4) : 1;
    const dim3 grid((unsigned)tile_blocks, channel_blocks(p, V));
    if (dtype == 1) return vec ? conv_fwd_v<bf16, 8>(p, grid, st) : conv_fwd_v<bf16, 1>(p, grid, st);
    return vec ? conv_fwd_v<float, 4>(p, grid, st) : conv_fwd_v<float, 1>(p, grid, st);
}

hipError_t launch_conv_bwd(int dtype, bool vec, const ConvParams& p, int tile_blocks, hipStream_t st) {
    const int V = vec ? (dtype == 1 ? 4 : 2) : 1;
    const dim3 grid((unsigned)tile_blocks, channel_blocks(p, V));
    if (dtype == 1) return vec ? conv_bwd_v<bf16, 4>(p, grid, st) : conv_bwd_v<bf16, 1>(p, grid, st);
    return vec ? conv_bwd_v<float, 2>(p, grid, st) : conv_bwd_v<float, 1>(p, grid, st);
}

hipError_t launch_conv_step(int dtype, bool vec, int N, int D, int W, int act, const void* x, size_t xs,
                            const float* w, const float* b, void* s, void* y, hipStream_t st) {
    if (dtype == 1)
        return vec ? conv_step_v<bf16, 8>(N, D, W, act, x, xs, w, b, s, y, st)
                   : conv_step_v<bf16, 1>(N, D, W, act, x, xs, w, b, s, y, st);
    return vec ? conv_step_v<float, 4>(N, D, W, act, x, xs, w, b, s, y, st)
               : conv_step_v<float, 1>(N, D, W, act, x, xs, w, b, s, y, st);
}

hipError_t launch_sum_rows(const float* part, int rows, int M, int D, float* out0, int M0, float* out1,
                           hipStream_t st) {
    if (D <= 0 || M <= 0) return hipSuccess;
    hipLaunchKernelGGL(kda_sum_rows_kernel, dim3((unsigned)((D + 31) / 32), (unsigned)M), dim3(256), 0, st, part, rows,
                       M, D, out0, M0, out1);
    return hipGetLastError();
}

}  // namespace kda
