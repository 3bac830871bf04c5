// Group norm over channels-last rows with an activation or a gate, forward
// and backward.  A row is one token; each of its G groups of Cg = C / G
// channels is normalised by itself:
//
//   u = x  (gate_first: x act(z)),   m = mean(u) (center) or 0
//   n = (u - m) rsqrt(mean((u - m)^2) + eps) weight + bias
//   y = n act(z) | n (gate_first) | act(n) (no gate)
//
// Memory bound (about 12 flops a value forward, 30 backward).  A team of lanes
// holds one group of one row in registers, so every value is read once and the
// statistics are two passes over registers, in fp32.  Teams are up to a wave
// (reduced by lane exchanges) or, for wide groups, a whole block (joined in LDS).
// Measured: forward with gate, 8192 rows of 32 x 128 bf16 (201 MB) 36 us, 5.6
// TB/s; backward behind a gate, 16384 rows of 2048 bf16 (336 MB) 79 us, 4.3
// TB/s, and 6 us for the row sums.
#include "kda_mixer.h"
#include "kda_mixer_device.h"

namespace kda {

namespace {

// Sums over a team: lanes of a wave (team <= 64), or the whole block through
// LDS.  Consecutive block sums take the two halves of `red` in turn, so one
// barrier each is enough: a wave that writes a half again has passed the
// barrier of the sum between, before which every wave read the half.
template <bool WAVE> struct Team {
    int team;
    float* red;     // [2][2][16]
    int turn;
    __device__ __forceinline__ void sum2(float& a, float& b, bool both) {
        const int w = WAVE ? team : 64;
        for (int m = w >> 1; m > 0; m >>= 1) {
            a += __shfl_xor(a, m);
            if (both) b += __shfl_xor(b, m);
        }
        if constexpr (!WAVE) {
            const int nw = team >> 6;
            float* r = red + 32 * turn;
            turn ^= 1;
            if ((threadIdx.x & 63) == 0) {
                r[threadIdx.x >> 6] = a;
                if (both) r[16 + (threadIdx.x >> 6)] = b;
            }
            __syncthreads();
            a = b = 0.f;
            for (int k = 0; k < nw; ++k) {
                a += r[k];
                if (both) b += r[16 + k];
            }
        }
    }
    __device__ __forceinline__ float sum(float a) {
        float b = 0.f;
        sum2(a, b, false);
        return a;
    }
};

template <typename T, int V, int R> struct Row {
    Vec<T, V> x[R];
    __device__ __forceinline__ void load(const T* p, int lane, int team, int Cg) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (lane + r * team) * V;
            if (c < Cg)
                x[r].load(p + c);
            else
                x[r].zero();
        }
    }
};

template <int V, int R>
__device__ __forceinline__ void load_channels(const float* p, float none, int lane, int team, int Cg, float (&o)[R][V]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (lane + r * team) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) o[r][i] = none;
        if (p && c < Cg) {
            if constexpr (V % 4 == 0) {
#pragma unroll
                for (int i = 0; i < V; i += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(p + c + i);
                    o[r][i] = v.x; o[r][i + 1] = v.y; o[r][i + 2] = v.z; o[r][i + 3] = v.w;
                }
            } else {
                o[r][0] = p[c];
            }
        }
    }
}

// u and its root mean square: u centred, rstd returned
template <typename T, int V, int R, bool WAVE>
__device__ __forceinline__ float normalise(const NormParams& p, Team<WAVE>& tm, const Row<T, V, R>& x,
                                           const Row<T, V, R>& z, int lane, float inv, float (&u)[R][V]) {
    const bool pre = p.z && p.gate_first;
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            // lanes behind the group's end hold zeros in x
            u[r][i] = x.x[r].f(i);
            if (pre) u[r][i] *= act_of<T>(z.x[r].f(i), p.act);
            sum += u[r][i];
        }
    if (p.center) {
        const float mean = tm.sum(sum) * inv;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = (lane + r * tm.team) * V < p.Cg;
#pragma unroll
            for (int i = 0; i < V; ++i) u[r][i] = in ? u[r][i] - mean : 0.f;
        }
    }
    float sq = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < V; ++i) sq = fmaf(u[r][i], u[r][i], sq);
    return 1.f / sqrtf(tm.sum(sq) * inv + p.eps);
}

// A team keeps to one group (its weights stay in registers) and walks rows,
// the next row's loads in flight behind the current row.  Consecutive teams
// take consecutive groups of a row.
template <typename T, int V, int R, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void kda_norm_fwd_kernel(NormParams p) {
    __shared__ float red[WAVE ? 1 : 64];
    Team<WAVE> tm{WAVE ? p.team : (int)blockDim.x, red, 0};
    const int lane = WAVE ? (threadIdx.x & (tm.team - 1)) : threadIdx.x;
    const unsigned per = WAVE ? 256u / tm.team : 1u;
    const unsigned q = blockIdx.x * per + (WAVE ? threadIdx.x / tm.team : 0);
    const unsigned slots = gridDim.x * per / p.G;       // row slots; the host gives one at least
    const unsigned slot = q / p.G, grp = q - slot * p.G;
    if (slot >= slots) return;      // whole teams (whole blocks where a team is one)
    const int c0 = (int)grp * p.Cg;
    const float inv = 1.f / (float)p.Cg;
    const bool gated = p.z != nullptr;
    const T* xp = reinterpret_cast<const T*>(p.x) + c0;
    const T* zp = gated ? reinterpret_cast<const T*>(p.z) + c0 : nullptr;
    float wt[R][V], bs[R][V];
    load_channels<V, R>(p.weight ? p.weight + c0 : nullptr, 1.f, lane, tm.team, p.Cg, wt);
    load_channels<V, R>(p.bias ? p.bias + c0 : nullptr, 0.f, lane, tm.team, p.Cg, bs);
    Row<T, V, R> nx, nz;
    size_t row = slot;
    if (row < (size_t)p.rows) {
        nx.load(xp + row * p.x_stride, lane, tm.team, p.Cg);
        if (gated) nz.load(zp + row * p.z_stride, lane, tm.team, p.Cg);
    }
    for (; row < (size_t)p.rows; row += slots) {
        const Row<T, V, R> x = nx, z = nz;
        if (row + slots < (size_t)p.rows) {
            nx.load(xp + (row + slots) * p.x_stride, lane, tm.team, p.Cg);
            if (gated) nz.load(zp + (row + slots) * p.z_stride, lane, tm.team, p.Cg);
        }
        float u[R][V];
        const float rstd = normalise<T, V, R, WAVE>(p, tm, x, z, lane, inv, u);
        T* y = reinterpret_cast<T*>(p.y) + row * p.C + c0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (lane + r * tm.team) * V;
            Vec<T, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float n = fmaf(u[r][i] * rstd, wt[r][i], bs[r][i]);
                if (!gated)
                    n = act_of<T>(n, p.act);
                else if (!p.gate_first)
                    n *= act_of<T>(z.x[r].f(i), p.act);
                o.set(i, n);
            }
            if (c < p.Cg) o.store(y + c);
        }
    }
}

// Backward: with hat = (u - m) rstd and g = d_n weight,
//   d_u = rstd (g - hat mean(g hat) - [center] mean(g))
//   dweight = sum d_n hat, dbias = sum d_n
// A block's teams share one group (blockIdx.y) and walk rows; the parameter
// sums stay in registers, are joined across the block's teams in LDS and leave
// as one partial row per block, summed in a fixed order by the row-sum kernel.
// A block so reads 2 C / G bytes of each row (bf16), for narrow groups a part of
// a cache line: 8192 x 4096 bf16 behind a gate (336 MB), 32 or 8 groups 73 us,
// 128 groups 82, 512 groups 142; one group (512 threads a block, each sum over
// eight waves) 149.
template <typename T, int V, int R, bool WAVE, int BLOCK>
__global__ __launch_bounds__(BLOCK) void kda_norm_bwd_kernel(NormParams p) {
    __shared__ float red[WAVE ? 256 * V : 64];
    Team<WAVE> tm{WAVE ? p.team : (int)blockDim.x, red, 0};
    const int teams = WAVE ? 256 / tm.team : 1;
    const int lane = WAVE ? (threadIdx.x & (tm.team - 1)) : threadIdx.x;
    const int slot = WAVE ? threadIdx.x / tm.team : 0;
    const int c0 = (int)blockIdx.y * p.Cg;
    const float inv = 1.f / (float)p.Cg;
    const bool gated = p.z != nullptr;
    const T* xp = reinterpret_cast<const T*>(p.x) + c0;
    const T* gp = reinterpret_cast<const T*>(p.d_y) + c0;
    const T* zp = gated ? reinterpret_cast<const T*>(p.z) + c0 : nullptr;
    float wt[R][V], bs[R][V], dw[R][V], db[R][V];
    load_channels<V, R>(p.weight ? p.weight + c0 : nullptr, 1.f, lane, tm.team, p.Cg, wt);
    load_channels<V, R>(p.bias ? p.bias + c0 : nullptr, 0.f, lane, tm.team, p.Cg, bs);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[r][i] = db[r][i] = 0.f;
    const size_t step = (size_t)gridDim.x * teams, rows = (size_t)p.rows;
    size_t row = (size_t)blockIdx.x * teams + slot;
    Row<T, V, R> nx, nz, ng;
    auto fetch = [&](size_t at) {
        nx.load(xp + at * p.x_stride, lane, tm.team, p.Cg);
        ng.load(gp + at * p.C, lane, tm.team, p.Cg);
        if (gated) nz.load(zp + at * p.z_stride, lane, tm.team, p.Cg);
    };
    if (row < rows) fetch(row);
    for (; row < rows; row += step) {
        const Row<T, V, R> x = nx, z = nz, g = ng;
        if (row + step < rows) fetch(row + step);
        float u[R][V];
        const float rstd = normalise<T, V, R, WAVE>(p, tm, x, z, lane, inv, u);
        // u <- hat, gv <- d_n weight; the gate behind the norm takes its gradient here
        float gv[R][V];
        float s1 = 0.f, s2 = 0.f;
        T* dz = p.dz ? reinterpret_cast<T*>(p.dz) + row * p.C + c0 : nullptr;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (lane + r * tm.team) * V;
            Vec<T, V> oz;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                u[r][i] *= rstd;
                float d = g.x[r].f(i);      // zero behind the group's end
                if (!gated) {
                    d *= dact_of<T>(fmaf(u[r][i], wt[r][i], bs[r][i]), p.act);
                } else if (!p.gate_first) {
                    const float zi = z.x[r].f(i);
                    oz.set(i, d * fmaf(u[r][i], wt[r][i], bs[r][i]) * dact_of<T>(zi, p.act));
                    d *= act_of<T>(zi, p.act);
                }
                dw[r][i] = fmaf(d, u[r][i], dw[r][i]);
                db[r][i] += d;
                d *= wt[r][i];
                gv[r][i] = d;
                s1 += d;
                s2 = fmaf(d, u[r][i], s2);
            }
            if (gated && !p.gate_first && c < p.Cg) oz.store(dz + c);
        }
        tm.sum2(s2, s1, p.center);
        s2 *= inv;
        s1 = p.center ? s1 * inv : 0.f;
        T* dx = reinterpret_cast<T*>(p.dx) + row * p.C + c0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (lane + r * tm.team) * V;
            Vec<T, V> ox, oz;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float d = rstd * (gv[r][i] - fmaf(u[r][i], s2, s1));
                if (gated && p.gate_first) {
                    const float zi = z.x[r].f(i);
                    oz.set(i, d * x.x[r].f(i) * dact_of<T>(zi, p.act));
                    d *= act_of<T>(zi, p.act);
                }
                ox.set(i, d);
            }
            if (c < p.Cg) {
                ox.store(dx + c);
                if (gated && p.gate_first) oz.store(dz + c);
            }
        }
    }
    if (!p.part) return;
    float* part = p.part + (size_t)blockIdx.x * 2 * p.C + c0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        for (int m = 0; m < 2; ++m) {
            if constexpr (WAVE) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < V; ++i) red[threadIdx.x * V + i] = m ? db[r][i] : dw[r][i];
                __syncthreads();
                for (int k = threadIdx.x; k < tm.team * V; k += 256) {
                    const int c = r * tm.team * V + k;
                    if (c >= p.Cg) continue;
                    float s = 0.f;
                    for (int t = 0; t < teams; ++t) s += red[t * tm.team * V + k];
                    part[(size_t)m * p.C + c] = s;
                }
            } else {
                const int c = (lane + r * tm.team) * V;
                if (c < p.Cg) {
#pragma unroll
                    for (int i = 0; i < V; ++i) part[(size_t)m * p.C + c + i] = m ? db[r][i] : dw[r][i];
                }
            }
        }
    }
}

template <typename T, int V, int R, bool WAVE>
hipError_t norm_launch(bool bwd, int block, const NormParams& p, int blocks, hipStream_t st) {
    const dim3 grid((unsigned)blocks, (unsigned)p.G);
    // blocks of up to 256 threads may use all registers: bounded for 1024 the
    // backward spills, 148 us instead of 124 us on 16384 rows of 2048
    if (bwd && block <= 256)
        hipLaunchKernelGGL((kda_norm_bwd_kernel<T, V, R, WAVE, 256>), grid, dim3(block), 0, st, p);
    else if (bwd)
        hipLaunchKernelGGL((kda_norm_bwd_kernel<T, V, R, WAVE, WAVE ? 256 : 1024>), grid, dim3(block), 0, st, p);
    else
        hipLaunchKernelGGL((kda_norm_fwd_kernel<T, V, R, WAVE>), dim3((unsigned)blocks), dim3(block), 0, st, p);
    return hipGetLastError();
}

template <typename T, int V>
hipError_t norm_pick(bool bwd, int R, int block, const NormParams& p, int blocks, hipStream_t st) {
    if (p.team <= 64) return norm_launch<T, V, 1, true>(bwd, block, p, blocks, st);
    if (R == 1) return norm_launch<T, V, 1, false>(bwd, block, p, blocks, st);
    if (R == 2) return norm_launch<T, V, 2, false>(bwd, block, p, blocks, st);
    if constexpr (V != 8) return norm_launch<T, V, 4, false>(bwd, block, p, blocks, st);
    return hipErrorInvalidValue;
}

hipError_t norm_any(bool bwd, int dtype, bool vec, int R, int block, const NormParams& p, int blocks, hipStream_t st) {
    if (dtype == 1)
        return vec ? norm_pick<bf16, 8>(bwd, R, block, p, blocks, st) : norm_pick<bf16, 1>(bwd, R, block, p, blocks, st);
    return vec ? norm_pick<float, 4>(bwd, R, block, p, blocks, st) : norm_pick<float, 1>(bwd, R, block, p, blocks, st);
}

}  // namespace

// The team of a group of Cg channels: the smallest power of two of lanes that
// holds it in one access each, up to a wave; then whole waves up to a block of
// 1024 threads; then 1024 threads with two or four accesses (16 values a lane).
// Wider groups have no kernel.
bool norm_variant(int dtype, bool vec, int Cg, int* R, int* team, int* block) {
    const int V = vec ? (dtype == 1 ? 8 : 4) : 1;
    const int n = (Cg + V - 1) / V;
    *R = 1;
    if (n <= 64) {
        int t = 1;
        while (t < n) t <<= 1;
        *team = t;
        *block = 256;
        return true;
    }
    *block = *team = n < 1024 ? (n + 63) / 64 * 64 : 1024;
    if (n <= 1024) return true;
    *R = n <= 2048 ? 2 : 4;
    return n <= (V == 8 ? 2048 : 4096);
}

hipError_t launch_norm_fwd(int dtype, bool vec, int R, int block, const NormParams& p, int blocks, hipStream_t st) {
    return norm_any(false, dtype, vec, R, block, p, blocks, st);
}
hipError_t launch_norm_bwd(int dtype, bool vec, int R, int block, const NormParams& p, int row_blocks,
                           hipStream_t st) {
    return norm_any(true, dtype, vec, R, block, p, row_blocks, st);
}

}  // namespace kda
