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
#include "kda_mixer.h"
#include "kda_mixer_device.h"

namespace kda {

namespace {

// Sum over a team: lanes of a wave (team <= 64), or the whole block.
template <bool WAVE>
__device__ __forceinline__ float team_sum(float v, int team, float* red) {
    const int w = WAVE ? team : 64;
    for (int m = w >> 1; m > 0; m >>= 1) v += __shfl_xor(v, m);
    if constexpr (!WAVE) {
        const int nw = blockDim.x >> 6;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
        for (int k = 0; k < nw; ++k) v += red[k];
    }
    return v;
}

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

template <typename T, int V, int R, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void kda_norm_fwd_kernel(NormParams p) {
    __shared__ float red[16];
    const int team = WAVE ? p.team : (int)blockDim.x;
    const int lane = WAVE ? (threadIdx.x & (team - 1)) : threadIdx.x;
    const long long unit = WAVE ? ((long long)blockIdx.x * (256 / team) + threadIdx.x / team) : blockIdx.x;
    const long long units = (long long)p.rows * p.G;
    if (unit >= units) return;      // WAVE only: no barrier follows
    const long long row = unit / p.G;
    const int c0 = (int)(unit - row * p.G) * p.Cg;
    Row<T, V, R> x, z;
    x.load(reinterpret_cast<const T*>(p.x) + (size_t)row * p.x_stride + c0, lane, team, p.Cg);
    const bool gated = p.z != nullptr;
    if (gated) z.load(reinterpret_cast<const T*>(p.z) + (size_t)row * p.z_stride + c0, lane, team, p.Cg);
    float u[R][V];
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool in = (lane + r * team) * V < p.Cg;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            u[r][i] = x.x[r].f(i);
            if (gated && p.gate_first) u[r][i] = in ? u[r][i] * act_of<T>(z.x[r].f(i), p.act) : 0.f;
            sum += u[r][i];
        }
    }
    const float inv = 1.f / (float)p.Cg;
    if (p.center) {
        const float mean = team_sum<WAVE>(sum, team, red) * inv;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = (lane + r * team) * V < p.Cg;
#pragma unroll
            for (int i = 0; i < V; ++i) u[r][i] = in ? u[r][i] - mean : 0.f;
        }
    }
    float sq = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < V; ++i) sq = fmaf(u[r][i], u[r][i], sq);
    const float rstd = 1.f / sqrtf(team_sum<WAVE>(sq, team, red) * inv + p.eps);
    T* y = reinterpret_cast<T*>(p.y) + (size_t)row * p.C + c0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (lane + r * team) * V;
        if (c >= p.Cg) continue;
        Vec<T, V> o;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float n = u[r][i] * rstd;
            if (p.weight) n *= p.weight[c0 + c + i];
            if (p.bias) n += p.bias[c0 + c + i];
            if (!gated)
                n = act_of<T>(n, p.act);
            else if (!p.gate_first)
                n *= act_of<T>(z.x[r].f(i), p.act);
            o.set(i, n);
        }
        o.store(y + c);
    }
}

// Backward: with hat = (u - m) rstd and g = d_n weight,
//   d_u = rstd (g - hat mean(g hat) - [center] mean(g))
//   dweight = sum d_n hat, dbias = sum d_n
// A block's teams share one group (blockIdx.y) and walk rows; the parameter
// sums stay in registers, are joined across the block's teams in LDS and leave
// as one partial row per block, summed in a fixed order by the row-sum kernel.
template <typename T, int V, int R, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void kda_norm_bwd_kernel(NormParams p) {
    __shared__ float red[WAVE ? 256 * V : 16];
    const int team = WAVE ? p.team : (int)blockDim.x;
    const int teams = WAVE ? 256 / team : 1;
    const int lane = WAVE ? (threadIdx.x & (team - 1)) : threadIdx.x;
    const int slot = WAVE ? threadIdx.x / team : 0;
    const int c0 = (int)blockIdx.y * p.Cg;
    const float inv = 1.f / (float)p.Cg;
    const bool gated = p.z != nullptr;
    float wt[R][V], bs[R][V], dw[R][V], db[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (lane + r * team) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            wt[r][i] = p.weight && c < p.Cg ? p.weight[c0 + c + i] : 1.f;
            bs[r][i] = p.bias && c < p.Cg ? p.bias[c0 + c + i] : 0.f;
            dw[r][i] = db[r][i] = 0.f;
        }
    }
    for (long long row = (long long)blockIdx.x * teams + slot; row < p.rows; row += (long long)gridDim.x * teams) {
        Row<T, V, R> x, z, g;
        x.load(reinterpret_cast<const T*>(p.x) + (size_t)row * p.x_stride + c0, lane, team, p.Cg);
        g.load(reinterpret_cast<const T*>(p.d_y) + (size_t)row * p.C + c0, lane, team, p.Cg);
        if (gated) z.load(reinterpret_cast<const T*>(p.z) + (size_t)row * p.z_stride + c0, lane, team, p.Cg);
        float u[R][V];
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = (lane + r * team) * V < p.Cg;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                u[r][i] = x.x[r].f(i);
                if (gated && p.gate_first) u[r][i] = in ? u[r][i] * act_of<T>(z.x[r].f(i), p.act) : 0.f;
                sum += u[r][i];
            }
        }
        if (p.center) {
            const float mean = team_sum<WAVE>(sum, team, red) * inv;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool in = (lane + r * team) * V < p.Cg;
#pragma unroll
                for (int i = 0; i < V; ++i) u[r][i] = in ? u[r][i] - mean : 0.f;
            }
        }
        float sq = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < V; ++i) sq = fmaf(u[r][i], u[r][i], sq);
        const float rstd = 1.f / sqrtf(team_sum<WAVE>(sq, team, red) * inv + p.eps);
        // u <- hat, gv <- d_n weight; the gate behind the norm takes its gradient here
        float gv[R][V];
        float s1 = 0.f, s2 = 0.f;
        T* dz = p.dz ? reinterpret_cast<T*>(p.dz) + (size_t)row * p.C + c0 : nullptr;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (lane + r * team) * V;
            Vec<T, V> oz;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                u[r][i] *= rstd;
                float d = g.x[r].f(i);
                if (!gated) {
                    d *= dact_of<T>(fmaf(u[r][i], wt[r][i], bs[r][i]), p.act);
                } else if (!p.gate_first) {
                    const float zi = z.x[r].f(i);
                    oz.set(i, d * fmaf(u[r][i], wt[r][i], bs[r][i]) * dact_of<T>(zi, p.act));
                    d *= act_of<T>(zi, p.act);
                }
                if (c >= p.Cg) d = 0.f;
                dw[r][i] = fmaf(d, u[r][i], dw[r][i]);
                db[r][i] += d;
                d *= wt[r][i];
                gv[r][i] = d;
                s1 += d;
                s2 = fmaf(d, u[r][i], s2);
            }
            if (gated && !p.gate_first && c < p.Cg) oz.store(dz + c);
        }
        s2 = team_sum<WAVE>(s2, team, red) * inv;
        s1 = p.center ? team_sum<WAVE>(s1, team, red) * inv : 0.f;
        T* dx = reinterpret_cast<T*>(p.dx) + (size_t)row * p.C + c0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (lane + r * team) * V;
            if (c >= p.Cg) continue;
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
            ox.store(dx + c);
            if (gated && p.gate_first) oz.store(dz + c);
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
                for (int k = threadIdx.x; k < team * V; k += 256) {
                    const int c = r * team * V + k;
                    if (c >= p.Cg) continue;
                    float s = 0.f;
                    for (int t = 0; t < teams; ++t) s += red[t * team * V + k];
                    part[(size_t)m * p.C + c] = s;
                }
            } else {
                const int c = (lane + r * team) * V;
                if (c < p.Cg) {
#pragma unroll
                    for (int i = 0; i < V; ++i) part[(size_t)m * p.C + c + i] = m ? db[r][i] : dw[r][i];
                }
            }
        }
    }
}

template <typename T, int V, int R, bool WAVE>
hipError_t norm_launch(bool bwd, int block, const NormParams& p, int row_blocks, hipStream_t st) {
    if (bwd) {
        hipLaunchKernelGGL((kda_norm_bwd_kernel<T, V, R, WAVE>), dim3((unsigned)row_blocks, (unsigned)p.G),
                           dim3(block), 0, st, p);
    } else {
        const long long units = (long long)p.rows * p.G;
        const long long per = WAVE ? 256 / p.team : 1;
        hipLaunchKernelGGL((kda_norm_fwd_kernel<T, V, R, WAVE>), dim3((unsigned)((units + per - 1) / per)),
                           dim3(block), 0, st, p);
    }
    return hipGetLastError();
}

template <typename T, int V>
hipError_t norm_pick(bool bwd, int R, int block, const NormParams& p, int rb, hipStream_t st) {
    if (p.team <= 64) {
        if (R == 1) return norm_launch<T, V, 1, true>(bwd, block, p, rb, st);
        if (R == 2) return norm_launch<T, V, 2, true>(bwd, block, p, rb, st);
        return norm_launch<T, V, 4, true>(bwd, block, p, rb, st);
    }
    if (R == 2) return norm_launch<T, V, 2, false>(bwd, block, p, rb, st);
    return norm_launch<T, V, 4, false>(bwd, block, p, rb, st);
}

hipError_t norm_any(bool bwd, int dtype, bool vec, int R, int block, const NormParams& p, int rb, hipStream_t st) {
    if (dtype == 1)
        return vec ? norm_pick<bf16, 8>(bwd, R, block, p, rb, st) : norm_pick<bf16, 1>(bwd, R, block, p, rb, st);
    return vec ? norm_pick<float, 4>(bwd, R, block, p, rb, st) : norm_pick<float, 1>(bwd, R, block, p, rb, st);
}

}  // namespace

// The team of a group: the smallest power of two of lanes (up to a wave) that
// holds it in one access each, a wave with two or four, else a block of 256 or
// 1024 threads with two or four.  Wider groups have no kernel.
bool norm_variant(int dtype, bool vec, int Cg, int* R, int* team, int* block) {
    const int V = vec ? (dtype == 1 ? 8 : 4) : 1;
    const int n = (Cg + V - 1) / V;
    *block = 256;
    if (n <= 64) {
        int t = 1;
        while (t < n) t <<= 1;
        *team = t;
        *R = 1;
        return true;
    }
    if (n <= 256) {
        *team = 64;
        *R = n <= 128 ? 2 : 4;
        return true;
    }
    for (int b = 256; b <= 1024; b <<= 2) {
        // 1024 threads have 128 registers each: two 16-byte accesses of bf16 at most
        if (n <= (b == 1024 && V == 8 ? 2 : 4) * b) {
            *block = *team = b;
            *R = n <= 2 * b ? 2 : 4;
            return true;
        }
    }
    return false;
}

hipError_t launch_norm_fwd(int dtype, bool vec, int R, int block, const NormParams& p, hipStream_t st) {
    return norm_any(false, dtype, vec, R, block, p, 0, st);
}
hipError_t launch_norm_bwd(int dtype, bool vec, int R, int block, const NormParams& p, int row_blocks,
                           hipStream_t st) {
    return norm_any(true, dtype, vec, R, block, p, row_blocks, st);
}

}  // namespace kda
