// Device helpers of the selective scan, forward and backward.
#pragma once

#include "kda_mixer.h"
#include "kda_mixer_device.h"

namespace kda {

// delta = softplus(raw) = log1p(exp(raw)), kept from overflowing; its
// derivative is sigmoid(raw)
__device__ __forceinline__ float softplus_of(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

// 2^e for an fp64 exponent as fp32: the fraction on the transcendental unit,
// the integer part exactly.  An fp32 e of magnitude 100 would be off by
// 100 * 2^-24 already; here only the fraction is rounded.
__device__ __forceinline__ float exp2_of(double e) {
    const double r = rint(e);
    const float f = fast_exp2((float)(e - r));
    return ldexpf(f, (int)fmin(fmax(r, -1000.0), 1000.0));
}

// Position in the call's chunks.
struct ChunkWalk {
    SeqView sv;
    const int* off;
    int per_seq;
    int seq, k, nk;     // sequence, chunk in it, its chunks
    int s0, len_seq;

    // a wave's chunks are the wave's: what is read stays in scalar registers
    static __device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }
    __device__ __forceinline__ void enter(int s) {
        seq = s;
        if (sv.cu) {
            nk = scalar(off[s + 1] - off[s]);
            s0 = scalar(min(max(sv.cu[s], 0), sv.T));
            len_seq = scalar(max(min(sv.cu[s + 1], sv.T) - s0, 0));
        } else {
            nk = per_seq;
            s0 = s * sv.T;
            len_seq = sv.T;
        }
    }
    __device__ __forceinline__ void init(const SsmParams& p, int c) {
        sv = p.sv;
        off = p.chunk_off;
        per_seq = p.chunks_per_seq;
        if (sv.cu) {
            int lo = 0, hi = sv.N;      // off[lo] <= c < off[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (scalar(off[mid]) <= c)
                    lo = mid;
                else
                    hi = mid;
            }
            enter(lo);
            k = c - scalar(off[lo]);
        } else {
            const int s = c / per_seq;
            enter(s);
            k = c - s * per_seq;
        }
    }
    __device__ __forceinline__ void next() {
        if (++k == nk && seq + 1 < sv.N) {
            enter(seq + 1);
            k = 0;
        }
    }
    __device__ __forceinline__ void prev() {
        if (--k < 0 && seq > 0) {
            enter(seq - 1);
            k = nk - 1;
        }
    }
    __device__ __forceinline__ bool first() const { return k == 0; }
    __device__ __forceinline__ bool last() const { return k == nk - 1; }
    __device__ __forceinline__ int t0() const { return s0 + k * kSsmChunk; }
    __device__ __forceinline__ int len() const { return min(kSsmChunk, max(len_seq - k * kSsmChunk, 0)); }
};

__device__ __forceinline__ int total_chunks(const SsmParams& p) {
    return p.sv.cu ? min(__builtin_amdgcn_readfirstlane(p.chunk_off[p.sv.N]), p.chunks) : p.chunks;
}

// Workgroups go to the 8 XCDs in turn.  The work index of a block such that
// each XCD takes a contiguous range: the heads of a segment, which read the
// same B and C rows, then meet in one XCD's L2.
__device__ __forceinline__ int xcd_swizzle(int id, int total) {
    const int q = total >> 3, r = total & 7, x = id & 7;
    return x * q + min(x, r) + (id >> 3);
}

// Padding of an LDS tile's rows (elements of T) that transposing reads touch:
// four rows of 32 bytes go out together, which rows of 256 bytes need 32 bytes
// between them for; shorter and longer rows do with 16.
template <typename T> constexpr int tr_pad(int width) { return width * (int)sizeof(T) == 256 ? 32 / (int)sizeof(T) : 16 / (int)sizeof(T); }

// ---- fragments whose slots run over the tokens (rows) of an LDS tile ----------------
// lane l: column n0 + l % 16, slots (g, i) -> token tok0 + 16 (i / 4) + 4 g + i % 4
// (the permuted slots of ld_frag_perm).
// bf16: ds_read_b64_tr_b16 transposes 16 tokens x 16 columns across 16 lanes:
// lane r of a group reads four columns of token r / 4, and gets four tokens of
// column r.
__device__ __forceinline__ bf16x4 ld_tr4(const bf16* p) {
    typedef __attribute__((address_space(3))) bf16x4 lds_x4;
    return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_x4*)p);
}
__device__ __forceinline__ bf16x8 ld_frag_tokens(const bf16* tile, int ld, int tok0, int n0, int lane) {
    const int g = lane >> 4, r = lane & 15;
    const bf16* p = tile + (tok0 + 4 * g + (r >> 2)) * ld + n0 + 4 * (r & 3);
    const bf16x4 a = ld_tr4(p), b = ld_tr4(p + 16 * ld);
    bf16x8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) { f[i] = a[i]; f[4 + i] = b[i]; }
    return f;
}
__device__ __forceinline__ f32x8 ld_frag_tokens(const float* tile, int ld, int tok0, int n0, int lane) {
    const int g = lane >> 4, r = lane & 15;
    const float* p = tile + (tok0 + 4 * g) * ld + n0 + r;
    f32x8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) { f[i] = p[i * ld]; f[4 + i] = p[(16 + i) * ld]; }
    return f;
}

// LDS tiles whose columns are a reduction axis, in slot order: in every 32
// columns the groups of four go 0, 4, 1, 5, 2, 6, 3, 7, so that a lane's eight
// permuted slots (4 g .. and 16 + 4 g ..) are one 16-byte read.
__device__ __forceinline__ int slot_col(int col) {      // of a multiple of four
    return (col & ~31) + ((col & 12) << 1) + ((col & 16) >> 2);
}
// a 16-byte piece of a row (columns col ..), stored in slot order
__device__ __forceinline__ void st_slots(bf16* row, int col, uint4 v) {
    *reinterpret_cast<uint2*>(row + slot_col(col)) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(row + slot_col(col + 4)) = make_uint2(v.z, v.w);
}
__device__ __forceinline__ void st_slots(float* row, int col, uint4 v) {
    *reinterpret_cast<uint4*>(row + slot_col(col)) = v;
}

// ---- fp32 operands of bf16 products ---------------------------------------------------
// v = hi + mid + lo with eight significant bits each, by truncation: exact for
// fp32, so that three bf16 products keep an fp32 state at fp32 accuracy.
struct Split3 {
    bf16x8 hi, mid, lo;
};
__device__ __forceinline__ unsigned hi16_pair(float a, float b) {
    // the upper halves of a (low lane) and b (high lane)
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ float trunc_bf16(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }
__device__ __forceinline__ Split3 split3(const float* v) {
    unsigned h[4], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = v[2 * i], b = v[2 * i + 1];
        h[i] = hi16_pair(a, b);
        const float a1 = a - trunc_bf16(a), b1 = b - trunc_bf16(b);
        m[i] = hi16_pair(a1, b1);
        l[i] = hi16_pair(a1 - trunc_bf16(a1), b1 - trunc_bf16(b1));
    }
    Split3 s;
    s.hi = *reinterpret_cast<bf16x8*>(h);
    s.mid = *reinterpret_cast<bf16x8*>(m);
    s.lo = *reinterpret_cast<bf16x8*>(l);
    return s;
}
// acc += a * v over one slab, v fp32 (a exact in T)
__device__ __forceinline__ f32x4 mma_exact(f32x4 acc, bf16x8 a, const Split3& v) {
    acc = mma(acc, a, v.lo);
    acc = mma(acc, a, v.mid);
    return mma(acc, a, v.hi);
}
__device__ __forceinline__ f32x4 mma_exact(f32x4 acc, f32x8 a, const f32x8& v) { return mma(acc, a, v); }
template <typename T> struct Exact;
template <> struct Exact<bf16> {
    typedef Split3 type;
    static __device__ __forceinline__ Split3 of(const float* v) { return split3(v); }
};
template <> struct Exact<float> {
    typedef f32x8 type;
    static __device__ __forceinline__ f32x8 of(const float* v) { return frag_from<float>(v); }
};

// v = hi + lo, hi by truncation, lo rounded: off by 2^-16 relative at most.
// What an output that is rounded to bf16 behind its products takes of an fp32
// operand; one bf16 alone would add half as much again as the output's own
// rounding.  (hi rounded too: 2^-17, and the output pass 3 % slower.)
struct Split2 {
    bf16x8 hi, lo;
};
__device__ __forceinline__ Split2 split2(const float* v) {
    unsigned h[4];
    Split2 s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = hi16_pair(v[2 * i], v[2 * i + 1]);
        s.lo[2 * i] = (bf16)(v[2 * i] - trunc_bf16(v[2 * i]));
        s.lo[2 * i + 1] = (bf16)(v[2 * i + 1] - trunc_bf16(v[2 * i + 1]));
    }
    s.hi = *reinterpret_cast<bf16x8*>(h);
    return s;
}
// acc[i] += v b[i] or v[i] b: all lower halves first, so that the products of
// one accumulator are apart
template <int N> __device__ __forceinline__ void mma_near(f32x4 (&acc)[N], const Split2 (&v)[N], bf16x8 b) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = mma(acc[i], v[i].lo, b);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = mma(acc[i], v[i].hi, b);
}
template <int N> __device__ __forceinline__ void mma_near(f32x4 (&acc)[N], const f32x8 (&v)[N], f32x8 b) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = mma(acc[i], v[i], b);
}
template <int N> __device__ __forceinline__ void mma_near(f32x4 (&acc)[N], const Split2& v, const bf16x8 (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = mma(acc[i], v.lo, b[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = mma(acc[i], v.hi, b[i]);
}
template <int N> __device__ __forceinline__ void mma_near(f32x4 (&acc)[N], const f32x8& v, const f32x8 (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = mma(acc[i], v, b[i]);
}
template <typename T> struct Near;
template <> struct Near<bf16> {
    typedef Split2 type;
    static __device__ __forceinline__ Split2 of(const float* v) { return split2(v); }
};
template <> struct Near<float> {
    typedef f32x8 type;
    static __device__ __forceinline__ f32x8 of(const float* v) { return frag_from<float>(v); }
};
// the same, of four values stored to two tiles (fp32: to one)
__device__ __forceinline__ void st_near4(bf16* hi, bf16* lo, const float* v) {
    bf16x4 l;
#pragma unroll
    for (int i = 0; i < 4; ++i) l[i] = (bf16)(v[i] - trunc_bf16(v[i]));
    *reinterpret_cast<uint2*>(hi) = make_uint2(hi16_pair(v[0], v[1]), hi16_pair(v[2], v[3]));
    *reinterpret_cast<bf16x4*>(lo) = l;
}
__device__ __forceinline__ void st_near4(float* hi, float*, const float* v) { st_run<4>(hi, v); }

// Step sizes and decays of one chunk and head, five arrays of 64 floats:
//   c      log2 of the decay from the chunk's start to token j, rounded
//   delta
//   near   delta times the decay from j to the end of its 16 tokens
//   w      delta times the decay from j to the chunk's end
//   rest   c's rounding error
enum Gate { kGateC = 0, kGateDelta = 1, kGateNear = 2, kGateW = 3, kGateRest = 4, kGates = 5 };
// 2^{c + rest}
__device__ __forceinline__ float exp2_pair(float c, float rest) {
    return fast_exp2(c) * fmaf(rest, 0.6931471805599453f, 1.f);
}

// one token's delta for one head
__device__ __forceinline__ float delta_of(float raw, int softplus) { return softplus ? softplus_of(raw) : raw; }

// inclusive sums over each row of 16 lanes (row_shr) and over the 64 lanes of a
// wave (the rows' last lanes broadcast on), fp64
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
    const unsigned long long u = __builtin_bit_cast(unsigned long long, v);
    const unsigned lo = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)u, CTRL, ROWS, 0xf, true);
    const unsigned hi = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)(u >> 32), CTRL, ROWS, 0xf, true);
    return v + __builtin_bit_cast(double, ((unsigned long long)hi << 32) | lo);
}
__device__ __forceinline__ double row_prefix(double v) {
    v = dpp_add<0x111, 0xf>(v);
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    return dpp_add<0x118, 0xf>(v);
}
__device__ __forceinline__ double wave_prefix(double v) {
    v = row_prefix(v);
    v = dpp_add<0x142, 0xa>(v);     // row_bcast:15 into rows 1 and 3
    return dpp_add<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
}
// the value of lane 15 of each row of 16 lanes
__device__ __forceinline__ double row_last(double v) {
    const unsigned long long u = __builtin_bit_cast(unsigned long long, v);
    const unsigned lo = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)u, 0x15f, 0xf, 0xf, true);
    const unsigned hi = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)(u >> 32), 0x15f, 0xf, 0xf, true);
    return __builtin_bit_cast(double, ((unsigned long long)hi << 32) | lo);
}
// lane 63's value, as a scalar
__device__ __forceinline__ double last_lane(double v) {
    const unsigned long long u = __builtin_bit_cast(unsigned long long, v);
    const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)u, 63);
    const unsigned hi = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)(u >> 32), 63);
    return __builtin_bit_cast(double, ((unsigned long long)hi << 32) | lo);
}

// A resource over the rows t0 .. t0 + len - 1 of a token tensor (row stride in
// elements): loads of rows behind them return zeros, stores there do nothing.
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const void* base, size_t stride, int t0, int len, int width) {
    const int t = __builtin_amdgcn_readfirstlane(t0), n = __builtin_amdgcn_readfirstlane(len);
    const unsigned bytes = n > 0 ? (unsigned)(((size_t)(n - 1) * stride + width) * sizeof(T)) : 0u;
    return make_rsrc_n(reinterpret_cast<const T*>(base) + (size_t)t * stride, bytes);
}
__device__ __forceinline__ void buf_store4(__amdgpu_buffer_rsrc_t r, unsigned voff, unsigned soff, const float* x, const bf16*) {
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
    bf16x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (bf16)x[i];
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, v), r, (int)voff, (int)soff, 0);
}
__device__ __forceinline__ void buf_store4(__amdgpu_buffer_rsrc_t r, unsigned voff, unsigned soff, const float* x, const float*) {
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    const f32x4 v = {x[0], x[1], x[2], x[3]};
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, (int)voff, (int)soff, 0);
}

}  // namespace kda
