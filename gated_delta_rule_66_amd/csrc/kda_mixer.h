// Host-side declarations of the mixer operators (short convolution, selective
// scan, group norm): launch parameters and launchers.  The contracts are in
// include/kda.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace kda {

// Sequences of a call: a regular batch (cu null: N sequences of T tokens) or a
// packed axis of T tokens with the N + 1 offsets cu.
struct SeqView {
    const int* cu;
    int N, T;
};

// ---- short convolution -------------------------------------------------------------
struct ConvParams {
    SeqView sv;
    int D, W, act;          // act: kda_activation
    int tiles;              // token tiles (regular batch: N * tiles_per_seq)
    int tiles_per_seq;      // regular batch only
    int tile_tokens;
    int cx_log2;            // threads of a block along the channels: 1 << cx_log2
    const void* x;
    size_t x_stride;        // elements between token rows
    const float* weight;    // [D][W]
    const float* bias;      // [D] or null
    const void* s0;         // [N][W-1][D] or null (zeros)
    void* y;                // [tokens][D]
    void* sT;               // [N][W-1][D] or null
    // backward
    const void* d_y;        // [tokens][D]
    const void* d_sT;       // [N][W-1][D] or null
    void* dx;
    float* part;            // [blocks of tiles][W + 1][D]: sums of one block
    void* d_s0;             // [N][W-1][D] or null
};
hipError_t launch_conv_fwd(int dtype, bool vec, const ConvParams& p, int tile_blocks, hipStream_t st);
hipError_t launch_conv_bwd(int dtype, bool vec, const ConvParams& p, int tile_blocks, hipStream_t st);
hipError_t launch_conv_step(int dtype, bool vec, int N, int D, int W, int act, const void* x, size_t x_stride,
                            const float* weight, const float* bias, void* state, void* y, hipStream_t st);
// out0[d][m] (m < M0) and out1[d] (m = M0) = the sums over rows of part [rows][M][D]
hipError_t launch_sum_rows(const float* part, int rows, int M, int D, float* out0, int M0, float* out1,
                           hipStream_t st);

// ---- group norm --------------------------------------------------------------------
struct NormParams {
    int rows, C, G, Cg;
    int act, center, gate_first;
    float eps;
    const void* x;
    size_t x_stride;
    const void* z;          // gate or null
    size_t z_stride;
    const float* weight;    // [C] or null
    const float* bias;      // [C] or null
    void* y;                // [rows][C]
    const void* d_y;        // [rows][C]
    void* dx;
    void* dz;               // [rows][C] (with a gate)
    float* part;            // [row blocks][2][C] or null
    int team;               // lanes that share one group of one row
};
// lanes (team), accesses a lane (R) and block of a group; false: too wide
bool norm_variant(int dtype, bool vec, int Cg, int* R, int* team, int* block);
hipError_t launch_norm_fwd(int dtype, bool vec, int R, int block, const NormParams& p, int blocks, hipStream_t st);
hipError_t launch_norm_bwd(int dtype, bool vec, int R, int block, const NormParams& p, int row_blocks,
                           hipStream_t st);

// ---- selective scan ----------------------------------------------------------------
// Chunks of 64 tokens are numbered over the whole call: sequence i has
// max(1, ceil(len_i / 64)) of them, so a sequence without tokens has one empty
// chunk, which passes its state on.  A segment is a run of cps chunks.
struct SsmParams {
    SeqView sv;
    int H, G, K, P;             // heads, groups, state rows, head columns
    int softplus;
    const void* x;              // [tokens][H][P]
    size_t x_stride;            // elements between token rows
    const void* dt;             // [tokens][H]
    size_t dt_stride;
    const float* A;             // [H]
    const float* dt_bias;       // [H] or null
    const float* Dskip;         // [H] or null
    const void* B;              // [tokens][G][K]
    size_t b_stride;
    const void* C;
    size_t c_stride;
    const float* s0;            // [N][H][K][P] or null (zeros)
    void* y;                    // [tokens][H][P]
    float* sT;                  // [N][H][K][P] or null
    int chunks;                 // chunks of the call (packed: their bound)
    int chunks_per_seq;         // regular batch
    const int* chunk_off;       // packed: [N + 1]
    int n_seg, cps;
    int seg0;                   // first segment of the launch
    int reverse;                // 1: the adjoint's recurrence, from the last chunk to the first
    int in_place;               // 1: sT is s0, and there are segments (kda_ssm_chunk_kernel)
    float* gates;               // [chunks][H][5][64] (kda_ssm_device.h)
    // what one segment does to its start state: local states [n_seg][H][K][P]
    // (after the combine: start states) and decays [n_seg][H] (negative: a
    // sequence starts in the segment, nothing of the start state is left)
    float* seg_state;
    float* seg_decay;
    float* states;              // [chunks][H][K][P]: the state before each chunk (the states pass)
};
constexpr int kSsmChunk = 64;
// chunk_off[i] = chunks of the sequences before i
hipError_t launch_ssm_prep(const SeqView& sv, int* chunk_off, int max_chunks, hipStream_t st);
// step sizes and decays of every chunk and head
size_t ssm_gate_bytes(int chunks, int H);
hipError_t launch_ssm_gates(int dtype, const SsmParams& p, hipStream_t st);
// One or two recurrences of the same sizes in one launch (the second: the
// backward's adjoint)
struct SsmPair {
    SsmParams p[2];
};
enum SsmPass {
    kSsmOutput,     // y and the final states
    kSsmSummary,    // each segment's local state and decay
    kSsmStates      // the state before each chunk, and the final states
};
hipError_t launch_ssm_chunks(int dtype, SsmPass pass, int cols, const SsmPair& a, int n, int segs, hipStream_t st);
hipError_t launch_ssm_combine(const SsmPair& a, int n, hipStream_t st);
// in_place: the final states that the output pass left in the segments' slots
hipError_t launch_ssm_final(const SsmParams& p, hipStream_t st);

// Gradients of the scan from the state before each chunk and the adjoint
// behind it.  A workgroup takes one chunk and heads_per of the heads of a group.
struct SsmBwdParams {
    SsmParams f;                // the forward's inputs and gates
    const void* d_y;            // [tokens][H][P]
    const float* start;         // [chunks][H][K][P]
    const float* dend;          // [chunks][H][K][P]
    void* dx;
    size_t dx_stride;
    void* ddt;                  // [tokens][H]
    void* dB;                   // one part: [tokens][G][K] with its stride
    size_t db_stride;
    void* dC;
    size_t dc_stride;
    float* dB_part;             // [parts][tokens][G][K] (more than one part)
    float* dC_part;
    float* sums;                // [chunks][3][H]: dA, ddt_bias, dD of each chunk
    int parts, heads_per;
};
hipError_t launch_ssm_bwd(int dtype, const SsmBwdParams& p, hipStream_t st);
// dB, dC: the parts summed, rounded to dt
hipError_t launch_ssm_bwd_join(int dtype, const SsmBwdParams& p, long long tokens, hipStream_t st);
hipError_t launch_ssm_bwd_sums(const float* sums, int rows, int H, float* dA, float* dbias, float* dD, hipStream_t st);
hipError_t launch_ssm_step(int dtype, int N, int H, int G, int K, int P, int softplus, const void* x, size_t x_stride,
                           const void* dt, size_t dt_stride, const float* A, const void* B, size_t b_stride, const void* C,
                           size_t c_stride, const float* Dskip, const float* dt_bias, float* state, void* y,
                           hipStream_t st);

}  // namespace kda
