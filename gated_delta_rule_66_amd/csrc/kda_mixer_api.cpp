// C ABI of the mixer operators: argument validation, launch plans, launches.
// The declarations and their contracts are in include/kda.h.
#include "kda.h"
#include "kda_host.h"
#include "kda_internal.h"
#include "kda_mixer.h"

using namespace kda;

namespace {

// rows of `width` elements, `stride` apart, start and end on whole accesses
bool vec_ok(kda_dtype dt, long long width, long long stride, const void* p, size_t bytes = 16) {
    const long long n = (long long)(bytes / esize(dt));
    return width % n == 0 && stride % n == 0 && aligned(p, bytes);
}

// ---- short convolution ---------------------------------------------------------------

// Tiles (no more than tokens) and sequences are counted in ints that step past
// their end: by the tile slots of the backward's grid (2^19 at most), and by the
// threads that pass on empty sequences (a 64th of the sequences and 256).
constexpr long long kConvCount = (1LL << 31) - (1LL << 26);

kda_status conv_sizes(int N, int T, int D, int W, kda_dtype dt, kda_activation act, const int* cu, long long* M) {
    if (N < 0 || T < 0 || D < 0 || !dtype_ok(dt) || !act_ok(act)) return KDA_ERR_INVALID_ARG;
    if (W < 2 || W > 4) return KDA_ERR_UNSUPPORTED;
    if (!token_count(cu, N, T, M) || *M > kConvCount || N > kConvCount || (long long)N * (W - 1) > 2147483647LL ||
        D > (1 << 21))
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// threads of a block along the channels: as many as the channels fill, at most `most`
int cx_log2_for(int D, int V, int most_log2) {
    int l = 0;
    while (l < most_log2 && (V << l) < D) ++l;
    return l;
}

// Tiles of a call: short ones re-read more halo rows, long ones leave a short
// call with few threads.
void conv_tiles(ConvParams& p, long long M, int tile) {
    p.tile_tokens = tile;
    if (p.sv.cu) {
        p.tiles_per_seq = 0;
        p.tiles = (int)((M + tile - 1) / tile);
    } else {
        p.tiles_per_seq = (p.sv.T + tile - 1) / tile;
        p.tiles = p.sv.N * p.tiles_per_seq;
    }
}

// Blocks of the backward along the tiles: enough threads to cover the card,
// each block leaving one partial row of parameter sums.
struct ConvBwdPlan {
    int cx_log2, tile, blocks;
};
ConvBwdPlan conv_bwd_plan(bool packed, int N, int T, int D, int V) {
    ConvBwdPlan b;
    b.cx_log2 = cx_log2_for(D, V, 6);
    const long long tys = 256 >> b.cx_log2, cb = (D + (V << b.cx_log2) - 1) / (V << b.cx_log2);
    const long long M = packed ? (long long)T : (long long)N * T;
    // bf16 x 2304 channels, tiles of 16, 32, 64 tokens: 32768 tokens 142, 121,
    // 108 us; 8192 tokens 40, 35, 40; 4096 tokens 25, 27, 32; 512 tokens 16, 20,
    // 29 (fp32 in the same order): long tiles leave a short call few threads
    const long long work = M * (D / V);
    b.tile = work >= (1LL << 23) ? 64 : work >= (1LL << 21) ? 32 : 16;
    const long long tiles = packed ? (M + b.tile - 1) / b.tile : (long long)N * ((T + b.tile - 1) / b.tile);
    long long want = (tiles + tys - 1) / tys, most = cb > 0 ? 2048 / cb : 1;
    if (most < 64) most = 64;
    if (want > most) want = most;
    b.blocks = (int)(want > 0 ? want : 1);
    return b;
}

}  // namespace

extern "C" {

kda_status kda_short_conv_fwd(int N, const int* cu_seqlens, int T, int D, int W, kda_dtype dt, kda_activation act,
                              const void* x, long long x_stride, const float* weight, const float* bias,
                              const void* initial_state, void* y, void* final_state, hipStream_t stream) {
    long long M;
    kda_status s = conv_sizes(N, T, D, W, dt, act, cu_seqlens, &M);
    if (s != KDA_OK) return s;
    if (N == 0 || D == 0) return KDA_OK;
    const size_t es = esize(dt);
    if (!weight || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(cu_seqlens, 4)) return KDA_ERR_INVALID_ARG;
    if (M > 0 && (!x || !y || x_stride < D)) return KDA_ERR_INVALID_ARG;
    for (const void* t : {x, initial_state, (const void*)y, (const void*)final_state})
        if (!aligned(t, es)) return KDA_ERR_INVALID_ARG;
    const long long le = (long long)es, row = D * le;
    const size_t state = (size_t)N * (W - 1) * D * es, par = (size_t)D * sizeof(float);
    if (clash({{y, M, row, row}, flat_span(final_state, state)},
              {{x, M, x_stride * le, row}, flat_span(initial_state, state), flat_span(weight, W * par), flat_span(bias, par)}))
        return KDA_ERR_INVALID_ARG;
    if (M == 0 && !final_state) return KDA_OK;
    ConvParams p{};
    p.sv = SeqView{cu_seqlens, N, T};
    p.D = D; p.W = W; p.act = (int)act;
    p.x = x; p.x_stride = (size_t)x_stride;
    p.weight = weight; p.bias = bias; p.s0 = initial_state;
    p.y = y; p.sT = final_state;
    const bool vec = vec_ok(dt, D, M > 1 ? x_stride : D, x) && aligned(y, 16) && aligned(initial_state, 16) &&
                     aligned(final_state, 16);
    const int V = vec ? (int)(16 / es) : 1;
    p.cx_log2 = cx_log2_for(D, V, 8);
    // bf16, tiles of 8, 16, 32, 64 tokens: 8192 x 12288 16 on 95, 91, 93 us;
    // x 2304 channels: 32768 tokens 98, 82, 72, 77; 16384 tokens 46, 40, 42, 44;
    // 2048 tokens 12.7, 11.9, 15.7, 23.7; 512 tokens 8.6, 10.7, 16, 27 (fp32 in
    // the same order): long tiles leave a short call few threads
    const long long work = M * (D / V);
    conv_tiles(p, M, work >= (1LL << 23) ? 32 : work >= (1LL << 21) ? 16 : 8);
    const int tys = 256 >> p.cx_log2;
    // blocks of their own pass on the states of sequences without tokens, at
    // most 64 sequences a thread
    const int pass = final_state && (cu_seqlens || T == 0) ? (N + 64 * tys - 1) / (64 * tys) : 0;
    const int blocks = (p.tiles + tys - 1) / tys + pass;
    if (blocks == 0) return KDA_OK;
    if ((long long)blocks * 256 >= 1LL << 32) return KDA_ERR_UNSUPPORTED;
    KDA_LAUNCH("short_conv", launch_conv_fwd((int)dt, vec, p, blocks, stream));
    return KDA_OK;
}

size_t kda_short_conv_bwd_workspace_size(int N, int packed, int T, int D, int W, kda_dtype dt) {
    long long M;
    const int some = 0;
    if (conv_sizes(N, T, D, W, dt, KDA_ACT_NONE, packed ? &some : nullptr, &M) != KDA_OK) return (size_t)-1;
    if (N == 0 || D == 0) return 0;
    // either access width: the narrow one has the fewer channels a block
    const ConvBwdPlan a = conv_bwd_plan(packed != 0, N, T, D, 1), b = conv_bwd_plan(packed != 0, N, T, D, (int)(8 / esize(dt)));
    return (size_t)(a.blocks > b.blocks ? a.blocks : b.blocks) * (W + 1) * D * sizeof(float);
}

kda_status kda_short_conv_bwd(int N, const int* cu_seqlens, int T, int D, int W, kda_dtype dt, kda_activation act,
                              const void* x, long long x_stride, const float* weight, const float* bias,
                              const void* initial_state, const void* d_y, const void* d_final_state, void* dx,
                              float* dweight, float* dbias, void* d_initial_state, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
    long long M;
    kda_status s = conv_sizes(N, T, D, W, dt, act, cu_seqlens, &M);
    if (s != KDA_OK) return s;
    if (D == 0) return KDA_OK;
    const size_t es = esize(dt);
    if (!weight || !dweight) return KDA_ERR_INVALID_ARG;
    for (const void* t : {(const void*)weight, (const void*)bias, (const void*)cu_seqlens, (const void*)dweight,
                          (const void*)dbias})
        if (!aligned(t, 4)) return KDA_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && (!x || !d_y || !dx || x_stride < D)) return KDA_ERR_INVALID_ARG;
    for (const void* t : {x, initial_state, d_y, d_final_state, (const void*)dx, (const void*)d_initial_state})
        if (!aligned(t, es)) return KDA_ERR_INVALID_ARG;
    if (!aligned(workspace, 16)) return KDA_ERR_INVALID_ARG;
    const long long le = (long long)es, row = D * le;
    const size_t state = (size_t)N * (W - 1) * D * es, par = (size_t)D * sizeof(float);
    if (clash({{dx, M, row, row}, flat_span(d_initial_state, state), flat_span(dweight, W * par), flat_span(dbias, par)},
              {{x, M, x_stride * le, row}, {d_y, M, row, row}, flat_span(initial_state, state),
               flat_span(d_final_state, state), flat_span(weight, W * par), flat_span(bias, par)}))
        return KDA_ERR_INVALID_ARG;
    if (N == 0) {
        KDA_LAUNCH("short_conv_bwd_sums", launch_sum_rows(nullptr, 0, W + 1, D, dweight, W, dbias, stream));
        return KDA_OK;
    }
    if (!workspace || workspace_bytes < kda_short_conv_bwd_workspace_size(N, cu_seqlens != nullptr, T, D, W, dt))
        return KDA_ERR_WORKSPACE;
    ConvParams p{};
    p.sv = SeqView{cu_seqlens, N, T};
    p.D = D; p.W = W; p.act = (int)act;
    p.x = x; p.x_stride = (size_t)x_stride;
    p.weight = weight; p.bias = bias; p.s0 = initial_state;
    p.d_y = d_y; p.d_sT = d_final_state; p.dx = dx; p.d_s0 = d_initial_state;
    p.part = reinterpret_cast<float*>(workspace);
    // accesses of eight bytes
    bool vec = vec_ok(dt, D, M > 1 ? x_stride : D, x, 8);
    for (const void* t : {initial_state, d_y, d_final_state, (const void*)dx, (const void*)d_initial_state})
        vec = vec && aligned(t, 8);
    const ConvBwdPlan b = conv_bwd_plan(cu_seqlens != nullptr, N, T, D, vec ? (int)(8 / es) : 1);
    p.cx_log2 = b.cx_log2;
    conv_tiles(p, M, b.tile);
    KDA_LAUNCH("short_conv_bwd", launch_conv_bwd((int)dt, vec, p, b.blocks, stream));
    KDA_LAUNCH("short_conv_bwd_sums", launch_sum_rows(p.part, b.blocks, W + 1, D, dweight, W, dbias, stream));
    return KDA_OK;
}

kda_status kda_short_conv_step(int N, int D, int W, kda_dtype dt, kda_activation act, const void* x,
                               long long x_stride, const float* weight, const float* bias, void* state, void* y,
                               hipStream_t stream) {
    long long M;
    kda_status s = conv_sizes(N, 1, D, W, dt, act, nullptr, &M);
    if (s != KDA_OK) return s;
    if (N == 0 || D == 0) return KDA_OK;
    const size_t es = esize(dt);
    if (!x || !weight || !state || !y || x_stride < D || !aligned(weight, 4) || !aligned(bias, 4)) return KDA_ERR_INVALID_ARG;
    for (const void* t : {x, (const void*)state, (const void*)y})
        if (!aligned(t, es)) return KDA_ERR_INVALID_ARG;
    const long long le = (long long)es, row = D * le;
    const size_t par = (size_t)D * sizeof(float);
    if (clash({{y, N, row, row}, flat_span(state, (size_t)N * (W - 1) * D * es)},
              {{x, N, x_stride * le, row}, flat_span(weight, W * par), flat_span(bias, par)}))
        return KDA_ERR_INVALID_ARG;
    const bool vec = vec_ok(dt, D, N > 1 ? x_stride : D, x) && aligned(state, 16) && aligned(y, 16);
    if ((long long)N * D / (vec ? (long long)(16 / es) : 1) >= (1LL << 32) - 256) return KDA_ERR_UNSUPPORTED;
    KDA_LAUNCH("short_conv_step", launch_conv_step((int)dt, vec, N, D, W, (int)act, x, (size_t)x_stride, weight, bias,
                                                   state, y, stream));
    return KDA_OK;
}

// ---- group norm ------------------------------------------------------------------------

static kda_status norm_check(int rows, int C, int groups, kda_dtype dt, kda_activation act, const void* x,
                             long long x_stride, const float* weight, const float* bias, const void* gate,
                             long long gate_stride, float eps) {
    if (!(eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (rows < 0 || C <= 0 || groups <= 0 || C % groups || !dtype_ok(dt) || !act_ok(act)) return KDA_ERR_INVALID_ARG;
    int R, team, block;
    if (!norm_variant((int)dt, false, C / groups, &R, &team, &block) &&
        !(norm_variant((int)dt, true, C / groups, &R, &team, &block) && (C / groups) % (16 / esize(dt)) == 0))
        return KDA_ERR_UNSUPPORTED;
    if ((long long)rows * groups > 2147483647LL || groups > 65535) return KDA_ERR_UNSUPPORTED;
    if (!aligned(weight, 4) || !aligned(bias, 4) || !aligned(x, esize(dt)) || !aligned(gate, esize(dt)))
        return KDA_ERR_INVALID_ARG;
    if (rows > 0 && (!x || x_stride < C || (gate && gate_stride < C))) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// fills the parameters and the kernel variant
static kda_status norm_setup(int rows, int C, int groups, kda_dtype dt, kda_activation act, int center,
                             int gate_first, float eps, const void* x, long long x_stride, const float* weight,
                             const float* bias, const void* gate, long long gate_stride, bool vec, NormParams* p,
                             int* R, int* block) {
    *p = NormParams{};
    p->rows = rows; p->C = C; p->G = groups; p->Cg = C / groups;
    p->act = (int)act; p->center = center != 0; p->gate_first = gate_first != 0; p->eps = eps;
    p->x = x; p->x_stride = (size_t)x_stride;
    p->z = gate; p->z_stride = (size_t)gate_stride;
    p->weight = weight; p->bias = bias;
    if (!norm_variant((int)dt, vec, p->Cg, R, &p->team, block)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status kda_group_norm_fwd(int rows, int C, int groups, kda_dtype dt, kda_activation act, int center,
                              int gate_first, float eps, const void* x, long long x_stride, const float* weight,
                              const float* bias, const void* gate, long long gate_stride, void* y,
                              hipStream_t stream) {
    kda_status s = norm_check(rows, C, groups, dt, act, x, x_stride, weight, bias, gate, gate_stride, eps);
    if (s != KDA_OK) return s;
    if (rows == 0) return KDA_OK;
    const size_t es = esize(dt);
    if (!y || !aligned(y, es)) return KDA_ERR_INVALID_ARG;
    // every value is read by the team that writes its place: y may be x or the
    // gate exactly, not partly
    const long long le = (long long)es, row = C * le;
    const size_t par = (size_t)C * sizeof(float);
    const bool as_x = x == y && (rows == 1 || x_stride == C), as_z = gate == y && (rows == 1 || gate_stride == C);
    if (clash({{y, rows, row, row}}, {{as_x ? nullptr : x, rows, x_stride * le, row},
                                      {as_z ? nullptr : gate, rows, gate_stride * le, row},
                                      flat_span(weight, par), flat_span(bias, par)}))
        return KDA_ERR_INVALID_ARG;
    bool vec = vec_ok(dt, C / groups, rows > 1 ? x_stride : C, x) && aligned(y, 16);
    if (gate) vec = vec && vec_ok(dt, C / groups, rows > 1 ? gate_stride : C, gate);
    vec = vec && aligned(weight, 16) && aligned(bias, 16);
    NormParams p;
    int R, block;
    s = norm_setup(rows, C, groups, dt, act, center, gate_first, eps, x, x_stride, weight, bias, gate, gate_stride, vec,
                   &p, &R, &block);
    if (s != KDA_OK) return s;
    p.y = y;
    // teams keep to one group each: sixteen waves a CU, or all there is to do
    const long long per = p.team <= 64 ? 256 / p.team : 1, units = (long long)rows * groups;
    long long blocks = (units + per - 1) / per, most = 256LL * 16 * 64 / block;
    const long long least = (groups + per - 1) / per;       // a row slot at least
    if (blocks > most) blocks = most > least ? most : least;
    KDA_LAUNCH("group_norm", launch_norm_fwd((int)dt, vec, R, block, p, (int)blocks, stream));
    return KDA_OK;
}

// Row blocks of the backward: about twelve waves a CU over all groups, each
// block leaving one partial row of parameter sums (8 C bytes, against at least
// 6 C bytes a row of bf16).
static int norm_row_blocks(int rows, int groups, int team, int block) {
    const long long teams = team <= 64 ? 256 / team : 1;
    long long want = (rows + teams - 1) / teams, most = 256LL * 12 * 64 / block / groups;
    if (most < 16) most = 16;
    return (int)(want < most ? (want > 0 ? want : 1) : most);
}

size_t kda_group_norm_bwd_workspace_size(int rows, int C, int groups, kda_dtype dt) {
    if (norm_check(0, C, groups, dt, KDA_ACT_NONE, nullptr, C, nullptr, nullptr, nullptr, C, 0.f) != KDA_OK || rows < 0)
        return (size_t)-1;
    int R, team, block, most = 1;
    for (int vec = 0; vec < 2; ++vec)
        if (norm_variant((int)dt, vec != 0, C / groups, &R, &team, &block)) {
            const int b = norm_row_blocks(rows, groups, team, block);
            most = b > most ? b : most;
        }
    return (size_t)most * 2 * C * sizeof(float);
}

kda_status kda_group_norm_bwd(int rows, int C, int groups, kda_dtype dt, kda_activation act, int center,
                              int gate_first, float eps, const void* x, long long x_stride, const float* weight,
                              const float* bias, const void* gate, long long gate_stride, const void* d_y, void* dx,
                              float* dweight, float* dbias, void* d_gate, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
    kda_status s = norm_check(rows, C, groups, dt, act, x, x_stride, weight, bias, gate, gate_stride, eps);
    if (s != KDA_OK) return s;
    const size_t es = esize(dt);
    for (const void* t : {d_y, (const void*)dx, (const void*)d_gate})
        if (!aligned(t, es)) return KDA_ERR_INVALID_ARG;
    if (!aligned(dweight, 4) || !aligned(dbias, 4) || !aligned(workspace, 16)) return KDA_ERR_INVALID_ARG;
    if (rows > 0 && (!d_y || !dx || (gate != nullptr) != (d_gate != nullptr))) return KDA_ERR_INVALID_ARG;
    const long long le = (long long)es, row = C * le;
    const size_t par = (size_t)C * sizeof(float);
    if (clash({{dx, rows, row, row}, {d_gate, rows, row, row}, flat_span(dweight, par), flat_span(dbias, par)},
              {{x, rows, x_stride * le, row}, {gate, rows, gate_stride * le, row}, {d_y, rows, row, row},
               flat_span(weight, par), flat_span(bias, par)}))
        return KDA_ERR_INVALID_ARG;
    const bool sums = dweight || dbias;
    if (sums && rows > 0 &&
        (!workspace || workspace_bytes < kda_group_norm_bwd_workspace_size(rows, C, groups, dt)))
        return KDA_ERR_WORKSPACE;
    int blocks = 0;
    NormParams p;
    if (rows > 0) {
        bool vec = vec_ok(dt, C / groups, rows > 1 ? x_stride : C, x) && aligned(d_y, 16) && aligned(dx, 16) &&
                   aligned(d_gate, 16);
        if (gate) vec = vec && vec_ok(dt, C / groups, rows > 1 ? gate_stride : C, gate);
        vec = vec && aligned(weight, 16) && aligned(bias, 16);
        int R, block;
        s = norm_setup(rows, C, groups, dt, act, center, gate_first, eps, x, x_stride, weight, bias, gate, gate_stride,
                       vec, &p, &R, &block);
        if (s != KDA_OK) return s;
        p.d_y = d_y; p.dx = dx; p.dz = d_gate;
        p.part = sums ? reinterpret_cast<float*>(workspace) : nullptr;
        blocks = norm_row_blocks(rows, groups, p.team, block);
        KDA_LAUNCH("group_norm_bwd", launch_norm_bwd((int)dt, vec, R, block, p, blocks, stream));
    }
    if (sums)
        KDA_LAUNCH("group_norm_bwd_sums", launch_sum_rows(reinterpret_cast<const float*>(workspace), blocks, 2, C,
                                                          dweight, 1, dbias, stream));
    return KDA_OK;
}

// ---- selective scan ----------------------------------------------------------------------

static kda_status ssm_sizes(int N, const int* cu, int T, int H, int G, int K, int P, kda_dtype dt, long long* M) {
    if (N < 0 || T < 0 || H < 0 || G <= 0 || K <= 0 || P <= 0 || !dtype_ok(dt)) return KDA_ERR_INVALID_ARG;
    if (H % G) return KDA_ERR_INVALID_ARG;
    if (!(K == 64 || K == 128) || !(P == 64 || P == 128)) return KDA_ERR_UNSUPPORTED;
    if (!token_count(cu, N, T, M)) return KDA_ERR_UNSUPPORTED;
    // chunks and workgroups stay within int, and every launch of 256 threads a
    // workgroup (gates: eight heads of a chunk; step: 64 columns of a head)
    // below 2^32 threads
    const long long chunks = *M / 64 + N;
    if (chunks >= 1LL << 24 || (long long)H * K * P > 1LL << 30 || chunks * ((H + 7) / 8) >= 1LL << 24 ||
        (long long)N * H * (P / 64) >= 1LL << 24)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// columns a workgroup: 128 (one head of 128, or two heads of 64 of one group,
// which share B, C and the scores) where the heads pair up
static int ssm_cols(int H, int G, int P) { return P == 128 || (H / G) % 2 == 0 ? 128 : 64; }

// Workgroups of a pass: two a CU, all the output pass has room for (2 x 8K x 16
// heads of 128: 512 workgroups 70 us, 768 84 us, 1024 74 us and a longer
// combine).  The backward's passes run two recurrences in one launch, so each
// takes half, in longer segments.
constexpr int kScanGroups = 512, kScanBwdGroups = 256;

struct SsmPlan {
    int cols, chunks, chunks_per_seq, n_seg, cps;
};
static SsmPlan ssm_plan(bool packed, int N, long long M, int T, int H, int G, int P, int workgroups) {
    SsmPlan pl;
    pl.cols = ssm_cols(H, G, P);
    pl.chunks_per_seq = T > 0 ? (T + 63) / 64 : 1;
    pl.chunks = packed ? (int)(M / 64 + N) : N * pl.chunks_per_seq;
    const long long units = H / (pl.cols / P);
    // Segments until `workgroups` run, each keeping at least four chunks: the
    // summaries and the combine cost as much as the walk they shorten.  In calls
    // short enough for the combine to load at most 32 segments at once, two; one
    // where even that leaves fewer than 128 workgroups.  bf16, K = 128, P = 64,
    // segments of four, two, one chunks: 512 tokens x 8 heads 45, 31, 25 us;
    // 1500 x 8 heads 46, 33, 30; 1024 x 32 heads 48, 40, 45; 256 x 32 heads in
    // one segment 29, in four 26.
    long long want = (workgroups + units - 1) / units, cap = pl.chunks / 4;
    const long long least = pl.chunks >= 4 && pl.chunks * units < 128 ? 1 : pl.chunks >= 8 ? 2 : 4;
    if (cap < 32) cap = pl.chunks / least < 32 ? pl.chunks / least : 32;
    if (want > cap) want = cap;
    if (want < 1 || units >= workgroups / 2) want = 1;
    pl.cps = (int)((pl.chunks + want - 1) / want);
    if (pl.cps < 1) pl.cps = 1;
    pl.n_seg = (pl.chunks + pl.cps - 1) / pl.cps;
    return pl;
}

struct SsmLayout {
    size_t off, gates, seg, dec, total;
};
static SsmLayout ssm_layout(bool packed, int N, int H, int K, int P, const SsmPlan& pl) {
    SsmLayout L;
    size_t o = 0;
    const size_t kp = (size_t)K * P * sizeof(float);
    L.off = o; o += packed ? align256((size_t)(N + 1) * sizeof(int)) : 0;
    L.gates = o; o += align256(ssm_gate_bytes(pl.chunks, H));
    L.seg = o; o += pl.n_seg > 1 ? align256((size_t)pl.n_seg * H * kp) : 0;
    L.dec = o; o += pl.n_seg > 1 ? align256((size_t)pl.n_seg * H * sizeof(float)) : 0;
    L.total = o;
    return L;
}

size_t kda_selective_scan_fwd_workspace_size(int N, int packed, int T, int H, int G, int K, int P, kda_dtype dt) {
    long long M;
    const int some = 0;
    if (ssm_sizes(N, packed ? &some : nullptr, T, H, G, K, P, dt, &M) != KDA_OK) return (size_t)-1;
    if (N == 0 || H == 0) return 0;
    return ssm_layout(packed != 0, N, H, K, P, ssm_plan(packed != 0, N, M, T, H, G, P, kScanGroups)).total;
}

// Elements between token rows in the chunk kernels, whose offsets inside a
// chunk's 64 rows are 32 bits (64 x 2^23 fp32: 2^31 bytes).
constexpr long long kScanStride = 1LL << 23;

// pointer checks shared by the scan's calls; most: the longest row stride
static kda_status ssm_pointers(long long M, int H, int G, int K, int P, kda_dtype dt, const void* x, long long xs,
                               const void* dtp, long long ds, const float* A, const void* B, long long bs, const void* Cm,
                               long long cs, const float* D, const float* dt_bias, const float* s0,
                               long long most = kScanStride) {
    const size_t es = esize(dt);
    if (!A || !aligned(A, 4) || !aligned(D, 4) || !aligned(dt_bias, 4) || !aligned(s0, 16)) return KDA_ERR_INVALID_ARG;
    if (M == 0) return KDA_OK;
    if (!x || !dtp || !B || !Cm || !aligned(dtp, es)) return KDA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(B, 16) || !aligned(Cm, 16)) return KDA_ERR_INVALID_ARG;
    const long long e = 16 / (long long)es;
    if (ds < H || xs < (long long)H * P || bs < (long long)G * K || cs < (long long)G * K || xs % e || bs % e || cs % e)
        return KDA_ERR_INVALID_ARG;
    for (const long long stride : {xs, ds, bs, cs, (long long)H * P})
        if (stride > most) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status kda_selective_scan_fwd(int N, const int* cu_seqlens, int T, int H, int G, int K, int P, kda_dtype dt,
                                  int dt_softplus, const void* x, long long x_stride, const void* delta,
                                  long long delta_stride, const float* A, const void* B, long long b_stride, const void* C,
                                  long long c_stride, const float* D, const float* dt_bias,
                                  const float* initial_state, void* y, float* final_state, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream) {
    long long M;
    kda_status s = ssm_sizes(N, cu_seqlens, T, H, G, K, P, dt, &M);
    if (s != KDA_OK) return s;
    if (N == 0 || H == 0) return KDA_OK;
    s = ssm_pointers(M, H, G, K, P, dt, x, x_stride, delta, delta_stride, A, B, b_stride, C, c_stride, D, dt_bias, initial_state);
    if (s != KDA_OK) return s;
    if (!aligned(cu_seqlens, 4) || !aligned(workspace, 16) || !aligned(final_state, 16) || !aligned(y, 16))
        return KDA_ERR_INVALID_ARG;
    if (M > 0 && !y) return KDA_ERR_INVALID_ARG;
    const size_t state = (size_t)N * H * K * P * sizeof(float), par = (size_t)H * sizeof(float);
    const long long le = (long long)esize(dt), xw = (long long)H * P * le, bw = (long long)G * K * le, dw = H * le;
    if (clash({{y, M, xw, xw}, flat_span(final_state, state)},
              {{x, M, x_stride * le, xw}, {B, M, b_stride * le, bw}, {C, M, c_stride * le, bw}, {delta, M, delta_stride * le, dw},
               flat_span(initial_state == final_state ? nullptr : initial_state, state), flat_span(A, par),
               flat_span(D, par), flat_span(dt_bias, par)}))
        return KDA_ERR_INVALID_ARG;
    const bool packed = cu_seqlens != nullptr;
    const SsmPlan pl = ssm_plan(packed, N, M, T, H, G, P, kScanGroups);
    const SsmLayout L = ssm_layout(packed, N, H, K, P, pl);
    if (L.total > 0 && (!workspace || workspace_bytes < L.total)) return KDA_ERR_WORKSPACE;
    unsigned char* ws = reinterpret_cast<unsigned char*>(workspace);
    SsmParams p{};
    p.sv = SeqView{cu_seqlens, N, T};
    p.H = H; p.G = G; p.K = K; p.P = P; p.softplus = dt_softplus != 0;
    p.x = x; p.x_stride = (size_t)x_stride;
    p.dt = delta; p.dt_stride = (size_t)delta_stride; p.A = A; p.dt_bias = dt_bias; p.Dskip = D;
    p.B = B; p.b_stride = (size_t)b_stride;
    p.C = C; p.c_stride = (size_t)c_stride;
    p.s0 = initial_state;
    p.chunks = pl.chunks; p.chunks_per_seq = pl.chunks_per_seq;
    p.n_seg = pl.n_seg; p.cps = pl.cps;
    if (packed) {
        int* off = reinterpret_cast<int*>(ws + L.off);
        KDA_LAUNCH("scan_prep", launch_ssm_prep(p.sv, off, pl.chunks, stream));
        p.chunk_off = off;
    }
    p.gates = reinterpret_cast<float*>(ws + L.gates);
    KDA_LAUNCH("scan_gates", launch_ssm_gates((int)dt, p, stream));
    if (pl.n_seg > 1) {
        p.in_place = initial_state && initial_state == final_state;
        p.seg_state = reinterpret_cast<float*>(ws + L.seg);
        p.seg_decay = reinterpret_cast<float*>(ws + L.dec);
        const SsmPair a{{p, p}};
        KDA_LAUNCH("scan_summary", launch_ssm_chunks((int)dt, kSsmSummary, pl.cols, a, 1, pl.n_seg - 1, stream));
        KDA_LAUNCH("scan_combine", launch_ssm_combine(a, 1, stream));
    }
    p.y = y;
    p.sT = final_state;
    const SsmPair a{{p, p}};
    KDA_LAUNCH("scan_output", launch_ssm_chunks((int)dt, kSsmOutput, pl.cols, a, 1, pl.n_seg, stream));
    if (p.in_place) KDA_LAUNCH("scan_final", launch_ssm_final(p, stream));
    return KDA_OK;
}

// Workgroups of the gradient kernel: one a (chunk, group, part of the group's
// heads).  One fills a CU's LDS, so they run in rounds of 256; a workgroup costs
// its heads and about one head more for its start (8K x 32 heads: 256
// workgroups of 16 heads 145 us, 512 of eight 154 us, 1024 of four 178 us).
// The parts with the fewest such steps; each beyond the first adds fp32 copies
// of dB and dC, so no more than four rounds' worth of workgroups from parts.
struct SsmBwdLayout {
    size_t off, gates, seg, dec, start, dend, sums, part_b, part_c, total;
    int parts, heads_per;
};
static SsmBwdLayout ssm_bwd_layout(bool packed, int N, long long M, int H, int G, int K, int P, const SsmPlan& pl) {
    SsmBwdLayout L;
    const int hpg = H / G;
    const long long base = (long long)pl.chunks * G;
    L.parts = 1;
    L.heads_per = hpg;
    long long best = -1;
    for (int per = hpg; per > 0; --per) {
        const int parts = (hpg + per - 1) / per;
        if (parts > 1 && base * parts > 1024) break;
        const long long steps = (base * parts + 255) / 256 * (per + 1);
        if (best < 0 || steps < best) {
            best = steps;
            L.parts = parts;
            L.heads_per = per;
        }
    }
    const size_t states = (size_t)pl.chunks * H * K * P * sizeof(float);
    const size_t part = L.parts > 1 ? (size_t)L.parts * M * G * K * sizeof(float) : 0;
    size_t o = 0;
    L.off = o; o += packed ? align256((size_t)(N + 1) * sizeof(int)) : 0;
    L.gates = o; o += align256(ssm_gate_bytes(pl.chunks, H));
    // segments of both recurrences
    L.seg = o; o += pl.n_seg > 1 ? 2 * align256((size_t)pl.n_seg * H * K * P * sizeof(float)) : 0;
    L.dec = o; o += pl.n_seg > 1 ? 2 * align256((size_t)pl.n_seg * H * sizeof(float)) : 0;
    L.start = o; o += align256(states);
    L.dend = o; o += align256(states);
    L.sums = o; o += align256((size_t)pl.chunks * 3 * H * sizeof(float));
    L.part_b = o; o += align256(part);
    L.part_c = o; o += align256(part);
    L.total = o;
    return L;
}

size_t kda_selective_scan_bwd_workspace_size(int N, int packed, int T, int H, int G, int K, int P, kda_dtype dt) {
    long long M;
    const int some = 0;
    if (ssm_sizes(N, packed ? &some : nullptr, T, H, G, K, P, dt, &M) != KDA_OK) return (size_t)-1;
    if (N == 0 || H == 0) return 0;
    return ssm_bwd_layout(packed != 0, N, M, H, G, K, P, ssm_plan(packed != 0, N, M, T, H, G, P, kScanBwdGroups)).total;
}

kda_status kda_selective_scan_bwd(int N, const int* cu_seqlens, int T, int H, int G, int K, int P, kda_dtype dt,
                                  int dt_softplus, const void* x, long long x_stride, const void* delta,
                                  long long delta_stride, const float* A, const void* B, long long b_stride,
                                  const void* C, long long c_stride, const float* D, const float* dt_bias,
                                  const float* initial_state, const void* d_y, const float* d_final_state, void* dx,
                                  long long dx_stride, void* d_delta, float* dA, void* dB, long long db_stride,
                                  void* dC, long long dc_stride, float* dD, float* d_dt_bias,
                                  float* d_initial_state, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream) {
    long long M;
    kda_status s = ssm_sizes(N, cu_seqlens, T, H, G, K, P, dt, &M);
    if (s != KDA_OK) return s;
    if (H == 0) return KDA_OK;
    s = ssm_pointers(M, H, G, K, P, dt, x, x_stride, delta, delta_stride, A, B, b_stride, C, c_stride, D, dt_bias,
                     initial_state);
    if (s != KDA_OK) return s;
    const size_t es = esize(dt), state = (size_t)N * H * K * P * sizeof(float);
    const long long e = 16 / (long long)es;
    for (const void* t : {(const void*)cu_seqlens, (const void*)dA, (const void*)dD, (const void*)d_dt_bias})
        if (!aligned(t, 4)) return KDA_ERR_INVALID_ARG;
    for (const void* t : {d_y, (const void*)d_final_state, (const void*)dx, (const void*)dB, (const void*)dC,
                          (const void*)d_initial_state, (const void*)workspace})
        if (!aligned(t, 16)) return KDA_ERR_INVALID_ARG;
    if (!dA || !aligned(d_delta, es)) return KDA_ERR_INVALID_ARG;
    if (M > 0 && N > 0) {
        if (!d_y || !dx || !d_delta || !dB || !dC) return KDA_ERR_INVALID_ARG;
        if (dx_stride < (long long)H * P || db_stride < (long long)G * K || dc_stride < (long long)G * K ||
            dx_stride % e || db_stride % e || dc_stride % e)
            return KDA_ERR_INVALID_ARG;
        if (dx_stride > kScanStride) return KDA_ERR_UNSUPPORTED;
    }
    const long long le = (long long)es;
    const long long xw = (long long)H * P * le, bw = (long long)G * K * le, dw = H * le;
    const size_t par = (size_t)H * sizeof(float);
    if (clash({{dx, M, dx_stride * le, xw}, {dB, M, db_stride * le, bw}, {dC, M, dc_stride * le, bw}, {d_delta, M, dw, dw},
               flat_span(d_initial_state, state), flat_span(dA, par), flat_span(dD, par), flat_span(d_dt_bias, par)},
              {{x, M, x_stride * le, xw}, {B, M, b_stride * le, bw}, {C, M, c_stride * le, bw}, {delta, M, delta_stride * le, dw},
               {d_y, M, xw, xw}, flat_span(initial_state, state), flat_span(d_final_state, state), flat_span(A, par),
               flat_span(D, par), flat_span(dt_bias, par)}))
        return KDA_ERR_INVALID_ARG;
    if ((M / 64 + N) * G >= 1LL << 23) return KDA_ERR_UNSUPPORTED;
    if (N == 0) {
        KDA_LAUNCH("scan_bwd_sums", launch_ssm_bwd_sums(nullptr, 0, H, dA, d_dt_bias, dD, stream));
        return KDA_OK;
    }
    const bool packed = cu_seqlens != nullptr;
    const SsmPlan pl = ssm_plan(packed, N, M, T, H, G, P, kScanBwdGroups);
    const SsmBwdLayout L = ssm_bwd_layout(packed, N, M, H, G, K, P, pl);
    if (!workspace || workspace_bytes < L.total) return KDA_ERR_WORKSPACE;
    unsigned char* ws = reinterpret_cast<unsigned char*>(workspace);
    SsmParams p{};
    p.sv = SeqView{cu_seqlens, N, T};
    p.H = H; p.G = G; p.K = K; p.P = P; p.softplus = dt_softplus != 0;
    p.x = x; p.x_stride = (size_t)x_stride;
    p.dt = delta; p.dt_stride = (size_t)delta_stride; p.A = A; p.dt_bias = dt_bias; p.Dskip = D;
    p.B = B; p.b_stride = (size_t)b_stride;
    p.C = C; p.c_stride = (size_t)c_stride;
    p.s0 = initial_state;
    p.chunks = pl.chunks; p.chunks_per_seq = pl.chunks_per_seq;
    p.n_seg = pl.n_seg; p.cps = pl.cps;
    if (packed) {
        int* off = reinterpret_cast<int*>(ws + L.off);
        KDA_LAUNCH("scan_prep", launch_ssm_prep(p.sv, off, pl.chunks, stream));
        p.chunk_off = off;
    }
    p.gates = reinterpret_cast<float*>(ws + L.gates);
    KDA_LAUNCH("scan_gates", launch_ssm_gates((int)dt, p, stream));
    // the state before each chunk, and the adjoint behind it: the same
    // recurrence backwards, with C for B and dy for x
    p.states = reinterpret_cast<float*>(ws + L.start);
    SsmParams q = p;
    q.reverse = 1;
    q.x = d_y; q.x_stride = (size_t)H * P;
    q.B = C; q.b_stride = (size_t)c_stride;
    q.s0 = d_final_state;
    q.sT = d_initial_state;
    q.states = reinterpret_cast<float*>(ws + L.dend);
    SsmPair a{{p, q}};
    if (pl.n_seg > 1) {
        for (int i = 0; i < 2; ++i) {
            a.p[i].seg_state = reinterpret_cast<float*>(ws + L.seg + i * align256((size_t)pl.n_seg * H * K * P * sizeof(float)));
            a.p[i].seg_decay = reinterpret_cast<float*>(ws + L.dec + i * align256((size_t)pl.n_seg * H * sizeof(float)));
        }
        // the last segment's end is read by nobody: the first's, backwards
        a.p[1].seg0 = 1;
        KDA_LAUNCH("scan_bwd_summary", launch_ssm_chunks((int)dt, kSsmSummary, pl.cols, a, 2, pl.n_seg - 1, stream));
        KDA_LAUNCH("scan_bwd_combine", launch_ssm_combine(a, 2, stream));
        a.p[1].seg0 = 0;
    }
    KDA_LAUNCH("scan_bwd_states", launch_ssm_chunks((int)dt, kSsmStates, pl.cols, a, 2, pl.n_seg, stream));
    SsmBwdParams b{};
    b.f = p;
    b.d_y = d_y;
    b.start = p.states;
    b.dend = q.states;
    b.dx = dx; b.dx_stride = (size_t)dx_stride;
    b.ddt = d_delta;
    b.dB = dB; b.db_stride = (size_t)db_stride;
    b.dC = dC; b.dc_stride = (size_t)dc_stride;
    b.dB_part = reinterpret_cast<float*>(ws + L.part_b);
    b.dC_part = reinterpret_cast<float*>(ws + L.part_c);
    b.sums = reinterpret_cast<float*>(ws + L.sums);
    b.parts = L.parts; b.heads_per = L.heads_per;
    KDA_LAUNCH("scan_bwd_grads", launch_ssm_bwd((int)dt, b, stream));
    if (L.parts > 1) KDA_LAUNCH("scan_bwd_join", launch_ssm_bwd_join((int)dt, b, M, stream));
    KDA_LAUNCH("scan_bwd_sums", launch_ssm_bwd_sums(b.sums, pl.chunks, H, dA, d_dt_bias, dD, stream));
    return KDA_OK;
}

kda_status kda_selective_scan_step(int N, int H, int G, int K, int P, kda_dtype dt, int dt_softplus, const void* x,
                                   long long x_stride, const void* delta, long long delta_stride, const float* A,
                                   const void* B,
                                   long long b_stride, const void* C, long long c_stride, const float* D,
                                   const float* dt_bias, float* state, void* y, hipStream_t stream) {
    long long M;
    kda_status s = ssm_sizes(N, nullptr, 1, H, G, K, P, dt, &M);
    if (s != KDA_OK) return s;
    if (N == 0 || H == 0) return KDA_OK;
    // the step addresses its rows in 64 bits: any stride whose rows (fewer than
    // 2^24) span less than 2^63 bytes
    s = ssm_pointers(M, H, G, K, P, dt, x, x_stride, delta, delta_stride, A, B, b_stride, C, c_stride, D, dt_bias, state,
                     1LL << 37);
    if (s != KDA_OK) return s;
    if (!state || !y || !aligned(y, 16)) return KDA_ERR_INVALID_ARG;
    const size_t par = (size_t)H * sizeof(float);
    const long long le = (long long)esize(dt), xw = (long long)H * P * le, bw = (long long)G * K * le, dw = H * le;
    if (clash({{y, N, xw, xw}, flat_span(state, (size_t)N * H * K * P * sizeof(float))},
              {{x, N, x_stride * le, xw}, {B, N, b_stride * le, bw}, {C, N, c_stride * le, bw}, {delta, N, delta_stride * le, dw},
               flat_span(A, par), flat_span(D, par), flat_span(dt_bias, par)}))
        return KDA_ERR_INVALID_ARG;
    KDA_LAUNCH("scan_step", launch_ssm_step((int)dt, N, H, G, K, P, dt_softplus != 0, x, (size_t)x_stride, delta, (size_t)delta_stride, A, B,
                                            (size_t)b_stride, C, (size_t)c_stride, D, dt_bias, state, y, stream));
    return KDA_OK;
}

}  // extern "C"
