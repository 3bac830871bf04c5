// C ABI of the paged cache operators: argument validation, launch plans,
// launches.  The declarations and their contracts are in include/kda.h.
#include "kda.h"
#include "kda_host.h"
#include "kda_internal.h"
#include "kda_paged.h"

#include <algorithm>

using namespace kda;

namespace {

int kv_size(kda_kv_dtype dt) { return dt == KDA_KV_F32 ? 4 : dt == KDA_KV_BF16 ? 2 : 1; }
bool coded(kda_kv_dtype dt) { return dt == KDA_KV_E4M3 || dt == KDA_KV_I8; }

// sizes and types of a call (no pointers)
kda_status cache_sizes(int N, const int* cu, int T, kda_dtype dt, const kda_paged_cache* c, long long* M) {
    if (!c || N < 0 || T < 0 || !dtype_ok(dt)) return KDA_ERR_INVALID_ARG;
    if (c->dt < KDA_KV_F32 || c->dt > KDA_KV_I8 || c->pages < 0 || c->heads <= 0 || c->blocks < 0)
        return KDA_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return KDA_ERR_UNSUPPORTED;
    const int ps = c->page_size;
    if (ps < 16 || ps > 256 || (ps & (ps - 1))) return KDA_ERR_UNSUPPORTED;
    if ((long long)c->blocks * ps > 1LL << 30 || c->heads > 65535) return KDA_ERR_UNSUPPORTED;
    if (!coded(c->dt) && (int)c->dt != (int)dt) return KDA_ERR_UNSUPPORTED;
    if (!token_count(cu, N, T, M)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

long long page_width(const kda_paged_cache* c) { return (long long)c->heads * c->page_size * c->head_dim; }

// `rows` rows of 4-byte elements `stride` apart stay within 62 bits of bytes
bool spans(long long rows, long long stride) { return rows <= 1 || (stride <= 1LL << 40 && stride <= (1LL << 60) / rows); }

kda_status cache_pointers(int N, const int* cu, const kda_paged_cache* c) {
    const int es = kv_size(c->dt);
    if (!aligned(cu, 4)) return KDA_ERR_INVALID_ARG;
    if (c->pages > 0) {
        if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return KDA_ERR_INVALID_ARG;
        if (c->pages > 1)
            for (long long st : {c->k_page_stride, c->v_page_stride}) {
                if (st < page_width(c) || st % (16 / es)) return KDA_ERR_INVALID_ARG;
                if (!spans(c->pages, st)) return KDA_ERR_UNSUPPORTED;
            }
        if (coded(c->dt) && (!c->k_scale || !c->v_scale)) return KDA_ERR_INVALID_ARG;
    }
    if (!coded(c->dt) && (c->k_scale || c->v_scale)) return KDA_ERR_INVALID_ARG;
    if (!aligned(c->k_scale, 16) || !aligned(c->v_scale, 16)) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (!c->seq_lens || !aligned(c->seq_lens, 4))) return KDA_ERR_INVALID_ARG;
    if (N > 0 && c->blocks > 0 && (!c->block_table || !aligned(c->block_table, 4))) return KDA_ERR_INVALID_ARG;
    if (N > 1 && c->block_table_stride < c->blocks) return KDA_ERR_INVALID_ARG;
    if (!spans(N, c->block_table_stride)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

PagedCache view_of(const kda_paged_cache* c) {
    PagedCache v{};
    const size_t es = (size_t)kv_size(c->dt);
    v.k = (char*)c->k; v.v = (char*)c->v;
    v.ks = c->k_scale; v.vs = c->v_scale;
    v.k_page = (c->pages > 1 ? (size_t)c->k_page_stride : 0) * es;
    v.v_page = (c->pages > 1 ? (size_t)c->v_page_stride : 0) * es;
    v.table = c->block_table; v.table_stride = c->block_table_stride;
    v.lens = c->seq_lens;
    v.pages = c->pages; v.blocks = c->blocks; v.Hk = c->heads;
    while ((1 << v.lg_page) < c->page_size) ++v.lg_page;
    return v;
}

// the bytes of the cache's tensors
Span pages_span(const kda_paged_cache* c, const void* p, long long stride) {
    const long long es = kv_size(c->dt), w = page_width(c) * es;
    return Span{p, c->pages, c->pages > 1 ? stride * es : w, w};
}
Span scale_span(const kda_paged_cache* c, const void* p) {
    return flat_span(p, (size_t)c->pages * c->heads * c->page_size);
}
Span table_span(int N, const kda_paged_cache* c) {
    return Span{c->block_table, N, (N > 1 ? c->block_table_stride : c->blocks) * 4LL, c->blocks * 4LL};
}
// token rows that an access of 16 bytes a lane takes
bool rows_ok(const void* p, long long M, long long width, long long stride, kda_dtype dt) {
    return p && aligned(p, 16) && (M <= 1 || (stride >= width && stride % (long long)(16 / esize(dt)) == 0));
}

// Heads of a block: all of them where the tokens fill the card (the table is
// looked up once for a block), else fewer.
int io_heads(long long token_blocks, int heads) {
    int n = heads;
    while (n > 1 && token_blocks * ((heads + n - 1) / n) < 2048) n = (n + 1) / 2;
    return n;
}

kda_status cache_io(bool write, int N, const int* cu, int T, kda_dtype dt, void* k, long long k_stride, void* v,
                    long long v_stride, const kda_paged_cache* c, hipStream_t stream) {
    long long M;
    kda_status s = cache_sizes(N, cu, T, dt, c, &M);
    if (s != KDA_OK) return s;
    if (N == 0 || M == 0) return KDA_OK;
    s = cache_pointers(N, cu, c);
    if (s != KDA_OK) return s;
    const long long width = (long long)c->heads * c->head_dim, es = (long long)esize(dt);
    if (!rows_ok(k, M, width, k_stride, dt) || !rows_ok(v, M, width, v_stride, dt)) return KDA_ERR_INVALID_ARG;
    if (!spans(M, k_stride) || !spans(M, v_stride)) return KDA_ERR_UNSUPPORTED;
    const Span sk{k, M, k_stride * es, width * es}, sv{v, M, v_stride * es, width * es};
    const Span ck = pages_span(c, c->k, c->k_page_stride), cv = pages_span(c, c->v, c->v_page_stride);
    const Span ks = scale_span(c, c->k_scale), vs = scale_span(c, c->v_scale);
    const Span tab = table_span(N, c), len = flat_span(c->seq_lens, (size_t)N * 4);
    const Span off = flat_span(cu, (size_t)(N + 1) * 4);
    if (write ? clash({ck, cv, ks, vs}, {sk, sv, tab, len, off}) : clash({sk, sv}, {ck, cv, ks, vs, tab, len, off}))
        return KDA_ERR_INVALID_ARG;
    CacheIoParams p{};
    p.sv = SeqView{cu, N, T};
    p.c = view_of(c);
    p.k = (char*)k; p.v = (char*)v;
    p.k_stride = (size_t)(k_stride * es); p.v_stride = (size_t)(v_stride * es);
    p.M = (int)M;
    const long long tb = (M + 15) / 16;
    p.heads_per_block = io_heads(tb, c->heads);
    const int hb = (c->heads + p.heads_per_block - 1) / p.heads_per_block;
    if (tb * hb * 256 >= 1LL << 32) return KDA_ERR_UNSUPPORTED;
    if (write)
        KDA_LAUNCH("cache_write", launch_cache_write((int)dt, (int)c->dt, c->head_dim, p, (int)tb, hb, stream));
    else
        KDA_LAUNCH("cache_read", launch_cache_read((int)dt, (int)c->dt, c->head_dim, p, (int)tb, hb, stream));
    return KDA_OK;
}

struct AttnPlan {
    AttnKind kind;
    int M, splits, split_len;
    long long tiles;
    int tiles_per_seq;
    size_t part, bytes;     // of the parts, of the workspace
};
// The plan goes by sizes alone, so that a call's plan is its workspace's.
AttnPlan attn_plan(int N, bool packed, int T, int H, kda_dtype dt, const kda_paged_cache* c) {
    AttnPlan a{};
    const long long G = H / c->heads, M = packed ? (long long)T : (long long)N * T;
    const long long per = N > 0 ? M * G / N : 0;        // rows of a sequence, on average
    // Few rows go to the kernel that splits positions over its waves, 16 or 32
    // rows a workgroup, more to the one that splits rows.  64 sequences of up to
    // 8K x 8 heads of 128, 16 / 32 / chunk, bf16: 16 rows 199, 196, 258 us; 32 rows
    // 233, 205, 262; 64 rows 340, 247, 270 (4 sequences: 42, 37, 33); 128 rows 609,
    // 361, 285.  e4m3: 16 rows 122, 126, 250; 64 rows 243, 192, 260 (39, 35, 35); 128
    // rows 434, 316, 278.
    a.kind = dt == KDA_F32 ? kAttnF32 : per <= 16 ? kAttnStep16 : per <= (coded(c->dt) ? 64 : 32) ? kAttnStep32 : kAttnChunk;
    // Rows of a chunk's workgroup, 128 or 256.  Heads of 128, eight waves of 32:
    // half the reads of the cache (4 x 2K over 32K in e4m3 3.9 and 4.2 ms, a 4K
    // prompt 143 and 152 us), but there have to be enough of them for the card (2K
    // prompt 63 and 52 us, 8 x 300 over 3K 81 and 66) and sequences that fill them
    // (64 x up to 200 over 4K 341 and 325).  Heads of 64, four waves of 64: a code
    // is turned into bf16 half as often and V is read from LDS half as often (4 x
    // 2K over 32K 1.11 and 1.18 ms, in int8 1.25 and 1.43; 512 over 64K in int8 338
    // and 408 us), but with two waves a SIMD instead of three, which pays where a
    // workgroup walks some thousand positions (512 over 32K in int8 178 and 211 us,
    // over 8K 58 and 55, a 4K prompt 106 and 95, 2K 53 and 39).  Sequences of a batch
    // are taken for half as long as their table is wide, and have to fill several
    // tiles (packed, 32 heads over 8, 6 up to 600 over up to 16K 344 and 166, 8 up to
    // 777 353 and 320; 4 x 2K over 32K, 12 over 3, in int8 958 and 1047).
    if (a.kind == kAttnChunk && per >= 1024) {
        const long long units = M * G / 256 * c->heads, at_a_time = units < 512 ? units : 512;
        const long long before = (long long)c->blocks * c->page_size / (N > 1 ? 2 : 1) - M / N / 2;
        if (c->head_dim == 128 ? units >= 512 : (N == 1 || per >= 4096) && before * at_a_time >= 512 * 3800) a.kind = kAttnChunk256;
    }
    a.M = a.kind == kAttnStep16 ? 16 : a.kind == kAttnChunk ? 128 : a.kind == kAttnChunk256 ? 256 : 32;
    const bool step = a.kind == kAttnStep16 || a.kind == kAttnStep32;
    a.tiles_per_seq = packed ? 0 : (int)((T * G + a.M - 1) / a.M);
    a.tiles = packed ? M * G / a.M + N : (long long)N * a.tiles_per_seq;
    const long long units = a.tiles * c->heads, ctx = (long long)c->blocks * c->page_size;
    // Ranges: as many as the card takes at a time where tiles alone are fewer
    // (chunks of 128 rows, two workgroups a CU: 512 tokens over 8K with 256, 512,
    // 1024 wanted 88, 82, 94 us, 2K over 2K 52, 52, 71; a 1M step with 64, 192, 384
    // ranges a head 376, 387, 398), three times that for the lengths of a batch of
    // single tokens, which differ (64 sequences x 8 heads with 3, 6, 12: 228, 230,
    // 234); many of them are split in three all the same (256 x 8 heads: 771 -> 743
    // us), up to 12288 ranges, whose parts are 200 MB at most.  At least 512
    // positions, 1024 in chunks: below that the join's launch costs more than the
    // ranges save (a 1K prompt in two 34 us, in one 27).
    // Chunks of a batch differ in length too, and its longest would end alone: up to
    // four times as many where that splits a tile in three or more (12 heads of 128
    // over 3, 4 x 777 over up to 32K 527 -> 294 us, in int8 776 -> 359; 3 packed up
    // to 1500, 32 heads over 8, 1172 -> 1030; equal lengths that fill the card as they
    // are, 2 x 1K over 16K, 488 -> 529), at least 2048 positions each.  In two costs
    // the join for little (8 packed up to 777 over up to 16K 491 and 583).  Of 256 rows
    // (4 x 2K over 32K, 12 heads of 64 over 3, in int8) 512, 1024: 1205, 958 us.
    auto length = [&](long long n) { return n > 1 ? ((ctx + n - 1) / n + 127) / 128 * 128 : (ctx + 127) / 128 * 128; };
    const bool joined = M * H < 1LL << 23 && units > 0, batch = joined && N > 1;
    const long long want = step && N > 1 ? 1536 : a.kind == kAttnChunk256 && N > 1 && units < 512 ? 1024 : 512;
    long long n = joined ? want / units : 1;
    if (batch && step && n < 3 && 3 * units <= 12288) n = 3;
    long long len = std::max(length(n), step || a.kind == kAttnF32 ? 512LL : 1024LL);
    if (batch && a.kind == kAttnChunk && 2048 / units >= 3) len = std::min(len, std::max(length(2048 / units), 2048LL));
    a.split_len = (int)len;
    a.splits = ctx > 0 ? (int)((ctx + len - 1) / len) : 1;
    if (a.splits > 1) {
        const size_t rows = (size_t)units * a.splits * a.M;
        a.part = align256(rows * c->head_dim * sizeof(float));
        a.bytes = a.part + rows * 2 * sizeof(float);
    }
    return a;
}

kda_status attn_sizes(int N, const int* cu, int T, int H, kda_dtype dt, const kda_paged_cache* c, long long* M) {
    kda_status s = cache_sizes(N, cu, T, dt, c, M);
    if (s != KDA_OK) return s;
    if (H <= 0 || H % c->heads) return KDA_ERR_INVALID_ARG;
    if (H > 65535 || *M * (H / c->heads) > 2147483647LL - 4096) return KDA_ERR_UNSUPPORTED;
    if (N == 0) return KDA_OK;
    const AttnPlan a = attn_plan(N, cu != nullptr, T, H, dt, c);
    if (a.tiles > 2147483647LL || a.tiles * a.splits * c->heads * 512 >= 1LL << 32) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_kv_cache_write(int N, const int* cu_seqlens, int T, kda_dtype dt, const void* k, long long k_stride,
                              const void* v, long long v_stride, const kda_paged_cache* cache, hipStream_t stream) {
    return cache_io(true, N, cu_seqlens, T, dt, const_cast<void*>(k), k_stride, const_cast<void*>(v), v_stride, cache,
                    stream);
}

kda_status kda_kv_cache_read(int N, const int* cu_seqlens, int T, kda_dtype dt, void* k, void* v,
                             const kda_paged_cache* cache, hipStream_t stream) {
    const long long row = cache ? (long long)cache->heads * cache->head_dim : 0;
    return cache_io(false, N, cu_seqlens, T, dt, k, row, v, row, cache, stream);
}

size_t kda_paged_attn_workspace_size(int N, int packed, int T, int H, kda_dtype dt, const kda_paged_cache* cache) {
    long long M;
    const int some = 0;
    if (attn_sizes(N, packed ? &some : nullptr, T, H, dt, cache, &M) != KDA_OK) return (size_t)-1;
    return N == 0 || M == 0 ? 0 : attn_plan(N, packed != 0, T, H, dt, cache).bytes;
}

kda_status kda_paged_attn(int N, const int* cu_seqlens, int T, int H, kda_dtype dt, float scale, const void* q,
                          long long q_stride, const void* gate, long long gate_stride, void* o,
                          const kda_paged_cache* cache, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    long long M;
    kda_status s = attn_sizes(N, cu_seqlens, T, H, dt, cache, &M);
    if (s != KDA_OK) return s;
    const float c_log2 = scale * 1.4426950408889634f;
    if (!(scale > 0.f) || !(c_log2 <= 3.4028234e38f)) return KDA_ERR_INVALID_ARG;
    if (N == 0 || M == 0) return KDA_OK;
    s = cache_pointers(N, cu_seqlens, cache);
    if (s != KDA_OK) return s;
    const kda_paged_cache* c = cache;
    const long long width = (long long)H * c->head_dim, es = (long long)esize(dt);
    if (!rows_ok(q, M, width, q_stride, dt) || (gate && !rows_ok(gate, M, width, gate_stride, dt)) || !o ||
        !aligned(o, 16) || !aligned(workspace, 16))
        return KDA_ERR_INVALID_ARG;
    if (!spans(M, q_stride) || (gate && !spans(M, gate_stride))) return KDA_ERR_UNSUPPORTED;
    const AttnPlan a = attn_plan(N, cu_seqlens != nullptr, T, H, dt, c);
    const Span so{o, M, width * es, width * es}, sq{q, M, q_stride * es, width * es};
    const Span sz{gate, M, gate_stride * es, width * es};
    if (clash({so, flat_span(workspace, a.bytes)},
              {sq, sz, pages_span(c, c->k, c->k_page_stride), pages_span(c, c->v, c->v_page_stride),
               scale_span(c, c->k_scale), scale_span(c, c->v_scale), table_span(N, c),
               flat_span(c->seq_lens, (size_t)N * 4), flat_span(cu_seqlens, (size_t)(N + 1) * 4)}))
        return KDA_ERR_INVALID_ARG;
    if (a.bytes && (!workspace || workspace_bytes < a.bytes)) return KDA_ERR_WORKSPACE;
    AttnParams p{};
    p.sv = SeqView{cu_seqlens, N, T};
    p.c = view_of(c);
    p.q = (const char*)q; p.q_stride = (size_t)(q_stride * es);
    p.z = (const char*)gate; p.z_stride = (size_t)(gate_stride * es);
    p.o = (char*)o;
    p.H = H; p.G = H / c->heads;
    p.c_log2 = c_log2;
    p.M = a.M; p.tiles = (int)a.tiles; p.tiles_per_seq = a.tiles_per_seq;
    p.splits = a.splits; p.split_len = a.split_len;
    while ((1 << p.lg_m) < p.M) ++p.lg_m;
    p.by_g.set((unsigned)p.G);
    p.by_hk.set((unsigned)c->heads);
    p.by_splits.set((unsigned)p.splits);
    p.by_tiles.set((unsigned)(p.tiles_per_seq > 0 ? p.tiles_per_seq : 1));
    p.by_len.set((unsigned)p.split_len);
    p.by_h.set((unsigned)H);
    p.by_t.set((unsigned)(T > 0 ? T : 1));
    // Workgroups of chunks bound by their products end together if long tiles
    // come first (48 sequences over int8 216 -> 166 us, 16 in fp32 136 -> 116); a lane a sequence finds the
    // order, and with more sequences than lanes chance does what is needed.
    p.by_length = (a.kind == kAttnChunk || a.kind == kAttnChunk256 || a.kind == kAttnF32) && N > 1 && N <= 64;
    p.part = (float*)workspace;
    p.ml = (float*)((char*)workspace + a.part);
    const char* name = a.kind == kAttnF32 ? "attn_f32" : a.kind == kAttnChunk || a.kind == kAttnChunk256 ? "attn_chunk" : "attn_step";
    KDA_LAUNCH(name, launch_attn(a.kind, (int)c->dt, c->head_dim, p, stream));
    if (a.splits > 1) KDA_LAUNCH("attn_join", launch_attn_join((int)dt, c->head_dim, p, (int)M, stream));
    return KDA_OK;
}

}  // extern "C"
