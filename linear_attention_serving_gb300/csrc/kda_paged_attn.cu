// kda_paged_attn.cu -- kda_paged_attn: argument checks, workspace layout and
// the launches of paged attention.
#include <cmath>
#include <cstring>

#include "kda_paged.cuh"

namespace kda {
namespace {

// ---------------------------------------------------------------- workspace
// [leads][slots] of the kernel for few rows (or fp32), then of the tile kernel: per
// block one lead (two int4) and two slots
struct PagedSet {
    size_t off_lead, off_slots;
    int blocks, slot_rows;
};
struct PagedWs {
    PagedSet rows, tile;
    int parts;  // of a tile block's work
    size_t total;
};

PagedSet paged_set(size_t &off, int blocks, int64_t rows, int cap) {
    PagedSet p;
    p.blocks = blocks;
    p.slot_rows = rows >= cap ? cap : rows < 16 ? 16 : (int)((rows + 15) / 16 * 16);
    p.off_lead = off;
    off = align_up(off + (size_t)blocks * 2 * sizeof(int4), 256);
    p.off_slots = off;
    off = align_up(off + (size_t)blocks * 2 * paged_slot_floats(p.slot_rows) * sizeof(float), 256);
    return p;
}

PagedWs paged_ws(int64_t T, int Hq, int Hkv) {
    PagedWs w;
    const int64_t rows = T * (Hq / Hkv);
    w.total = 0;
    w.rows = paged_set(w.total, paged_rows_blocks(), rows, PAGED_ROWS_CAP);  // (the most blocks of the two)
    // (a call of fewer rows has not the work that makes parts pay)
    w.parts = rows >= 2048 ? 4 : 1;
    w.tile = paged_set(w.total, paged_tile_blocks() * w.parts, rows, PAGED_TILE_CAP);
    return w;
}

// ---------------------------------------------------------------- join
// Merges the pieces of the items that block borders cut.  Blocks (c, y), all y,
// take the item whose first piece the attention's block c left.  Few pieces: a
// warp to a row.  Many: a block to a row, its warps taking every eighth piece
// and meeting in shared memory.  Pieces are taken in block order either way.
constexpr int JOIN_WARPS = 8;
constexpr int JOIN_FEW = 12;

struct JoinSet {
    const int4 *lead;
    float *parts;
    int blocks, slot_rows;
};

__global__ void __launch_bounds__(JOIN_WARPS * 32) paged_join_kernel(PagedAttn a, const JoinSet s0, const JoinSet s1, int f32) {
    __shared__ float4 acc_s[JOIN_WARPS][32];
    __shared__ float2 ml_s[JOIN_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const JoinSet &js = (int)blockIdx.x < s0.blocks ? s0 : s1;
    const int c = (int)blockIdx.x < s0.blocks ? blockIdx.x : blockIdx.x - s0.blocks;
    const int4 y = js.lead[2 * c + 1], x = js.lead[2 * c];
    if (!y.w) return;
    a.parts = js.parts;
    a.slot_rows = js.slot_rows;
    const int h = x.y, r0 = x.z, R = x.w, c0 = y.y, np = y.z - y.y + 1;
    const float vs = a.v_scale ? a.v_scale[h] : 1.f;
    const bool few = np <= JOIN_FEW;
    auto slot = [&](int p) { return paged_slot(a, p == 0 ? y.x : 2 * (c0 + p)); };
    const int step = few ? 1 : JOIN_WARPS, p0 = few ? 0 : warp;
    for (int r = few ? blockIdx.y * JOIN_WARPS + warp : blockIdx.y; r < R; r += gridDim.y * (few ? JOIN_WARPS : 1)) {
        float M = -INFINITY, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        // four pieces at a time, all their loads in flight at once
        for (int p = p0; p < np; p += 4 * step) {
            float2 ml[4];
            float4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool have = p + i * step < np;
                const float *sp = slot(have ? p + i * step : p);
                ml[i] = reinterpret_cast<const float2 *>(sp)[r];
                v[i] = reinterpret_cast<const float4 *>(sp + 2 * a.slot_rows)[r * (D / 4) + lane];
                if (!have) ml[i] = make_float2(-INFINITY, 0.f);
            }
            const float m = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M);
            const float ref = m == -INFINITY ? 0.f : m, f0 = tc::ex2(M - ref);
            L *= f0;
            acc.x *= f0;
            acc.y *= f0;
            acc.z *= f0;
            acc.w *= f0;
            M = m;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // what an empty piece holds has no say; one whose scores are all NaN has no maximum
                // either, but a NaN for its sum
                if (ml[i].y == 0.f) continue;
                const float f = tc::ex2(ml[i].x - ref);
                L += f * ml[i].y;
                acc.x += f * v[i].x;
                acc.y += f * v[i].y;
                acc.z += f * v[i].z;
                acc.w += f * v[i].w;
            }
        }
        if (!few) {
            acc_s[warp][lane] = acc;
            if (lane == 0) ml_s[warp] = make_float2(M, L);
            __syncthreads();
            if (warp == 0) {
                M = -INFINITY;
#pragma unroll
                for (int w = 0; w < JOIN_WARPS; ++w) M = fmaxf(M, ml_s[w].x);
                const float rf = M == -INFINITY ? 0.f : M;
                acc = make_float4(0.f, 0.f, 0.f, 0.f);
                L = 0.f;
#pragma unroll
                for (int w = 0; w < JOIN_WARPS; ++w) {
                    const float f = tc::ex2(ml_s[w].x - rf);
                    const float4 v = acc_s[w][lane];
                    L += f * ml_s[w].y;
                    acc.x += f * v.x;
                    acc.y += f * v.y;
                    acc.z += f * v.z;
                    acc.w += f * v.w;
                }
            }
        }
        if (few || warp == 0) {
            const int rr = r0 + r, j = rr / a.G;
            paged_store_row(a, f32, x.x + j, h * a.G + (rr - j * a.G), lane, acc, M, L, vs);
        }
        if (!few) __syncthreads();
    }
}

constexpr int FEW_ROWS = 16;

int launch_join(const PagedAttn &a, const JoinSet &s0, const JoinSet &s1, int64_t max_rows, bool f32, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(s0.blocks + s1.blocks, (unsigned)(max_rows < 16 ? max_rows : 16));
    cfg.blockDim = dim3(JOIN_WARPS * 32);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_join_kernel, a, s0, s1, (int)f32);
    note_launch("paged_join", s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_paged_attn_workspace_size(int64_t T_total, int n_seqs, int Hq, int Hkv) {
    if (T_total < 0 || n_seqs < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv) return 0;
    return paged_ws(T_total, Hq, Hkv).total;
}

int kda_paged_attn(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_table,
                   const int32_t *cu_q, const int32_t *kv_len, int n_seqs, int64_t T_total, int max_q, int Hq,
                   int Hkv, int Dm, int dtype, int cache_dtype, const float *k_scale, const float *v_scale,
                   int n_pages, int page_size, int64_t page_stride, int max_blocks, float sm_scale, int window,
                   void *o, float *lse, void *workspace, size_t workspace_bytes, int32_t *error_word,
                   kda_stream_t stream) {
    int rc = check_paged_cache(Hkv, Dm, dtype, cache_dtype, k_scale, v_scale, k_cache, v_cache, n_pages, page_size,
                               page_stride);
    if (rc) return rc;
    if (Hq < Hkv || Hq % Hkv || n_seqs < 1 || max_blocks < 1 || max_q < 0 || window < 0) return KDA_ERR_INVALID_ARG;
    if (T_total < 0 || T_total * (Hq / Hkv) >= (int64_t)INT32_MAX / 2) return KDA_ERR_INVALID_ARG;
    // key positions are int32, with room for a tile past the end
    if ((int64_t)max_blocks * page_size > (int64_t)INT32_MAX - 65536) return KDA_ERR_INVALID_ARG;
    if (!(sm_scale > 0.0f) || sm_scale > 1e30f) return KDA_ERR_INVALID_ARG;
    if (!block_table || !cu_q || !kv_len) return KDA_ERR_INVALID_ARG;
    if (T_total > 0 && (!q || !o)) return KDA_ERR_INVALID_ARG;
    if (((uintptr_t)q & 15u) || ((uintptr_t)o & 15u)) return KDA_ERR_INVALID_ARG;
    const PagedWs w = paged_ws(T_total, Hq, Hkv);
    if (!workspace || workspace_bytes < w.total || ((uintptr_t)workspace & 255u)) return KDA_ERR_WORKSPACE;
    if (T_total == 0) return KDA_OK;
    cudaStream_t s = (cudaStream_t)stream;
    note_begin(s);
    PagedAttn a;
    memset(&a, 0, sizeof(a));
    a.q = q;
    a.o = o;
    a.lse = lse;
    a.table = block_table;
    a.cu = cu_q;
    a.kv = kv_len;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.err = error_word;
    a.n_seqs = n_seqs;
    a.T = (int)T_total;
    a.max_q = max_q == 0 || max_q > T_total ? (int)T_total : max_q;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.page_size = page_size;
    a.n_pages = n_pages;
    a.max_blocks = max_blocks;
    // (no position is further back than the table reaches: such a window is none, and what is left
    // stays clear of 2^31 where positions are added to it)
    a.window = window >= (int64_t)max_blocks * page_size ? 0 : window;
    a.scale_log2 = sm_scale * 1.4426950408889634f;
    a.wait_budget = wait_budget();
    char *ws = (char *)workspace;
    const int64_t max_rows = (int64_t)a.max_q * a.G;
    JoinSet js[2] = {{nullptr, nullptr, 0, 1}, {nullptr, nullptr, 0, 1}};
    auto use = [&](const PagedSet &p, int blocks) {
        a.lead = (int4 *)(ws + p.off_lead);
        a.parts = (float *)(ws + p.off_slots);
        a.slot_rows = p.slot_rows;
        return JoinSet{a.lead, a.parts, blocks, p.slot_rows};
    };
    a.row_lo = 0;
    a.row_hi = INT32_MAX;
    if (dtype == KDA_F32) {
        js[0] = use(w.rows, paged_rows_blocks());
        if ((rc = launch_paged_rows(a, k_cache, v_cache, page_stride, s))) return rc;
        return launch_join(a, js[0], js[1], max_rows, true, s);
    }
    // Up to 16 rows of a kv head fit the few-rows kernel at once; over that the tile
    // kernel, which has room for 128 rows at one cost, is faster (256 windows over up to
    // 4,096 keys of 8 heads: 255 us for 16 rows in the one, then for 20, 24 and 32 rows 251,
    // 254 and 253 us in the other, against 279, 296 and 319 us).  With longer requests in
    // the call it takes them, and the few-rows kernel the single tokens.
    const bool tiles = cache_dtype == KDA_BF16 && a.G <= 128 && max_rows > FEW_ROWS;
    // every request long enough for the tile kernel: one of T_total tokens, or all
    // of max_q (the offsets may still say less: the tile kernel then takes that too)
    const bool few = !tiles || (a.G <= FEW_ROWS && n_seqs > 1 && T_total != (int64_t)n_seqs * a.max_q);
    if (few) {
        if (tiles) a.row_hi = FEW_ROWS;
        js[0] = use(w.rows, paged_few_blocks());
        if ((rc = launch_paged_few(a, cache_dtype, k_cache, v_cache, page_stride, tiles ? FEW_ROWS : max_rows, s))) return rc;
    }
    if (tiles) {
        a.row_lo = few ? FEW_ROWS : 0;
        a.row_hi = INT32_MAX;
        // (the kernel takes parts by the bytes that the lengths say; a table that cannot
        // hold as many asks for none, which spares the join their leads)
        const int parts = (int64_t)n_seqs * max_blocks * page_size * Hkv * D * 4 > (64 << 20) ? w.parts : 1;
        js[1] = use(w.tile, paged_tile_blocks() * parts);
        if ((rc = launch_paged_tile(a, k_cache, v_cache, page_stride, parts, few, s))) return rc;
    }
    return launch_join(a, js[0], js[1], max_rows, false, s);
}

}  // extern "C"
