// kda_paged_attn.cu -- kda_paged_attn: argument checks, workspace layout and
// the launches of paged attention.
#include <cmath>
#include <cstring>

#include "kda_paged.cuh"

namespace kda {
namespace {

struct PagedWs {
    size_t off_slots, total;
    int slot_rows;
};

// [leads][slots]: two leads' int4 and two slots per block of the rows kernel
PagedWs paged_ws(int64_t T, int Hq, int Hkv) {
    PagedWs w;
    const int64_t rows = T * (Hq / Hkv);
    w.slot_rows = rows >= PAGED_ROWS_CAP ? PAGED_ROWS_CAP : rows < 1 ? 16 : (int)((rows + 15) / 16 * 16);
    const int blocks = paged_rows_blocks();
    w.off_slots = align_up((size_t)blocks * 2 * sizeof(int4), 256);
    w.total = align_up(w.off_slots + (size_t)blocks * 2 * paged_slot_floats(w.slot_rows) * sizeof(float), 256);
    return w;
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
    a.window = window;
    a.scale_log2 = sm_scale * 1.4426950408889634f;
    a.row_lo = 0;
    a.row_hi = INT32_MAX;
    a.lead = (int4 *)workspace;
    a.parts = (float *)((char *)workspace + w.off_slots);
    a.slot_rows = w.slot_rows;
    if ((rc = launch_paged_rows(a, cache_dtype, k_cache, v_cache, page_stride, s))) return rc;
    const int64_t rows = (int64_t)a.max_q * a.G;
    return launch_paged_join(a, paged_rows_blocks(), dtype == KDA_F32, (int)(rows < PAGED_ROWS_CAP ? rows : PAGED_ROWS_CAP), s);
}

}  // extern "C"
