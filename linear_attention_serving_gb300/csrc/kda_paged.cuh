// kda_paged.cuh -- what the paged attention kernels share: arguments, a
// request's geometry, the split of the work over blocks, and the pieces that
// blocks leave for the join.
//
// Rows.  The G = Hq / Hkv query heads of one kv head share its keys, so the
// kernels work on rows r = j G + g of one (request, kv head): new token j,
// query head h G + g, position pos0 + r / G.
//
// Work.  A launch's work is one line of key tiles, ordered by request, kv head,
// row group, tile.  Block c takes the tiles [c per, (c + 1) per): every block
// has the same number whatever the lengths are, so a batch with one long
// request keeps all SMs busy.  An item (request, kv head, row group) that a
// block holds whole is finished there; one cut by a block border leaves one
// piece per block, (running maximum, sum, unnormalised output) in fp32, and the
// join merges them in block order (so the result does not depend on timing).
#pragma once

#include "kda_internal.cuh"
#include "kda_tc.cuh"

namespace kda {

struct PagedAttn {
    const void *q;
    void *o;
    float *lse;
    const int32_t *table, *cu, *kv;
    const float *k_scale, *v_scale;  // e4m3 caches
    int32_t *err;
    int n_seqs, T, max_q, Hq, Hkv, G, page_size, n_pages, max_blocks, window;
    float scale_log2;                // sm_scale * log2(e)
    int row_lo, row_hi;              // this launch takes the requests with row_lo < rows <= row_hi
    int box, box_log;                // keys that one copy takes from a page (a power of two, divides page_size)
    // pieces: lead[c] describes the item whose first piece block c left last;
    // slot 2 c is the piece of block c's first segment, 2 c + 1 of its last
    int4 *lead;
    float *parts;
    int slot_rows;                   // rows per slot
    long long wait_budget;           // clock cycles that a wait may take, where it is under SHORT_BUDGET
};

constexpr long long SHORT_BUDGET = 1000000;  // clock cycles; launches with less take kernels that look at it

struct PagedMaps {
    CUtensorMap k, v;
};

// One request, checked: rows = 0 when there is nothing to do for it.
struct PagedReq {
    int tok0, rows, pos0, k0, kend;  // first token, rows, first query's position, keys [k0, kend)
};

// The first key that a query at position pos sees (pos < 0: it sees none, and pos - window may be
// below -2^31).
__device__ __forceinline__ int first_seen(const PagedAttn &a, int pos) {
    return a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
}
// window - 1 - pos0, which may be past 2^31 for a position before 0; a request has under 2^30 rows, so
// none is further from its first than 2^30.
__device__ __forceinline__ int window_from(const PagedAttn &a, int pos0) {
    const int64_t d = (int64_t)a.window - 1 - pos0;
    return d < (1 << 30) ? (int)d : 1 << 30;
}

// `err` collects what is wrong (only one block records it).
__device__ __forceinline__ PagedReq paged_req(const PagedAttn &a, int i, int *err) {
    PagedReq r{0, 0, 0, 0, 0};
    const int b = a.cu[i], e = a.cu[i + 1];
    int kv = a.kv[i];
    if (b < 0 || e < b || e > a.T || e - b > a.max_q) {
        if (err) *err |= KDA_DEVERR_CU_SEQLENS;
        return r;
    }
    if (kv < 0 || kv > (int64_t)a.max_blocks * a.page_size) {
        if (err) *err |= KDA_DEVERR_LENGTHS;
        kv = 0;
    }
    const int64_t rows = (int64_t)(e - b) * a.G;
    if (rows <= a.row_lo || rows > a.row_hi) return r;
    r.tok0 = b;
    r.rows = (int)rows;
    r.pos0 = kv - (e - b);
    r.kend = kv;
    r.k0 = first_seen(a, r.pos0) & ~(a.box - 1);
    return r;
}

__device__ __forceinline__ int64_t paged_warp_scan(int64_t x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// Where this block's part of the line begins.
struct PagedLine {
    int64_t P0, P1, per;  // the block's units, units per block
    int64_t before;       // units before the request that holds P0
    int64_t units;        // and that request's
    int64_t total;        // the line's
    int req;
};

// All NTHR threads of the block call it; `units(i, err)` counts request i's, `parts(total)`
// says how many parts a block takes, a grid's length apart (this is the first).  `per` is
// at least min_per.  scratch: NTHR / 32 + 3 words.
template <int NTHR, class F, class S>
__device__ __forceinline__ PagedLine paged_line(const PagedAttn &a, int64_t *scratch, int64_t min_per, F units, S parts) {
    constexpr int W = NTHR / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int64_t *found = scratch + W;
    int err = 0;
    int64_t first = tid < a.n_seqs ? units(tid, &err) : 0, total = 0;
    if (a.n_seqs > NTHR) {  // the line's length, when one round does not see all requests
        int64_t sum = first;
        for (int i = tid + NTHR; i < a.n_seqs; i += NTHR) sum += units(i, &err);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) scratch[warp] = sum;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) total += scratch[w];
        __syncthreads();
    }
    if (err && blockIdx.x == 0 && a.err) atomicOr(a.err, err);
    PagedLine r;
    int64_t carry = 0;
    for (int base = 0;; base += NTHR) {
        const int i = base + tid;
        const int64_t t = base == 0 ? first : i < a.n_seqs ? units(i, nullptr) : 0;
        const int64_t inc = paged_warp_scan(t, lane);
        if (lane == 31) scratch[warp] = inc;
        if (tid == 0) found[0] = -1;
        __syncthreads();
        int64_t off = carry, all = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w < warp) off += scratch[w];
            all += scratch[w];
        }
        if (base == 0) {
            if (a.n_seqs <= NTHR) total = all;
            // (units fit 32 bits in all but the longest lines: a short division)
            const uint32_t n = gridDim.x * (uint32_t)parts(total);
            r.total = total;
            r.per = total < INT32_MAX ? (int64_t)(((uint32_t)total + n - 1) / n) : (total + n - 1) / n;
            if (r.per < min_per) r.per = min_per;
            r.P0 = (int64_t)blockIdx.x * r.per;
            r.P1 = r.P0 + r.per < total ? r.P0 + r.per : total;
            r.req = 0;
            r.before = r.units = 0;
            if (r.P0 >= r.P1) return r;
        }
        if (r.P0 >= off + inc - t && r.P0 < off + inc) {
            found[0] = i;
            found[1] = off + inc - t;
            found[2] = t;
        }
        carry += all;
        __syncthreads();
        if (found[0] >= 0 || base + NTHR >= a.n_seqs) break;
        __syncthreads();
    }
    r.req = (int)found[0];
    r.before = found[1];
    r.units = found[2];
    return r;
}

// ---------------------------------------------------------------- pieces
// slot: [slot_rows] {maximum (log2), sum}, then [slot_rows][128] fp32 outputs
__host__ __device__ __forceinline__ size_t paged_slot_floats(int slot_rows) { return (size_t)slot_rows * (2 + D); }
__device__ __forceinline__ float *paged_slot(const PagedAttn &a, int64_t slot) {
    return a.parts + slot * paged_slot_floats(a.slot_rows);
}

// The final value of one row: 4 output channels of lane `lane`.
__device__ __forceinline__ void paged_store_row(const PagedAttn &a, bool f32, int64_t tok, int head, int lane, float4 x,
                                                float m, float l, float vscale) {
    const float f = vscale / l;  // (a NaN of a seen key passes through)
    x.x = l == 0.f ? 0.f : x.x * f;
    x.y = l == 0.f ? 0.f : x.y * f;
    x.z = l == 0.f ? 0.f : x.z * f;
    x.w = l == 0.f ? 0.f : x.w * f;
    const int64_t row = tok * a.Hq + head;
    if (f32) {
        reinterpret_cast<float4 *>(a.o)[row * (D / 4) + lane] = x;
    } else {
        __nv_bfloat162 p = __floats2bfloat162_rn(x.x, x.y), q = __floats2bfloat162_rn(x.z, x.w);
        reinterpret_cast<uint2 *>(a.o)[row * (D / 4) + lane] =
            make_uint2(*reinterpret_cast<uint32_t *>(&p), *reinterpret_cast<uint32_t *>(&q));
    }
    if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

int make_paged_maps(const void *k, const void *v, int cache_dtype, int Hkv, int page_size, int n_pages,
                    int64_t page_stride, int box_rows, PagedMaps *out);

int make_paged_row_maps(const void *k, const void *v, int Hkv, int page_size, int n_pages, int64_t page_stride, int box_rows,
                        PagedMaps *out);
int make_paged_q_map(const void *q, int64_t T, int Hq, int G, int tokens, CUtensorMap *out);

constexpr int PAGED_ROWS_CAP = 64;   // rows of one item of the fp32 kernel (the kernel for few rows takes 32 at most)
constexpr int PAGED_TILE_CAP = 256;  // and of the tile kernel

int check_paged_cache(int Hkv, int Dm, int dtype, int cache_dtype, const float *k_scale, const float *v_scale,
                      const void *k_cache, const void *v_cache, int n_pages, int page_size, int64_t page_stride);
int paged_rows_blocks();
int paged_few_blocks();
int paged_tile_blocks();
int launch_paged_rows(PagedAttn a, const void *k, const void *v, int64_t page_stride, cudaStream_t s);
// max_rows: the most rows that one of its requests can have
int launch_paged_few(PagedAttn a, int cache_dtype, const void *k, const void *v, int64_t page_stride, int64_t max_rows,
                     cudaStream_t s);
// after_rows: the launch before it on the stream is another kernel of the same call (they may overlap);
// max_parts: leads and slots are there for so many parts of a block's work
int launch_paged_tile(PagedAttn a, const void *k, const void *v, int64_t page_stride, int max_parts, bool after_rows,
                      cudaStream_t s);

}  // namespace kda
