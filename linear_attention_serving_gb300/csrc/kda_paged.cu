// kda_paged.cu -- bookkeeping and writes of the paged key/value cache:
// kda_paged_tables (block tables, slot map, positions, offsets) and
// kda_paged_append (new keys and values into their pages).
#include <cuda_fp8.h>

#include "kda_internal.cuh"

namespace kda {
namespace {

// ---------------------------------------------------------------- tables
// Every block scans all requests by itself (two prefix sums in shared memory:
// new tokens, new pages), so that one launch suffices and no block waits for
// another; then each thread places TPT consecutive tokens.  The token that
// opens a page writes that page's table entry: a new page's first token is
// always new.  With few tokens the time is the launch and the chain of dependent
// loads (3.5 us for 256 requests); with many the same chain and the 12 bytes a token
// written, which the L2 cache takes (1.0 M tokens of 150 requests: 7.4 us, 1.7 TB/s).
// Small blocks finish their scan sooner, and no more of them are started than are
// resident at once, each of which scans once (512 threads in two waves: 11.7 us).
constexpr int TAB_THREADS = 256;
constexpr int TAB_BLOCKS = 4;  // an SM
constexpr int TAB_MAX_SEQS = 16384;  // three int32 per request in shared memory

struct TablesArgs {
    const int32_t *new_len, *ctx_len, *free_pages, *free_head;
    int32_t *block_table, *free_head_next, *positions, *cu_q, *kv_len, *err;
    int64_t *slot_map;
    int n_seqs, T, max_blocks, n_free, page_size, n_pages;
};

__device__ __forceinline__ int64_t warp_incl_scan(int64_t x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

template <int TPT>
__global__ void __launch_bounds__(TAB_THREADS) tables_kernel(const TablesArgs a) {
    extern __shared__ int32_t tab_sm[];
    int32_t *cu = tab_sm;                      // [n + 1] first token of each request
    int32_t *first = tab_sm + a.n_seqs + 1;    // [n] free-list index of block 0 if all blocks were new: f_i - had
    int32_t *ctx = first + a.n_seqs;           // [n]
    __shared__ int64_t wtok[TAB_THREADS / 32], wpage[TAB_THREADS / 32];
    __shared__ int bad;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = a.n_seqs, ps = a.page_size;
    const int64_t room = (int64_t)a.max_blocks * ps;
    const int head = *a.free_head;
    if (tid == 0) bad = 0;
    __syncthreads();

    // chunks of TAB_THREADS requests with a running carry
    int64_t tok0 = 0, page0 = 0;
    bool wrong = false;
    for (int base = 0; base < n; base += TAB_THREADS) {
        const int i = base + tid;
        int nw = 0, cx = 0;
        if (i < n) {
            nw = a.new_len[i];
            cx = a.ctx_len[i];
            if (nw < 0 || cx < 0 || (int64_t)nw + cx > room) {
                wrong = true;
                nw = cx = 0;
            }
        }
        const int had = (int)(((int64_t)cx + ps - 1) / ps);
        const int have = (int)(((int64_t)cx + nw + ps - 1) / ps);
        const int64_t t = warp_incl_scan(nw, lane), p = warp_incl_scan(have - had, lane);
        if (lane == 31) {
            wtok[warp] = t;
            wpage[warp] = p;
        }
        __syncthreads();
        int64_t tb = tok0, pb = page0, tsum = 0, psum = 0;
#pragma unroll
        for (int w = 0; w < TAB_THREADS / 32; ++w) {
            if (w < warp) {
                tb += wtok[w];
                pb += wpage[w];
            }
            tsum += wtok[w];
            psum += wpage[w];
        }
        if (i < n) {
            const int64_t c = tb + t - nw, f = head + pb + p - (have - had) - had;
            cu[i] = (int)(c > INT32_MAX ? INT32_MAX : c);
            first[i] = (int)(f > INT32_MAX ? INT32_MAX : f);  // (an overflow fails the checks below)
            ctx[i] = cx;
        }
        tok0 += tsum;
        page0 += psum;
        __syncthreads();
    }
    if (wrong || tok0 != a.T) atomicOr(&bad, KDA_DEVERR_LENGTHS);
    if (head < 0 || head + page0 > a.n_free) atomicOr(&bad, KDA_DEVERR_NO_PAGES);
    if (tid == 0) cu[n] = a.T;
    __syncthreads();
    const int why = bad;
    if (blockIdx.x == 0 && tid == 0) {
        *a.free_head_next = why ? head : (int)(head + page0);
        if (why && a.err) atomicOr(a.err, why);
    }
    const int gid = blockIdx.x * TAB_THREADS + tid, gsize = gridDim.x * TAB_THREADS;
    if (why) {  // a step without tokens: what follows on the stream writes and reads no page by what stood here
        for (int i = gid; i <= n; i += gsize) {
            a.cu_q[i] = 0;
            if (i < n) a.kv_len[i] = a.ctx_len[i];
        }
        for (int64_t t = gid; t < a.T; t += gsize) {
            a.slot_map[t] = -1;
            if (a.positions) a.positions[t] = 0;
        }
        return;
    }
    for (int i = gid; i <= n; i += gsize) {
        a.cu_q[i] = cu[i];
        if (i < n) a.kv_len[i] = ctx[i] + cu[i + 1] - cu[i];
    }

    bool badpage = false;
    for (int64_t t0 = (int64_t)gid * TPT; t0 < a.T; t0 += (int64_t)gsize * TPT) {
        int i, hi = n;  // the last request with cu[i] <= t0
        {
            int lo = 0;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= (int)t0) lo = mid;
                else hi = mid;
            }
            i = lo;
        }
        int end = cu[i + 1], pos = 0, b = 0, off = 0, page = -1;
        bool fresh = true;
        int64_t slot[TPT];
        int ppos[TPT];
#pragma unroll
        for (int j = 0; j < TPT; ++j) {
            const int64_t t = t0 + j;
            slot[j] = -1;
            ppos[j] = 0;
            if (t < a.T) {
                if (j > 0 && t >= end) {
                    do ++i;
                    while (cu[i + 1] <= (int)t);
                    end = cu[i + 1];
                    fresh = true;
                }
                if (fresh) {
                    pos = ctx[i] + (int)(t - cu[i]);
                    b = pos / ps;
                    off = pos - b * ps;
                } else {
                    ++pos;
                    if (++off == ps) {
                        off = 0;
                        ++b;
                    }
                }
                if (fresh || off == 0) {
                    const int had = (int)(((uint32_t)ctx[i] + (uint32_t)ps - 1) / (uint32_t)ps);
                    const bool is_new = b >= had;
                    int32_t *entry = a.block_table + (int64_t)i * a.max_blocks + b;
                    page = is_new ? a.free_pages[first[i] + b] : *entry;
                    if (page < 0 || page >= a.n_pages) {
                        badpage = true;
                        page = -1;
                    }
                    if (is_new && off == 0) *entry = page;
                }
                fresh = false;
                slot[j] = page < 0 ? -1 : (int64_t)page * ps + off;
                ppos[j] = pos;
            }
        }
        if (TPT == 4 && t0 + 4 <= a.T) {  // t0 is a multiple of 4
            longlong2 *s = reinterpret_cast<longlong2 *>(a.slot_map + t0);
            s[0] = make_longlong2(slot[0], slot[1]);
            s[1] = make_longlong2(slot[2 % TPT], slot[3 % TPT]);
            if (a.positions)
                *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(ppos[0], ppos[1 % TPT], ppos[2 % TPT], ppos[3 % TPT]);
        } else {
#pragma unroll
            for (int j = 0; j < TPT; ++j)
                if (t0 + j < a.T) {
                    a.slot_map[t0 + j] = slot[j];
                    if (a.positions) a.positions[t0 + j] = ppos[j];
                }
        }
    }
    if (badpage && a.err) atomicOr(a.err, KDA_DEVERR_PAGE);
}

// ---------------------------------------------------------------- append
// One pass over the new rows: a thread moves 16 input bytes of K and of V (a
// row of 128 bf16 takes 16 threads, of fp32 32), so both sides of the copy are
// coalesced within a row, which is one contiguous piece of a page.  Bound by
// HBM: every row is read once and written once.
template <typename T, bool E4M3>
__device__ __forceinline__ void put(const uint4 x, float scale, char *row, int c) {
    if (!E4M3) {
        reinterpret_cast<uint4 *>(row)[c] = x;
        return;
    }
    // x / scale in fp32, then one rounding to e4m3 (a true division: a product
    // with 1 / scale would round twice and move values across a border)
    const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&x);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t r = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 f = __bfloat1622float2(p[2 * i + j]);
            const __nv_fp8x2_storage_t b =
                __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f.x, scale), __fdiv_rn(f.y, scale)), __NV_SATFINITE, __NV_E4M3);
            r |= (uint32_t)b << (16 * j);
        }
        w[i] = r;
    }
    reinterpret_cast<uint2 *>(row)[c] = make_uint2(w[0], w[1]);
}

struct AppendArgs {
    const void *k, *v;
    const int64_t *slot_map;
    const float *k_scale, *v_scale;
    char *k_cache, *v_cache;
    int32_t *err;
    int64_t T, page_bytes, n_slots;
    int Hkv, page_size;
};

template <typename T, bool E4M3>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
    constexpr int PER = 16 / (int)sizeof(T);      // elements a thread moves
    constexpr int TPR = D / PER;                  // threads per row
    constexpr int OUT = E4M3 ? 1 : (int)sizeof(T);
    const int64_t gid = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t rows = a.T * a.Hkv;
    const int64_t r = gid / TPR;
    const int c = (int)(gid % TPR);
    if (r >= rows) return;
    const uint4 xk = __ldg(reinterpret_cast<const uint4 *>(a.k) + r * TPR + c);
    const uint4 xv = __ldg(reinterpret_cast<const uint4 *>(a.v) + r * TPR + c);
    int64_t t;
    int h;
    if (rows <= UINT32_MAX) {
        t = (uint32_t)r / (uint32_t)a.Hkv;
        h = (int)((uint32_t)r - (uint32_t)t * (uint32_t)a.Hkv);
    } else {
        t = r / a.Hkv;
        h = (int)(r - t * a.Hkv);
    }
    const int64_t slot = a.slot_map[t];
    if (slot < 0) return;
    if (slot >= a.n_slots) {
        if (c == 0 && h == 0 && a.err) atomicOr(a.err, KDA_DEVERR_PAGE);
        return;
    }
    int64_t page;
    int off;
    if (a.n_slots <= UINT32_MAX) {
        page = (uint32_t)slot / (uint32_t)a.page_size;
        off = (int)((uint32_t)slot - (uint32_t)page * (uint32_t)a.page_size);
    } else {
        page = slot / a.page_size;
        off = (int)(slot - page * a.page_size);
    }
    const int64_t at = page * a.page_bytes + ((int64_t)h * a.page_size + off) * D * OUT;
    put<T, E4M3>(xk, E4M3 ? a.k_scale[h] : 1.f, a.k_cache + at, c);
    put<T, E4M3>(xv, E4M3 ? a.v_scale[h] : 1.f, a.v_cache + at, c);
}

}  // namespace

// Checks that the paged calls share: the cache's geometry and types.
int check_paged_cache(int Hkv, int Dm, int dtype, int cache_dtype, const float *k_scale, const float *v_scale,
                      const void *k_cache, const void *v_cache, int n_pages, int page_size, int64_t page_stride) {
    if (Dm != D) return KDA_ERR_UNSUPPORTED;
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_INVALID_ARG;
    if (cache_dtype != dtype && !(dtype == KDA_BF16 && cache_dtype == KDA_E4M3)) {
        return cache_dtype == KDA_BF16 || cache_dtype == KDA_F32 || cache_dtype == KDA_E4M3 ? KDA_ERR_UNSUPPORTED
                                                                                           : KDA_ERR_INVALID_ARG;
    }
    if ((cache_dtype == KDA_E4M3) != (k_scale != nullptr) || (cache_dtype == KDA_E4M3) != (v_scale != nullptr))
        return KDA_ERR_INVALID_ARG;
    if (Hkv < 1 || n_pages < 1 || page_size < 16) return KDA_ERR_INVALID_ARG;
    if (page_size % 16) return KDA_ERR_UNSUPPORTED;
    // the rows of one page are a dimension of the cache's tensor maps, and slots
    // and block positions stay in range
    if ((int64_t)Hkv * page_size > (int64_t)INT32_MAX) return KDA_ERR_INVALID_ARG;
    const int el = cache_dtype == KDA_BF16 ? 2 : cache_dtype == KDA_F32 ? 4 : 1;
    if (page_stride < (int64_t)Hkv * page_size * D || (page_stride * el) % 16) return KDA_ERR_INVALID_ARG;
    if (page_stride > ((int64_t)1 << 38) / el) return KDA_ERR_INVALID_ARG;  // a tensor map's stride ends at 2^40 bytes
    if (!k_cache || !v_cache || ((uintptr_t)k_cache & 15u) || ((uintptr_t)v_cache & 15u)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace kda

using namespace kda;

extern "C" {

int kda_paged_tables(const int32_t *new_len, const int32_t *ctx_len, int n_seqs, int64_t T_total,
                     int32_t *block_table, int max_blocks, const int32_t *free_pages, int n_free,
                     const int32_t *free_head, int32_t *free_head_next, int page_size, int n_pages,
                     int64_t *slot_map, int32_t *positions, int32_t *cu_q, int32_t *kv_len, int32_t *error_word,
                     kda_stream_t stream) {
    if (n_seqs < 1 || T_total < 0 || T_total >= (int64_t)INT32_MAX || max_blocks < 1 || n_free < 0 || n_pages < 1 ||
        page_size < 16)
        return KDA_ERR_INVALID_ARG;
    if (n_seqs > TAB_MAX_SEQS || page_size % 16) return KDA_ERR_UNSUPPORTED;
    // positions are int32
    if ((int64_t)max_blocks * page_size > (int64_t)INT32_MAX) return KDA_ERR_INVALID_ARG;
    if (!new_len || !ctx_len || !block_table || !free_head || !free_head_next || !cu_q || !kv_len)
        return KDA_ERR_INVALID_ARG;
    if (free_head == free_head_next || (n_free > 0 && !free_pages) || (T_total > 0 && !slot_map))
        return KDA_ERR_INVALID_ARG;
    if (((uintptr_t)slot_map & 15u) || ((uintptr_t)positions & 15u)) return KDA_ERR_INVALID_ARG;
    // every block reads all lengths and pages, some while others write already
    const void *in[] = {new_len, ctx_len, free_pages, free_head};
    for (const void *x : in)
        if (x && (x == cu_q || x == kv_len || x == positions || x == slot_map || x == free_head_next || x == block_table))
            return KDA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    note_begin(s);
    const TablesArgs a{new_len,  ctx_len,   free_pages, free_head,  block_table, free_head_next, positions,
                       cu_q,     kv_len,    error_word, slot_map,   n_seqs,      (int)T_total,   max_blocks,
                       n_free,   page_size, n_pages};
    // One token a thread while that fits the blocks that are resident at once (the
    // dependent loads of a thread's tokens would only add up), else four with 16-byte stores.
    const int most = TAB_BLOCKS * device_sm_count();
    const bool four = T_total > (int64_t)most * TAB_THREADS;
    const int64_t threads = four ? (T_total + 3) / 4 : T_total;
    int64_t blocks = (threads + TAB_THREADS - 1) / TAB_THREADS;
    if (blocks < 1) blocks = 1;
    if (blocks > most) blocks = most;
    const void *f = four ? (const void *)tables_kernel<4> : (const void *)tables_kernel<1>;
    const int smem = (3 * n_seqs + 1) * (int)sizeof(int32_t);
    // (one entry of the launch-preparation cache per kernel, not one per batch size)
    const int rc = prepare_kernel(f, (3 * TAB_MAX_SEQS + 1) * (int)sizeof(int32_t), TAB_THREADS, nullptr);
    if (rc) return rc;
    if (four)
        tables_kernel<4><<<(int)blocks, TAB_THREADS, smem, s>>>(a);
    else
        tables_kernel<1><<<(int)blocks, TAB_THREADS, smem, s>>>(a);
    note_launch("paged_tables", s);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int kda_paged_append(const void *k, const void *v, const int64_t *slot_map, int64_t T_total, int Hkv, int Dm,
                     int dtype, int cache_dtype, const float *k_scale, const float *v_scale, void *k_cache,
                     void *v_cache, int n_pages, int page_size, int64_t page_stride, int32_t *error_word,
                     kda_stream_t stream) {
    const int rc = check_paged_cache(Hkv, Dm, dtype, cache_dtype, k_scale, v_scale, k_cache, v_cache, n_pages, page_size,
                                     page_stride);
    if (rc) return rc;
    if (T_total < 0 || T_total >= (int64_t)INT32_MAX) return KDA_ERR_INVALID_ARG;
    if (T_total == 0) return KDA_OK;
    if (!k || !v || !slot_map || ((uintptr_t)k & 15u) || ((uintptr_t)v & 15u)) return KDA_ERR_INVALID_ARG;
    const int el = cache_dtype == KDA_BF16 ? 2 : cache_dtype == KDA_F32 ? 4 : 1;
    const int tpr = dtype == KDA_BF16 ? D / 8 : D / 4;
    const int64_t blocks = (T_total * Hkv * tpr + 255) / 256;
    if (blocks > (int64_t)INT32_MAX) return KDA_ERR_UNSUPPORTED;
    cudaStream_t s = (cudaStream_t)stream;
    note_begin(s);
    const AppendArgs a{k, v, slot_map, k_scale, v_scale, (char *)k_cache, (char *)v_cache, error_word, T_total,
                       page_stride * el, (int64_t)n_pages * page_size, Hkv, page_size};
    if (cache_dtype == KDA_E4M3)
        append_kernel<__nv_bfloat16, true><<<(unsigned)blocks, 256, 0, s>>>(a);
    else if (dtype == KDA_BF16)
        append_kernel<__nv_bfloat16, false><<<(unsigned)blocks, 256, 0, s>>>(a);
    else
        append_kernel<float, false><<<(unsigned)blocks, 256, 0, s>>>(a);
    note_launch("paged_append", s);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
