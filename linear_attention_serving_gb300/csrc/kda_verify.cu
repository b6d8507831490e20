// kda_verify.cu -- kda_verify_drafts: drafted tokens against the target model's
// probabilities.
//
// One launch; a cluster of blocks takes a request.  Every warp works the tests out for
// itself (a lane to a draft: u q(d) < p(d), in fp64, where the product of two fp32 values is
// exact), then the cluster sums the weights of the one row that the next token comes from
// -- max(p - q, 0), or p -- and finds where the sum passes r times the total.
//
// Weights are summed as 64-bit integers, multiples of 2^-60: sums are then exact whatever
// their order, so the pieces that warps and blocks add up meet without rounding, and the
// place found is the same in every split.  (A value over 2^-37 loses nothing; V = 2^17
// smaller ones are off by under 2^-43 together.)
//
// The row is cut into segments of four vector loads a lane, from the 16 bytes on that it begins in (a row
// of q that lies otherwise is read element by element, through the L1 cache); each warp keeps a segment's sum
// in shared memory.  The blocks tell each other their totals through distributed shared
// memory; the one that holds the place finds the segment by a scan of its sums, and one warp
// reads that segment again.
#include <cooperative_groups.h>

#include "kda_internal.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int BLOCKS = 4;  // an SM
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_SEGS = 1024;  // of one block
constexpr int KEEP = MAX_SEGS / THREADS;
constexpr int LOADS = 4;   // of 16 bytes, of a lane at a time

struct VerifyArgs {
    const void *target, *draft;
    const int32_t *tokens, *n_draft;
    const float *uniforms;
    int32_t *accepted, *out, *err;
    int64_t t_seq, t_row, d_seq, d_row;
    int W, V, per_seg, segs;  // elements of a segment, segments of a block
};

template <typename T> __device__ __forceinline__ float as_float(T x);
template <> __device__ __forceinline__ float as_float(float x) { return x; }
template <> __device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// A weight in multiples of 2^-60, rounded down; what is no weight (negative, 2 or more, NaN): 0.
// Shifts of the significand: conversions to 64-bit integers run at a few a cycle and SM.
__device__ __forceinline__ uint64_t fixed(float x) {
    const uint32_t b = __float_as_uint(x);
    const uint64_t m = (uint64_t)((b << 5 & 0x0fffffffu) | 0x10000000u) << 32;  // 2^60 for 1.0
    uint64_t r;
    // 127 less the exponent, over 63 for all that counts as 0 (shifts by 64 and more give 0)
    asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"(m), "r"((0x3fffffffu - b) >> 23));
    return r;
}
// sum + max(p - q, 0)
__device__ __forceinline__ uint64_t add_over(uint64_t sum, float p, float q) {
    const int64_t w = (int64_t)(fixed(p) - fixed(q));
    return w >= 0 ? sum + (uint64_t)w : sum;
}

// The elements of 16 bytes.
template <typename T> constexpr int PER16 = 16 / (int)sizeof(T);
template <typename T> struct Load {
    uint4 x;
    __device__ __forceinline__ void get(const T *p) { x = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void none() { x = make_uint4(0, 0, 0, 0); }
    // one by one, from an address on no 16 bytes
    __device__ __forceinline__ void pieces(const T *p) {
        uint32_t w[4];
        if constexpr (sizeof(T) == 4) {
            const uint32_t *u = reinterpret_cast<const uint32_t *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __ldg(u + i);
        } else {
            const unsigned short *u = reinterpret_cast<const unsigned short *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = (uint32_t)__ldg(u + 2 * i) | (uint32_t)__ldg(u + 2 * i + 1) << 16;
        }
        x = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ float operator[](int i) const {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        if (sizeof(T) == 4) return __uint_as_float(w[i & 3]);
        return __uint_as_float(i & 1 ? w[(i >> 1) & 3] & 0xffff0000u : w[(i >> 1) & 3] << 16);
    }
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// The row that the token is drawn from.  q NULL: the weights are p's; gone: a token of no weight (-1: none).
// Places count from the 16 bytes that p begins in: element i stands at place i + skip.
template <typename T> struct Row {
    static constexpr int N = PER16<T>;
    const T *p, *q;
    int gone, skip;
    __device__ __forceinline__ void starts() { skip = (int)((uintptr_t)p & 15u) / (int)sizeof(T); }
    __device__ __forceinline__ uint64_t weight(int i) const {
        if (i == gone) return 0;
        return q ? add_over(0, as_float(p[i]), as_float(q[i])) : fixed(as_float(p[i]));
    }
    // this lane's part of the places [at, at + LOADS x 32 x N).  Q: 0 without q, 1 with both on the same place
    // of 16 bytes, 2 elsewhere
    template <int Q> __device__ __forceinline__ uint64_t part(int64_t at, int V, int lane) const {
        Load<T> a[LOADS], b[LOADS];
        const int64_t e0 = at - skip + lane * N;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int64_t e = e0 + i * 32 * N;
            const bool in = e >= 0 && e + N <= V;
            in ? a[i].get(p + e) : a[i].none();
            if (Q == 1) in ? b[i].get(q + e) : b[i].none();
            if (Q == 2) in ? b[i].pieces(q + e) : b[i].none();
        }
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) sum = Q ? add_over(sum, a[i][j], b[i][j]) : sum + fixed(a[i][j]);
        if (at < skip || at - skip + LOADS * 32 * N > V) {  // the 16 bytes that hold the row's ends and more
#pragma unroll 1
            for (int i = 0; i < LOADS; ++i) {
                const int64_t e = e0 + i * 32 * N;
                if (e >= 0 && e + N <= V) continue;
                for (int64_t k = e < 0 ? 0 : e; k < e + N && k < V; ++k)
                    sum = Q ? add_over(sum, as_float(p[k]), as_float(q[k])) : sum + fixed(as_float(p[k]));
            }
        }
        const int64_t g = (int64_t)gone + skip;  // (certain drafts)
        if (gone >= 0 && g >= at && g < at + LOADS * 32 * N && lane == 0) sum -= fixed(as_float(p[gone]));
        return sum;
    }
};

template <typename T>
__global__ void __launch_bounds__(THREADS, BLOCKS) verify_kernel(const VerifyArgs a) {
    __shared__ uint64_t seg_sum[MAX_SEGS];
    __shared__ uint64_t warp_tot[WARPS], block_tot[2][MAX_CLUSTER];
    __shared__ uint64_t found_left;
    __shared__ int found_seg;
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = (int)cluster.num_blocks(), c = (int)cluster.block_rank();
    const int n = blockIdx.x / CL, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const T *target = (const T *)a.target + n * a.t_seq, *draft = (const T *)a.draft + (a.draft ? n * a.d_seq : 0);
    const float *u = a.uniforms + (int64_t)n * a.W;

    // ---- the tests
    int m = a.n_draft ? a.n_draft[n] : a.W - 1;
    int d = lane < a.W - 1 ? a.tokens[(int64_t)n * (a.W - 1) + lane] : -1;
    const bool bad_m = m < 0 || m >= a.W;
    if (bad_m) m = 0;
    bool stands = false, bad_d = false;
    if (lane < m) {
        bad_d = d < 0 || d >= a.V;
        if (!bad_d) {
            const float p = as_float(target[lane * a.t_row + d]), q = a.draft ? as_float(draft[lane * a.d_row + d]) : 1.f;
            stands = (double)u[lane] * (double)q < (double)p;
        }
    }
    const int acc = __ffs(~__ballot_sync(0xffffffffu, stands)) - 1;  // (lane m, or 32 drafts' end, does not stand)
    const bool first = c == 0 && warp == 0;
    if (first) {
        const bool any_bad = __any_sync(0xffffffffu, bad_d);
        if (lane == 0) {
            a.accepted[n] = acc;
            const int why = (bad_m ? KDA_DEVERR_NUM_ACCEPTED : 0) | (any_bad ? KDA_DEVERR_TOKEN : 0);
            if (why && a.err) atomicOr(a.err, why);
        }
        if (lane < a.W && (lane != acc || bad_m)) a.out[(int64_t)n * a.W + lane] = lane < acc ? d : -1;
    }
    if (bad_m) return;  // (the whole cluster)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this block has begun

    // ---- the weights
    Row<T> row;
    row.p = target + acc * a.t_row;
    row.q = acc < m && a.draft ? draft + acc * a.d_row : nullptr;
    const int refused = __shfl_sync(0xffffffffu, d, acc & 31);
    row.gone = acc < m && !a.draft ? refused : -1;
    row.starts();
    const int s0 = c * a.segs, total_segs = (int)(((int64_t)a.V + row.skip + a.per_seg - 1) / a.per_seg);
    const int ns = max(0, min(a.segs, total_segs - s0));
    uint64_t before, mine, all, incl, excl;
    for (int pass = 0;; ++pass) {
        // (whether q's vectors lie as p's do)
        const int how = !row.q ? 0 : ((uintptr_t)row.p & 15u) == ((uintptr_t)row.q & 15u) ? 1 : 2;
        for (int s = warp; s < ns; s += WARPS) {
            uint64_t sum = 0;
            for (int64_t e = 0; e < a.per_seg; e += 32 * PER16<T> * LOADS) {
                const int64_t at = (int64_t)(s0 + s) * a.per_seg + e;
                sum += how == 0 ? row.template part<0>(at, a.V, lane) : how == 1 ? row.template part<1>(at, a.V, lane) : row.template part<2>(at, a.V, lane);
            }
            sum = warp_sum(sum);
            if (lane == 0) seg_sum[s] = sum;
        }
        __syncthreads();
        // scan: a thread has KEEP segments
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            if (tid * KEEP + i < ns) sum += seg_sum[tid * KEEP + i];
        incl = warp_scan(sum, lane);
        if (lane == 31) warp_tot[warp] = incl;
        __syncthreads();
        mine = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) incl += warp_tot[w];
            mine += warp_tot[w];
        }
        excl = incl - sum;
        if (pass == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // all have
        if (tid < CL) *cluster.map_shared_rank(&block_tot[pass][c], tid) = mine;
        cluster.sync();
        before = all = 0;
        for (int i = 0; i < CL; ++i) {
            if (i < c) before += block_tot[pass][i];
            all += block_tot[pass][i];
        }
        // p - q without any weight: q covers p, and p itself is what is left to draw from
        if (all != 0 || pass == 1 || (!row.q && row.gone < 0)) break;
        row.q = nullptr;
        row.gone = -1;
    }
    int32_t *out = a.out + (int64_t)n * a.W + acc;
    if (all == 0) {
        if (first && lane == 0) {
            *out = -1;
            if (a.err) atomicOr(a.err, KDA_DEVERR_PROBS);
        }
        return;
    }
    // ---- the place: the first partial sum over floor(r x total) (sums are whole numbers)
    float r = u[a.W - 1];
    r = fminf(fmaxf(r, 0.f), 0x1.fffffep-1f);  // (NaN: 0)
    const uint64_t bound = __umul64hi(all, __float2ull_rz(r * 0x1p64f));
    if (bound < before || bound - before >= mine) return;
    const uint64_t at = bound - before;
    if (at >= excl && at < incl) {
        uint64_t rest = at - excl;
        int s = tid * KEEP;
        while (rest >= seg_sum[s]) rest -= seg_sum[s++];  // (the thread's sums are more than rest)
        found_seg = s0 + s;
        found_left = rest;
    }
    __syncthreads();
    if (warp) return;
    uint64_t rest = found_left;
    const int64_t e0 = (int64_t)found_seg * a.per_seg;
    for (int64_t e = e0; e < e0 + a.per_seg; e += 32 * 16) {  // 16 elements a lane, in order
        const int64_t at = e + lane * 16 - row.skip;
        const int k0 = (int)max((int64_t)0, min((int64_t)a.V, at)), k1 = (int)max((int64_t)0, min((int64_t)a.V, at + 16));
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (k0 + i < k1) sum += row.weight(k0 + i);
        const uint64_t in = warp_scan(sum, lane), total = __shfl_sync(0xffffffffu, in, 31);
        if (rest < total) {
            // the lane that holds the place; its elements, one to a lane
            const int who = __ffs(__ballot_sync(0xffffffffu, rest < in)) - 1;
            const uint64_t left = rest - __shfl_sync(0xffffffffu, in - sum, who);
            const int k = __shfl_sync(0xffffffffu, k0, who) + lane, end = __shfl_sync(0xffffffffu, k1, who);
            const uint64_t to = warp_scan(k < end ? row.weight(k) : 0, lane);
            const int j = __ffs(__ballot_sync(0xffffffffu, left < to)) - 1;
            if (lane == j) *out = k;
            break;
        }
        rest -= total;
    }
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" int kda_verify_drafts(const void *target, const void *draft, const int32_t *draft_tokens, const float *uniforms,
                                 const int32_t *n_draft, int N, int W, int V, int dtype, int64_t target_seq_stride,
                                 int64_t target_row_stride, int64_t draft_seq_stride, int64_t draft_row_stride,
                                 int32_t *num_accepted, int32_t *tokens, int32_t *error_word, kda_stream_t stream) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_INVALID_ARG;
    if (N < 1 || W < 1 || V < 1) return KDA_ERR_INVALID_ARG;
    if (W > 32 || N > (1 << 24)) return KDA_ERR_UNSUPPORTED;
    if (!target || !uniforms || !num_accepted || !tokens || (W > 1 && !draft_tokens)) return KDA_ERR_INVALID_ARG;
    const int es = dtype == KDA_BF16 ? 2 : 4;
    if (((uintptr_t)target | (uintptr_t)draft) & (es - 1)) return KDA_ERR_INVALID_ARG;
    if (target_row_stride < V || target_seq_stride < 0 || (draft && (draft_row_stride < V || draft_seq_stride < 0)))
        return KDA_ERR_INVALID_ARG;
    // no output may be an input: blocks of a request read the one while another writes the other
    for (const void *o : {(const void *)num_accepted, (const void *)tokens})
        for (const void *x : {target, draft, (const void *)draft_tokens, (const void *)uniforms, (const void *)n_draft})
            if (x && o == x) return KDA_ERR_INVALID_ARG;
    if ((void *)num_accepted == (void *)tokens) return KDA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    note_begin(s);
    // (places, which count from the 16 bytes that a row begins in, go up to V + 7)
    const int64_t places = (int64_t)V + 7;
    int64_t per_seg = 32 * (16 / es) * LOADS;
    // blocks of a request: so many that the card is full, and none without a segment for each warp
    int cl = 1;
    const int sms = device_sm_count();
    while (cl < MAX_CLUSTER && (int64_t)N * cl < 4 * sms && (int64_t)V > per_seg * WARPS / 2 * cl) cl *= 2;
    while ((places + per_seg * cl - 1) / (per_seg * cl) > MAX_SEGS) per_seg *= 2;
    VerifyArgs a{target, draft, draft_tokens, n_draft, uniforms, num_accepted, tokens, error_word, target_seq_stride,
                 target_row_stride, draft_seq_stride, draft_row_stride, W, V, (int)per_seg,
                 (int)((places + per_seg * cl - 1) / (per_seg * cl))};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(N * cl));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cl;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const cudaError_t e = dtype == KDA_F32 ? cudaLaunchKernelEx(&cfg, verify_kernel<float>, a)
                                           : cudaLaunchKernelEx(&cfg, verify_kernel<__nv_bfloat16>, a);
    note_launch("verify_drafts", s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
