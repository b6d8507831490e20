// kda_verify.cu -- kda_verify_drafts: drafted tokens against the target model's
// probabilities.
//
// Two launches.  The first works the tests out (a warp to a request, a lane to a draft:
// u q(d) < p(d), in fp64, where the product of two fp32 values is exact), and sums the weights of
// the one row that the next token comes from -- max(p - q, 0), or p -- by segments.  The
// segments of all requests are one line, cut evenly over the blocks that are resident at once, so
// that few requests or many, the card is full and its blocks end together.  The second launch, a
// block to a request, scans the segments' sums, finds where the sum passes r times the
// total, and reads that one segment again.
//
// Weights are summed as 64-bit integers, multiples of 2^-60: sums are then exact whatever
// their order, and the place found is the same in every split.  (Each weight is rounded once;
// values over 2^-36 of p alone lose nothing.)
//
// Bound by HBM (one row of p, or of p and q, for each request), which takes copies in flight:
// each warp has bulk copies of its next pieces under way into shared memory, and neither
// registers nor other warps have a part in it.  256 requests of 131,072 tokens (four drafts, fp32, 234 MB read)
// 45 us, of which the second launch's part 3; 64 of 100,003 in bf16, no draft probabilities, 13 us, and one of
// 32,768 5.8 to 6.3 us, which are the chain of launch, tests, row, sums, place.  (A cluster of blocks to a
// request, registers for what is under way, took 59, 13.7 and 7.2 us.)
#include <algorithm>

#include "kda_internal.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int BLOCKS = 3;            // an SM
constexpr int STAGES = 2;            // pieces under way for each warp
// Bytes of p in a piece: a piece costs its warp some hundred instructions besides its weights (256
// requests of 131,072 tokens 58 us with 1 KB, 47 with 2, 54 with 4), but few pieces leave warps idle,
// and the last search is through one piece (one request of 32,768 5.8, 7.5 and 11 us).
constexpr int SMALL = 1024, LARGE = 2048;
// p; q from the 16 bytes on that it begins in
template <int PIECE> constexpr int ROOM_OF = 2 * PIECE + 16;
constexpr int MAX_SEGS = 1024;       // of a request
constexpr int KEEP = MAX_SEGS / THREADS;
constexpr int MAX_N = 1 << 24, MAX_W = 32;
constexpr int MAX_V = INT32_MAX - 4096;  // (a piece past the row's end stays clear of 2^31)

struct VerifyArgs {
    const void *target, *draft;
    const int32_t *tokens, *n_draft;
    const float *uniforms;
    int32_t *accepted, *out, *err;
    uint64_t *sums;  // [N][segs]
    int64_t t_seq, t_row, d_seq, d_row;
    int N, W, V, pieces, segs;  // pieces of a segment, segments of a request
};

template <typename T> __device__ __forceinline__ float as_float(T x);
template <> __device__ __forceinline__ float as_float(float x) { return x; }
template <> __device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// ---------------------------------------------------------------- weights
// The weight max(p - q, 0), p and q not negative, in multiples of 2^-60.
//   s + e = max(p, q) - q exactly: s = fl(p - q) and, as p >= q, e = fl(fl(p - s) - q) (Dekker 1971)
// Whole numbers are cut off by adding a power of two that leaves no place for a fraction: the sum's
// last bits are the nearest whole number, and what is left of the value is exact.  s in multiples
// of 2^-22 (s < 2: 23 bits) is A; what is left, and e, in multiples of 2^-45 are B and B'; what is
// left of both in multiples of 2^-60 is C, which alone is rounded.  The floats' bits are added up
// as they are, 32 of each at most, and put together then.
// (In packed fp32 operations, on pipes that have nothing else to do here; with shifts of
// the significands a pair of values took 40 instructions, and 256 requests 64 us.)
constexpr uint32_t A_BITS = 0x4b000000u, B_BITS = 0x4b400000u;  // of 2^23 and 3 x 2^22
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t both(float x) { return pack2(x, x); }
__device__ __forceinline__ uint32_t bits_lo(uint64_t x) { return (uint32_t)x; }
__device__ __forceinline__ uint32_t bits_hi(uint64_t x) { return (uint32_t)(x >> 32); }

struct Weights {
    uint32_t a = 0, b = 0, c = 0;
    // two values each (Q: of p and q, else of p alone)
    template <bool Q> __device__ __forceinline__ void add(float p0, float p1, float q0, float q1) {
        const uint64_t minus = both(-1.f), one_a = both(0x1p23f), one_b = both(0x1.8p23f);
        uint64_t s, e = 0;
        if (Q) {
            q0 = fmaxf(q0, 0.f), q1 = fmaxf(q1, 0.f);  // (NaN: 0)
            const uint64_t p = pack2(fmaxf(p0, q0), fmaxf(p1, q1)), q = pack2(q0, q1);
            s = fma2(q, minus, p);
            e = fma2(q, minus, fma2(s, minus, p));
        } else {
            s = pack2(fmaxf(p0, 0.f), fmaxf(p1, 0.f));
        }
        const uint64_t A = fma2(s, both(0x1p22f), one_a);
        const uint64_t r = fma2(s, both(0x1p22f), fma2(A, minus, one_a));
        const uint64_t B = fma2(r, both(0x1p23f), one_b);
        uint64_t left = fma2(r, both(0x1p23f), fma2(B, minus, one_b));
        a += bits_lo(A) + bits_hi(A);
        b += bits_lo(B) + bits_hi(B);
        if (Q) {
            const uint64_t B2 = fma2(e, both(0x1p45f), one_b);
            left = add2(left, fma2(e, both(0x1p45f), fma2(B2, minus, one_b)));
            b += bits_lo(B2) + bits_hi(B2);
        }
        const uint64_t C = fma2(left, both(0x1p15f), one_b);
        c += bits_lo(C) + bits_hi(C);
    }
    // the sum of n values (2 in each `add`)
    template <bool Q> __device__ __forceinline__ uint64_t sum(uint32_t n) const {
        const int64_t x = (int32_t)(a - n * A_BITS), y = (int32_t)(b - (Q ? 2 * n : n) * B_BITS), z = (int32_t)(c - n * B_BITS);
        return (uint64_t)(x * (1ll << 38) + y * (1 << 15) + z);
    }
    template <bool Q> static __device__ __forceinline__ uint64_t one(float p, float q) {
        Weights w;
        w.template add<Q>(p, 0.f, q, 0.f);
        return w.template sum<Q>(2);
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

// ---------------------------------------------------------------- rows
template <typename T, int PIECE> constexpr int PER_PIECE = PIECE / (int)sizeof(T);  // elements
template <typename T, int PIECE> constexpr int PER_LANE = PER_PIECE<T, PIECE> / 32;

// The row that the token is drawn from.  q NULL: the weights are p's; gone: a token of no weight (-1: none;
// a certain draft that is no token, which may be any number, takes no weight from anything).
// Places count from the 16 bytes that p begins in: element i stands at place i + skip.
template <typename T> struct Row {
    const T *p, *q;
    int gone, skip;
    __device__ __forceinline__ uint64_t weight(int i) const {
        if (i == gone) return 0;
        return q ? Weights::one<true>(as_float(p[i]), as_float(q[i])) : Weights::one<false>(as_float(p[i]), 0.f);
    }
};

struct Test {
    int acc, m, d;  // drafts that stand, drafts, the first that does not (where acc < m)
    bool bad;       // no drafts to speak of: the request is left out
};
// A whole warp, a lane to a draft.  write: the accepted drafts and their number too, -1 behind them.
template <typename T> __device__ __forceinline__ Test test_drafts(const VerifyArgs &a, int n, int lane, bool write) {
    Test t;
    t.m = a.n_draft ? a.n_draft[n] : a.W - 1;
    const int d = lane < a.W - 1 ? a.tokens[(int64_t)n * (a.W - 1) + lane] : -1;
    t.bad = t.m < 0 || t.m >= a.W;
    if (t.bad) t.m = 0;
    bool stands = false, bad_d = false;
    if (lane < t.m) {
        bad_d = d < 0 || d >= a.V;
        if (!bad_d) {
            const float p = as_float(((const T *)a.target + n * a.t_seq)[lane * a.t_row + d]);
            const float q = a.draft ? as_float(((const T *)a.draft + n * a.d_seq)[lane * a.d_row + d]) : 1.f;
            stands = (double)a.uniforms[(int64_t)n * a.W + lane] * (double)q < (double)p;
        }
    }
    t.acc = __ffs(~__ballot_sync(0xffffffffu, stands)) - 1;  // (lane m does not stand, nor lane 31)
    t.d = __shfl_sync(0xffffffffu, d, t.acc & 31);
    if (write) {
        const bool any_bad = __any_sync(0xffffffffu, bad_d);
        if (lane == 0) {
            a.accepted[n] = t.acc;
            const int why = (t.bad ? KDA_DEVERR_NUM_ACCEPTED : 0) | (any_bad ? KDA_DEVERR_TOKEN : 0);
            if (why && a.err) atomicOr(a.err, why);
        }
        if (lane < a.W) a.out[(int64_t)n * a.W + lane] = lane < t.acc ? d : -1;
    }
    return t;
}
template <typename T> __device__ __forceinline__ Row<T> row_of(const VerifyArgs &a, int n, const Test &t) {
    Row<T> r;
    r.p = (const T *)a.target + n * a.t_seq + t.acc * a.t_row;
    r.q = t.acc < t.m && a.draft ? (const T *)a.draft + n * a.d_seq + t.acc * a.d_row : nullptr;
    r.gone = t.acc < t.m && !a.draft && t.d >= 0 && t.d < a.V ? t.d : -1;
    r.skip = (int)((uintptr_t)r.p & 15u) / (int)sizeof(T);
    return r;
}

// ---------------------------------------------------------------- segments' sums
// What a warp does with one of its pieces.
template <typename T> struct __align__(16) Job {
    Row<T> row;
    int64_t place;  // its first
    int64_t to;     // segment of the line whose sum this piece ends, or -1
    int shift;      // elements that q begins into its room
    bool any;
};

// The elements that 16 bytes hold, two at a time.
template <typename T> __device__ __forceinline__ float element(const uint4 &x, int i) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if (sizeof(T) == 4) return __uint_as_float(w[i & 3]);
    return __uint_as_float(i & 1 ? w[(i >> 1) & 3] & 0xffff0000u : w[(i >> 1) & 3] << 16);
}
template <typename T, int PIECE, bool Q> __device__ __forceinline__ uint64_t aligned_piece(const uint8_t *sm, int lane) {
    constexpr int N = 16 / (int)sizeof(T), VECS = PIECE / 512;
    Weights w;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const uint4 x = reinterpret_cast<const uint4 *>(sm)[i * 32 + lane];
        const uint4 y = Q ? reinterpret_cast<const uint4 *>(sm + PIECE)[i * 32 + lane] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < N; j += 2)
            w.template add<Q>(element<T>(x, j), element<T>(x, j + 1), element<T>(y, j), element<T>(y, j + 1));
    }
    return w.template sum<Q>(VECS * N);
}
// q begins `shift` elements into its room.
template <typename T, int PIECE> __device__ __forceinline__ uint64_t shifted_piece(const uint8_t *sm, int shift, int lane) {
    const T *p = reinterpret_cast<const T *>(sm), *q = reinterpret_cast<const T *>(sm + PIECE) + shift;
    Weights w;
#pragma unroll
    for (int i = 0; i < PER_LANE<T, PIECE>; i += 2)
        w.template add<true>(as_float(p[i * 32 + lane]), as_float(p[i * 32 + 32 + lane]), as_float(q[i * 32 + lane]), as_float(q[i * 32 + 32 + lane]));
    return w.template sum<true>(PER_LANE<T, PIECE>);
}
// A piece that the row begins or ends in: elements [e0, e0 + PER_PIECE) of a row of V, to dst (where element
// e0's place within 16 bytes is kept, `off`): 16 bytes at a time where they are the row's, the
// elements at its ends one by one, zeros outside.  A whole warp; returns the bytes that come by copy.
template <typename T, int PIECE>
__device__ __forceinline__ uint32_t edge_piece(uint8_t *dst, const T *row, int64_t e0, int off, int V, uint64_t *bar, int lane) {
    constexpr int N = 16 / (int)sizeof(T);
    const int v0 = (int)min((int64_t)PER_PIECE<T, PIECE>, max((int64_t)0, -e0)), v1 = (int)max((int64_t)v0, min((int64_t)PER_PIECE<T, PIECE>, V - e0));
    T *at = reinterpret_cast<T *>(dst + off);
    const int o = off / (int)sizeof(T);
    const int a0 = min(v1, (v0 + o + N - 1) / N * N - o), a1 = max(a0, (v1 + o) / N * N - o);
    for (int i = lane; i < PER_PIECE<T, PIECE>; i += 32)
        if (i < v0 || i >= v1) at[i] = T(0.f);
    const int i = lane < 16 ? v0 + lane : a1 + lane - 16;
    if (lane < 16 ? i < a0 : i < v1) at[i] = row[e0 + i];
    const uint32_t bytes = (uint32_t)(a1 - a0) * sizeof(T);
    if (bytes && lane == 0) tc::bulk_g2s(at + a0, row + e0 + a0, bytes, bar);
    return bytes;
}

template <typename T, int PIECE>
__global__ void __launch_bounds__(THREADS, BLOCKS) verify_sums_kernel(const VerifyArgs a) {
    constexpr int ROOM = ROOM_OF<PIECE>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(128) uint8_t sm_all[];
    __shared__ uint64_t bars[WARPS][STAGES];
    __shared__ Job<T> jobs[WARPS][STAGES];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *sm = sm_all + warp * STAGES * ROOM;
    uint64_t *bar = bars[warp];
    Job<T> *job = jobs[warp];
    if (lane == 0) {
        for (int i = 0; i < STAGES; ++i) tc::mbar_init(&bar[i], 1);
        tc::mbar_fence_init();
    }
    __syncwarp();
    // the block's part of the line; its warps take every WARPS-th segment
    const int64_t line = (int64_t)a.N * a.segs, per = (line + gridDim.x - 1) / gridDim.x;
    const int64_t g0 = (int64_t)blockIdx.x * per, g1 = min(line, g0 + per);
    // the next piece: its segment (of the line; request i, segment s of it), its number there
    int64_t g = g0 + warp;
    int i = (int)(g / a.segs), s = (int)(g - (int64_t)i * a.segs), piece = 0;
    // the request's row; its pieces that are copied whole, [p0, p1), p1 < 0: the request is left out
    Row<T> row;
    int64_t p0 = 0, p1 = 0;
    int off = 0;
    bool fresh = true;
    auto issue = [&](int stage) -> bool {
        if (g >= g1) return false;
        if (fresh) {
            const Test t = test_drafts<T>(a, i, lane, s == 0);
            row = row_of<T>(a, i, t);
            off = row.q ? (int)((uintptr_t)(row.q - row.skip) & 15u) : 0;
            // (16 bytes more of q are read than the piece has, from the 16 bytes on that it begins in)
            const int more = off ? 16 / (int)sizeof(T) : 0;
            p0 = (row.skip + more + PER_PIECE<T, PIECE> - 1) / PER_PIECE<T, PIECE>;
            p1 = t.bad ? -1 : max((int64_t)0, ((int64_t)a.V + row.skip - more) / PER_PIECE<T, PIECE>);
            fresh = false;
        }
        const int64_t k = (int64_t)s * a.pieces + piece, e = k * PER_PIECE<T, PIECE> - row.skip;
        const bool whole = k >= p0 && k < p1;
        uint8_t *at = sm + stage * ROOM;
        uint32_t bytes = 0;
        if (!whole && p1 >= 0) {
            bytes = edge_piece<T, PIECE>(at, row.p, e, 0, a.V, &bar[stage], lane);
            if (row.q) bytes += edge_piece<T, PIECE>(at + PIECE, row.q, e, off, a.V, &bar[stage], lane);
            tc::fence_async_smem();  // (later copies overwrite what was stored here)
            __syncwarp();
        }
        if (lane == 0) {
            Job<T> &j = job[stage];
            j.row = row;
            j.place = k * PER_PIECE<T, PIECE>;
            j.to = piece == a.pieces - 1 ? g : -1;
            j.shift = off / (int)sizeof(T);
            j.any = p1 >= 0;
            if (whole) {
                const uint32_t qb = !row.q ? 0 : PIECE + (off ? 16 : 0);
                tc::mbar_expect_tx(&bar[stage], PIECE + qb);
                tc::bulk_g2s(at, row.p + e, PIECE, &bar[stage]);
                if (qb) tc::bulk_g2s(at + PIECE, (const uint8_t *)(row.q + e) - off, qb, &bar[stage]);
            } else {
                tc::mbar_expect_tx(&bar[stage], bytes);
            }
        }
        __syncwarp();
        if (++piece == a.pieces) {
            piece = 0;
            g += WARPS;
            for (s += WARPS; s >= a.segs; s -= a.segs) {
                ++i;
                fresh = true;
            }
        }
        return true;
    };
    int under_way = 0;
    for (int k = 0; k < STAGES; ++k) under_way += issue(k);
    uint64_t sum = 0;
    for (int x = 0; under_way > 0; ++x) {
        const int stage = x % STAGES;
        if (!__all_sync(0xffffffffu, tc::mbar_wait(&bar[stage], (x / STAGES) & 1))) {
            if (lane == 0 && a.err) atomicOr(a.err, KDA_DEVERR_TIMEOUT);
            for (int k = 0; k < under_way; ++k) tc::mbar_wait(&bar[(x + k) % STAGES], ((x + k) / STAGES) & 1);
            return;
        }
        const Job<T> j = job[stage];
        const uint8_t *at = sm + stage * ROOM;
        if (j.any) sum += !j.row.q ? aligned_piece<T, PIECE, false>(at, lane)
                          : !j.shift ? aligned_piece<T, PIECE, true>(at, lane) : shifted_piece<T, PIECE>(at, j.shift, lane);
        if (j.any && j.row.gone >= 0 && lane == 0) {  // (certain drafts)
            const int64_t e = j.row.gone + j.row.skip - j.place;
            if (e >= 0 && e < PER_PIECE<T, PIECE>) sum -= Weights::one<false>(as_float(j.row.p[j.row.gone]), 0.f);
        }
        if (j.to >= 0) {
            sum = warp_sum(sum);
            if (lane == 0) a.sums[j.to] = sum;
            sum = 0;
        }
        __syncwarp();  // (all have read the stage)
        if (!issue(stage)) --under_way;
    }
}

// ---------------------------------------------------------------- the place
// Sums of the request's segments before and with this thread's (KEEP of them), and of all.
struct Scan {
    uint64_t excl, incl, total;
};
__device__ __forceinline__ Scan scan_segments(uint64_t *warp_tot, int segs, const uint64_t *sums) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t sum = 0;
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
        if (tid * KEEP + i < segs) sum += sums[tid * KEEP + i];
    Scan r;
    r.incl = warp_scan(sum, lane);
    if (lane == 31) warp_tot[warp] = r.incl;
    __syncthreads();
    r.total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) r.incl += warp_tot[w];
        r.total += warp_tot[w];
    }
    r.excl = r.incl - sum;
    return r;
}
template <typename T, int PIECE>
__global__ void __launch_bounds__(THREADS, 2) verify_place_kernel(const VerifyArgs a) {
    __shared__ uint64_t warp_tot[2][WARPS];
    __shared__ uint64_t found_left;
    __shared__ int found_seg;
    const int n = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Test t;
    t.m = a.n_draft ? a.n_draft[n] : a.W - 1;
    const float u = a.uniforms[(int64_t)n * a.W + a.W - 1];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (t.m < 0 || t.m >= a.W) return;
    t.acc = a.accepted[n];
    t.d = t.acc < t.m ? a.tokens[(int64_t)n * (a.W - 1) + t.acc] : -1;
    Row<T> row = row_of<T>(a, n, t);
    uint64_t *mine = a.sums + (int64_t)n * a.segs;
    Scan sc = scan_segments(warp_tot[0], a.segs, mine);
    if (sc.total == 0 && (row.q || row.gone >= 0)) {
        // p - q without any weight: q covers p, and p itself is what is left to draw from (rare: the
        // block reads the row alone)
        row.q = nullptr;
        row.gone = -1;
        for (int s = warp; s < a.segs; s += WARPS) {
            uint64_t sum = 0;
            const int64_t k0 = (int64_t)s * a.pieces * PER_PIECE<T, PIECE> - row.skip, k1 = k0 + (int64_t)a.pieces * PER_PIECE<T, PIECE>;
            for (int64_t k = max((int64_t)0, k0) + lane; k < min((int64_t)a.V, k1); k += 32) sum += row.weight((int)k);
            sum = warp_sum(sum);
            if (lane == 0) mine[s] = sum;
        }
        __syncthreads();
        sc = scan_segments(warp_tot[1], a.segs, mine);
    }
    if (sc.total == 0) {
        if (tid == 0 && a.err) atomicOr(a.err, KDA_DEVERR_PROBS);
        return;
    }
    // the first partial sum over floor(r x total) (sums are whole numbers)
    const float r = fminf(fmaxf(u, 0.f), 0x1.fffffep-1f);  // (NaN: 0)
    const uint64_t at = __umul64hi(sc.total, __float2ull_rz(r * 0x1p64f));
    if (tid == 0) found_seg = -1;  // (rows that sum to too much may have no place)
    __syncthreads();
    if (at >= sc.excl && at < sc.incl) {
        uint64_t rest = at - sc.excl;
        int s = tid * KEEP;
        while (rest >= mine[s]) rest -= mine[s++];  // (the thread's sums are more than rest)
        found_seg = s;
        found_left = rest;
    }
    __syncthreads();
    if (warp || found_seg < 0) return;
    uint64_t rest = found_left;
    constexpr int E = PER_LANE<T, PIECE>;
    for (int i = 0; i < a.pieces; ++i) {  // PER_LANE elements a lane, in order
        const int64_t e = ((int64_t)found_seg * a.pieces + i) * PER_PIECE<T, PIECE> + lane * E - row.skip;
        const int k0 = (int)max((int64_t)0, min((int64_t)a.V, e)), k1 = (int)max((int64_t)0, min((int64_t)a.V, e + E));
        uint64_t sum = 0;
#pragma unroll
        for (int k = 0; k < E; ++k)
            if (k0 + k < k1) sum += row.weight(k0 + k);
        const uint64_t in = warp_scan(sum, lane), total = __shfl_sync(0xffffffffu, in, 31);
        if (rest < total) {
            // the lane that holds the place; its elements, one to a lane
            const int who = __ffs(__ballot_sync(0xffffffffu, rest < in)) - 1;
            const uint64_t left = rest - __shfl_sync(0xffffffffu, in - sum, who);
            const int k = __shfl_sync(0xffffffffu, k0, who) + lane, end = __shfl_sync(0xffffffffu, k1, who);
            const uint64_t to = warp_scan(k < end ? row.weight(k) : 0, lane);
            const int j = __ffs(__ballot_sync(0xffffffffu, left < to)) - 1;
            if (lane == j) a.out[(int64_t)n * a.W + t.acc] = k;
            return;
        }
        rest -= total;
    }
}

// Small pieces up to four for each warp of a full card (a constant, so that the workspace's size does not
// depend on the device).  Segments of a request: pieces, two, four .. of them where a row has over
// MAX_SEGS (places, which count from the 16 bytes that a row begins in, go up to V + 7).
constexpr int64_t SMALL_BYTES = (int64_t)4 * 152 * BLOCKS * WARPS * SMALL;
struct VerifyPlan {
    int piece, pieces, segs;
};
VerifyPlan plan_verify(int N, int V, int es) {
    VerifyPlan p;
    p.piece = (int64_t)N * V * es <= SMALL_BYTES ? SMALL : LARGE;
    p.pieces = 1;
    auto segs = [&] {
        const int64_t n = (int64_t)p.pieces * (p.piece / es);
        return ((int64_t)V + 7 + n - 1) / n;
    };
    while (segs() > MAX_SEGS) p.pieces *= 2;
    p.segs = (int)segs();
    return p;
}
// Fewer requests may take small pieces and then have more segments: the most segments of a call of up to N requests
// (28 requests of 131,072 fp32 tokens have 14,364, 29 have 7,453), so that one workspace serves a shrinking batch.
int64_t most_segments(int N, int V, int es) {
    const VerifyPlan p = plan_verify(N, V, es);
    const int64_t small = std::min<int64_t>(N, SMALL_BYTES / ((int64_t)V * es));  // requests that take small pieces
    return small < 1 ? (int64_t)N * p.segs : std::max((int64_t)N * p.segs, small * plan_verify((int)small, V, es).segs);
}
template <typename T, int PIECE> int launch_verify(const VerifyArgs &a, cudaStream_t s) {
    constexpr int SMEM = WARPS * STAGES * ROOM_OF<PIECE>;
    const int rc = prepare_kernel((const void *)verify_sums_kernel<T, PIECE>, SMEM, THREADS, nullptr);
    if (rc) return rc;
    // (no block without a segment for each of its warps)
    const int64_t line = (int64_t)a.N * a.segs, most = (int64_t)BLOCKS * device_sm_count(), blocks = (line + WARPS - 1) / WARPS;
    verify_sums_kernel<T, PIECE><<<(unsigned)(blocks < most ? blocks : most), THREADS, SMEM, s>>>(a);
    note_launch("verify_sums", s);
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at;
    cfg.gridDim = dim3((unsigned)a.N);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_place_kernel<T, PIECE>, a);
    note_launch("verify_place", s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_verify_drafts_workspace_size(int N, int W, int V, int dtype) {
    if (N < 1 || N > MAX_N || W < 1 || W > MAX_W || V < 1 || V > MAX_V || (dtype != KDA_F32 && dtype != KDA_BF16)) return 0;
    return (size_t)most_segments(N, V, dtype == KDA_BF16 ? 2 : 4) * sizeof(uint64_t);
}

int kda_verify_drafts(const void *target, const void *draft, const int32_t *draft_tokens, const float *uniforms,
                      const int32_t *n_draft, int N, int W, int V, int dtype, int64_t target_seq_stride,
                      int64_t target_row_stride, int64_t draft_seq_stride, int64_t draft_row_stride, int32_t *num_accepted,
                      int32_t *tokens, void *workspace, size_t workspace_bytes, int32_t *error_word, kda_stream_t stream) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_INVALID_ARG;
    if (N < 1 || W < 1 || V < 1) return KDA_ERR_INVALID_ARG;
    if (W > MAX_W || N > MAX_N || V > MAX_V) return KDA_ERR_UNSUPPORTED;
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
    const VerifyPlan p = plan_verify(N, V, es);
    const VerifyArgs a{target, draft, draft_tokens, n_draft, uniforms, num_accepted, tokens, error_word, (uint64_t *)workspace,
                       target_seq_stride, target_row_stride, draft_seq_stride, draft_row_stride, N, W, V, p.pieces, p.segs};
    if (!workspace || workspace_bytes < (size_t)N * p.segs * sizeof(uint64_t) || ((uintptr_t)workspace & 7u)) return KDA_ERR_WORKSPACE;
    cudaStream_t s = (cudaStream_t)stream;
    note_begin(s);
    if (dtype == KDA_F32) return p.piece == SMALL ? launch_verify<float, SMALL>(a, s) : launch_verify<float, LARGE>(a, s);
    return p.piece == SMALL ? launch_verify<__nv_bfloat16, SMALL>(a, s) : launch_verify<__nv_bfloat16, LARGE>(a, s);
}

}  // extern "C"
