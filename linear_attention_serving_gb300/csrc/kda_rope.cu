// kda_rope.cu -- rotary positions and per-head norms of queries and keys
// (kda_qk_rope), and the same with keys and values written into their pages
// (kda_paged_rope_append); kda_rope_frequencies on the host.
//
// One pass: a row (token, head) of 128 channels is held by 16 lanes, 8 channels each,
// and read and written once.  A lane's channels are two chunks of four chosen so that
// both halves of its four pairs are its own: chunks l and l + rot / 8 (half layout),
// 2 l and 2 l + 1 (interleaved), so turning needs no exchange between lanes; the norm
// takes four shuffles.
//
// Angles.  f is a fraction of a turn in 64-bit fixed point, so position * f modulo 2^64
// is the exact angle modulo a turn (fp32 products lose whole radians at positions of
// a million).  Its nearest quarter turn is taken off in integers, and what is left, at most
// an eighth of a turn, rounded to fp32: off by at most 2^-27 half turns, under 2^-25 radians.
// The sines and cosines of a token are worked out once, in shared memory, for all its heads
// (by each unit for itself where a unit has a token of its own), and multiplied with the norms'
// weights once for each kind of row, so that a row costs a scale and two packed products and
// sums for each two channels.
//
// Bound by HBM once there are some thousand tokens, by the launch and the chain position, angle,
// row below: 23,100 packed tokens of 32 + 2 x 8 heads (bf16, norms) into their pages 89 us, 6.4
// TB/s; 9,300 of 16 + 16 heads (fp32) 48 us, 6.3 TB/s; 1,280 tokens into an e4m3 cache 9.6 us; one
// token 2.8 us.  Two rows a unit in flight and two ahead of them, 64 registers: with four
// of each, 80 registers and three blocks an SM, the first was 92 to 109 us; with rows of all
// kinds in one stream of batches, 111.
#include <cuda_fp8.h>

#include <cmath>

#include "kda_internal.cuh"

namespace kda {

int check_paged_cache(int Hkv, int Dm, int dtype, int cache_dtype, const float *k_scale, const float *v_scale,
                      const void *k_cache, const void *v_cache, int n_pages, int page_size, int64_t page_stride);

namespace {

constexpr int THREADS = 256, UNITS = THREADS / 16;  // a unit of 16 lanes takes a row at a time
constexpr int PAIRS = D / 2;
constexpr int SOME = 2, MANY = 3, EACH = 4;         // tokens of a block (their logarithm; EACH: one for each unit)

enum { TO_ROWS = 0, TO_PAGES = 1, TO_E4M3 = 2 };

struct RopeArgs {
    const void *q, *k, *v;
    void *q_out, *k_out;                 // k_out: rows, or the cache of keys
    void *v_cache;
    const int32_t *positions;
    const int64_t *freq, *slot_map;
    const float *q_weight, *k_weight, *k_scale, *v_scale;
    int32_t *err;
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;  // elements
    int64_t page_stride, n_slots;
    int T, Hq, Hkv, rot, page_size, rows_per_y;
    float amplitude, eps;
};

// Two fp32 operations at once.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t r) {
    float2 x;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x.x), "=f"(x.y) : "l"(r));
    return x;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}

// Eight channels of a row, two chunks of four (c0 and c1), as they are held; and as four packed
// pairs of neighbours (a lane's pair i of y is channels 2 i, 2 i + 1 of the eight).
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint2 a, b;
    template <bool JOINED> __device__ __forceinline__ void load(const void *row, int c0, int c1) {
        if constexpr (JOINED) {
            const uint4 x = *(reinterpret_cast<const uint4 *>(row) + (c0 >> 1));
            a = make_uint2(x.x, x.y);
            b = make_uint2(x.z, x.w);
        } else {
            a = *(reinterpret_cast<const uint2 *>(row) + c0);
            b = *(reinterpret_cast<const uint2 *>(row) + c1);
        }
    }
    template <bool JOINED> __device__ __forceinline__ void store(void *row, int c0, int c1) const {
        if constexpr (JOINED) {
            *(reinterpret_cast<uint4 *>(row) + (c0 >> 1)) = make_uint4(a.x, a.y, b.x, b.y);
        } else {
            *(reinterpret_cast<uint2 *>(row) + c0) = a;
            *(reinterpret_cast<uint2 *>(row) + c1) = b;
        }
    }
    __device__ __forceinline__ void get(uint64_t *y) const {
        const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    __device__ __forceinline__ void set(const uint64_t *y) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(y[i]);
            const __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
            w[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
        a = make_uint2(w[0], w[1]);
        b = make_uint2(w[2], w[3]);
    }
};
template <> struct Eight<float> {
    float4 a, b;
    template <bool JOINED> __device__ __forceinline__ void load(const void *row, int c0, int c1) {
        a = *(reinterpret_cast<const float4 *>(row) + c0);
        b = *(reinterpret_cast<const float4 *>(row) + c1);
    }
    template <bool JOINED> __device__ __forceinline__ void store(void *row, int c0, int c1) const {
        *(reinterpret_cast<float4 *>(row) + c0) = a;
        *(reinterpret_cast<float4 *>(row) + c1) = b;
    }
    __device__ __forceinline__ void get(uint64_t *y) const {
        y[0] = pack2(a.x, a.y), y[1] = pack2(a.z, a.w), y[2] = pack2(b.x, b.y), y[3] = pack2(b.z, b.w);
    }
    __device__ __forceinline__ void set(const uint64_t *y) {
        const float2 p = unpack2(y[0]), q = unpack2(y[1]), r = unpack2(y[2]), t = unpack2(y[3]);
        a = make_float4(p.x, p.y, q.x, q.y);
        b = make_float4(r.x, r.y, t.x, t.y);
    }
};

// x / scale in fp32, then one rounding to e4m3 (a true division: a product with 1 / scale
// would round twice and move values across a border)
__device__ __forceinline__ uint32_t e4m3_4(const uint64_t *y, float scale) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 x = unpack2(y[i]);
        const __nv_fp8x2_storage_t b =
            __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x.x, scale), __fdiv_rn(x.y, scale)), __NV_SATFINITE, __NV_E4M3);
        r |= (uint32_t)b << (16 * i);
    }
    return r;
}

// Cosine and sine of position * f, by the exact angle modulo a turn.
__device__ __forceinline__ float2 turn_of(int pos, int64_t f, float amplitude) {
    const uint64_t phase = (uint64_t)(int64_t)pos * (uint64_t)f;
    const uint32_t t = (uint32_t)((phase + (1ull << 31)) >> 32);  // turns * 2^32
    const uint32_t quarter = (t + (1u << 29)) >> 30;              // 0 .. 3, the nearest
    const int rest = (int)(t - (quarter << 30));                  // at most an eighth of a turn either way
    float s, c;
    sincospif((float)rest * 0x1p-31f, &s, &c);
    const float x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s;
    return quarter & 2 ? make_float2(-x * amplitude, -y * amplitude) : make_float2(x * amplitude, y * amplitude);
}

// What a lane multiplies its channels by, from the weights w (NULL: ones) and the token's angles:
//   lanes that turn: y0 <- y0 m[0] + y1 n[0] ..: the pair (a, b) of weights (u, v) becomes
//   (a (u c) - b (v s), a (u s) + b (v c)), four numbers for each pair; others: y <- y m.
struct Turn {
    uint64_t m[4], n[4];
    template <bool INTER> __device__ __forceinline__ void set(const float *w, const float2 *turn, bool turns, int c0, int c1) {
        float4 u = make_float4(1.f, 1.f, 1.f, 1.f), v = u;
        if (w) {
            u = __ldg(reinterpret_cast<const float4 *>(w) + c0);
            v = __ldg(reinterpret_cast<const float4 *>(w) + c1);
        }
        m[0] = pack2(u.x, u.y), m[1] = pack2(u.z, u.w), m[2] = pack2(v.x, v.y), m[3] = pack2(v.z, v.w);
        if (!turns) return;
        const float4 p = reinterpret_cast<const float4 *>(turn)[0], q = reinterpret_cast<const float4 *>(turn)[1];
        if constexpr (INTER) {  // pairs (0, 1), (2, 3), ..: y + its swap
            n[0] = pack2(-u.y * p.y, u.x * p.y), n[1] = pack2(-u.w * p.w, u.z * p.w);
            n[2] = pack2(-v.y * q.y, v.x * q.y), n[3] = pack2(-v.w * q.w, v.z * q.w);
            m[0] = pack2(u.x * p.x, u.y * p.x), m[1] = pack2(u.z * p.z, u.w * p.z);
            m[2] = pack2(v.x * q.x, v.y * q.x), m[3] = pack2(v.z * q.z, v.w * q.z);
        } else {                // pairs (0, 4), (1, 5), ..
            n[0] = pack2(-v.x * p.y, -v.y * p.w), n[1] = pack2(-v.z * q.y, -v.w * q.w);
            n[2] = pack2(u.x * p.y, u.y * p.w), n[3] = pack2(u.z * q.y, u.w * q.w);
            m[0] = pack2(u.x * p.x, u.y * p.z), m[1] = pack2(u.z * q.x, u.w * q.z);
            m[2] = pack2(v.x * p.x, v.y * p.z), m[3] = pack2(v.z * q.x, v.w * q.z);
        }
    }
    template <bool INTER> __device__ __forceinline__ void apply(uint64_t *y, bool turns) const {
        if (!turns) {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], m[i]);
        } else if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2(y[i]);
                y[i] = fma2(y[i], m[i], mul2(pack2(f.y, f.x), n[i]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint64_t a = y[i], b = y[i + 2];
                y[i] = fma2(a, m[i], mul2(b, n[i]));
                y[i + 2] = fma2(b, m[i + 2], mul2(a, n[i + 2]));
            }
        }
    }
};

// Rows of a unit in flight (two batches of them: the next one's loads are issued before this one is worked on).
template <typename T> constexpr int AHEAD = sizeof(T) == 2 ? 2 : 1;

// `n` rows of one kind, `step` elements apart in `in` and `out_step` in `out`: normed (where w), turned
// (TURN) and stored; E4M3: as x / scale, the rows' scales `scale_step` apart.  x: the first batch.
template <typename T, bool INTER>
__device__ __forceinline__ void first_rows(Eight<T> (&x)[AHEAD<T>], const T *in, int step, int n, int c0, int c1) {
#pragma unroll
    for (int i = 0; i < AHEAD<T>; ++i)
        if (i < n) x[i].template load<INTER>(in + i * step, c0, c1);
}
template <typename T, bool INTER, bool TURN, bool E4M3>
__device__ __forceinline__ void unit_rows(Eight<T> (&x)[AHEAD<T>], const T *in, int step, char *out, int64_t out_step, int n, bool w,
                                          float eps, const Turn &tm, bool turns, int c0, int c1, uint32_t lanes, const float *scale,
                                          int scale_step) {
    constexpr int N = AHEAD<T>;
    Eight<T> next[N];
    for (; n > 0; n -= N) {
        in += N * step;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i + N < n) next[i].template load<INTER>(in + i * step, c0, c1);
        float f[N];
        if (TURN && w) {  // the norms of the batch's rows side by side
#pragma unroll
            for (int i = 0; i < N; ++i) {
                uint64_t y[4], ss;
                x[i].get(y);
                ss = mul2(y[0], y[0]);
#pragma unroll
                for (int e = 1; e < 4; ++e) ss = fma2(y[e], y[e], ss);
                const float2 s = unpack2(ss);
                f[i] = s.x + s.y;
            }
#pragma unroll
            for (int o = 8; o; o >>= 1)
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] += __shfl_xor_sync(lanes, f[i], o);
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = rsqrtf(fmaf(f[i], 1.f / D, eps));
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint64_t y[4];
            if (TURN || E4M3) x[i].get(y);
            if (TURN) {
                if (w) {
                    const uint64_t f2 = pack2(f[i], f[i]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], f2);
                }
                tm.apply<INTER>(y, turns);
            }
            if (i < n) {
                if constexpr (E4M3) {
                    const float sc = __ldg(scale + i * scale_step);
                    const uint32_t lo = e4m3_4(y, sc), hi = e4m3_4(y + 2, sc);
                    if constexpr (INTER) {
                        *(reinterpret_cast<uint2 *>(out) + (c0 >> 1)) = make_uint2(lo, hi);
                    } else {
                        *(reinterpret_cast<uint32_t *>(out) + c0) = lo;
                        *(reinterpret_cast<uint32_t *>(out) + c1) = hi;
                    }
                } else {
                    if (TURN) x[i].set(y);
                    x[i].template store<INTER>(out, c0, c1);
                }
            }
            out += out_step;
        }
        if (E4M3) scale += N * scale_step;
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = next[i];
    }
}

// LOG: a block takes 1 << LOG tokens, each by UNITS >> LOG units.
template <typename T, int TO, bool INTER, int LOG>
__global__ void __launch_bounds__(THREADS, 4) rope_kernel(const RopeArgs a) {
    constexpr int PER = UNITS >> LOG;  // units of a token: each takes every PER-th row
    __shared__ __align__(16) float2 turn[LOG == EACH ? 1 : 1 << LOG][PAIRS];
    __align__(16) float2 own[4];
    const float2 *angles = own;
    const int tid = threadIdx.x, l = tid & 15, unit = tid >> 4;
    const int mine = unit / PER, t0 = blockIdx.x << LOG, tok = t0 + mine;
    // this lane's chunks of four channels; lanes under rot / 8 hold pairs 4 l .. 4 l + 3
    const int turning = a.rot >> 3;
    const bool turns = l < turning, live = tok < a.T;
    const int c0 = INTER ? 2 * l : turns ? l : 2 * l, c1 = INTER ? c0 + 1 : turns ? l + turning : 2 * l + 1;
    const int r0 = blockIdx.y * a.rows_per_y + (unit - mine * PER), r1 = (blockIdx.y + 1) * a.rows_per_y;
    // the unit's rows among the block's, up to r1, of queries, keys and values, one kind after the other
    auto first = [&](int from) { return r0 >= from ? r0 - from : (PER - 1) & (r0 - from); };  // within a kind that begins at `from`
    auto count = [&](int f, int from, int rows) { return live ? (min(rows, r1 - from) - f + PER - 1) / PER : 0; };
    // the first queries are on their way while the angles are worked out
    const int hq = first(0), nq = count(hq, 0, a.Hq);
    const T *q = (const T *)a.q + (int64_t)tok * a.q_stride + hq * D;
    Eight<T> x[AHEAD<T>];
    first_rows<T, INTER>(x, q, PER * D, nq, c0, c1);
    // the tokens' angles
    if constexpr (LOG == EACH) {
        if (live && turns) {
            const int pos = a.positions[tok];
#pragma unroll
            for (int i = 0; i < 4; ++i) own[i] = turn_of(pos, a.freq[4 * l + i], a.amplitude);
        }
    } else {
        const int pairs = a.rot >> 1;
        for (int i = tid; i < (pairs << LOG); i += THREADS) {
            const int w = i / pairs, p = i - w * pairs;
            if (t0 + w < a.T) turn[w][p] = turn_of(a.positions[t0 + w], a.freq[p], a.amplitude);
        }
        angles = turn[mine] + 4 * l;
    }
    int64_t page = -1;
    int off = 0;
    if (TO != TO_ROWS && live) {
        const int64_t slot = a.slot_map[tok];
        if (slot >= a.n_slots) {
            if (unit == mine * PER && l == 0 && blockIdx.y == 0 && a.err) atomicOr(a.err, KDA_DEVERR_PAGE);
        } else if (slot >= 0) {
            if (a.n_slots <= (int64_t)UINT32_MAX) {
                page = (uint32_t)slot / (uint32_t)a.page_size;
                off = (int)((uint32_t)slot - (uint32_t)page * (uint32_t)a.page_size);
            } else {
                page = slot / a.page_size;
                off = (int)(slot - page * a.page_size);
            }
        }
    }
    if (LOG != EACH) __syncthreads();
    if (!live) return;
    const uint32_t lanes = tid & 16 ? 0xffff0000u : 0x0000ffffu;  // (shuffles stay among a unit's lanes)
    constexpr int ES = (int)sizeof(T);
    Turn tm;
    if (nq > 0) {
        tm.set<INTER>(a.q_weight, angles, turns, c0, c1);
        unit_rows<T, INTER, true, false>(x, q, PER * D, (char *)a.q_out + ((int64_t)tok * a.q_out_stride + hq * D) * ES, PER * D * ES, nq,
                                         a.q_weight, a.eps, tm, turns, c0, c1, lanes, nullptr, 0);
    }
    if (TO != TO_ROWS && page < 0) return;
    constexpr bool E4 = TO == TO_E4M3;
    constexpr int CS = E4 ? 1 : ES;
    const int h = first(a.Hq), n = count(h, a.Hq, a.Hkv);
    if (n > 0) {
        tm.set<INTER>(a.k_weight, angles, turns, c0, c1);
        const T *in = (const T *)a.k + (int64_t)tok * a.k_stride + h * D;
        first_rows<T, INTER>(x, in, PER * D, n, c0, c1);
        if constexpr (TO == TO_ROWS)
            unit_rows<T, INTER, true, false>(x, in, PER * D, (char *)a.k_out + ((int64_t)tok * a.k_out_stride + h * D) * ES, PER * D * ES, n,
                                             a.k_weight, a.eps, tm, turns, c0, c1, lanes, nullptr, 0);
        else
            unit_rows<T, INTER, true, E4>(x, in, PER * D, (char *)a.k_out + (page * a.page_stride + ((int64_t)h * a.page_size + off) * D) * CS,
                                          (int64_t)PER * a.page_size * D * CS, n, a.k_weight, a.eps, tm, turns, c0, c1, lanes,
                                          E4 ? a.k_scale + h : nullptr, PER);
    }
    if constexpr (TO != TO_ROWS) {
        const int from = a.Hq + a.Hkv, g = first(from), m = count(g, from, a.Hkv);
        const T *in = (const T *)a.v + (int64_t)tok * a.v_stride + g * D;
        first_rows<T, INTER>(x, in, PER * D, m, c0, c1);
        unit_rows<T, INTER, false, E4>(x, in, PER * D,
                                       (char *)a.v_cache + (page * a.page_stride + ((int64_t)g * a.page_size + off) * D) * CS,
                                       (int64_t)PER * a.page_size * D * CS, m, false, a.eps, tm, turns, c0, c1, lanes,
                                       E4 ? a.v_scale + g : nullptr, PER);
    }
}

template <typename T, int TO>
void launch_rope(const RopeArgs &a, bool inter, int log, dim3 grid, cudaStream_t s) {
    auto go = [&](auto kernel) { kernel<<<grid, THREADS, 0, s>>>(a); };
    if (inter)
        go(log == EACH ? rope_kernel<T, TO, true, EACH> : log == MANY ? rope_kernel<T, TO, true, MANY> : log == SOME ? rope_kernel<T, TO, true, SOME> : rope_kernel<T, TO, true, 0>);
    else
        go(log == EACH ? rope_kernel<T, TO, false, EACH> : log == MANY ? rope_kernel<T, TO, false, MANY> : log == SOME ? rope_kernel<T, TO, false, SOME> : rope_kernel<T, TO, false, 0>);
}

// What both calls check.
int check_rope(const void *q, const void *k, const int32_t *positions, const int64_t *freq, float amplitude,
               const float *q_weight, const float *k_weight, float eps, int64_t T, int Hq, int Hkv, int Dm, int rot,
               int layout, int dtype, int64_t q_stride, int64_t k_stride, const void *q_out, int64_t q_out_stride) {
    if (Dm != D) return KDA_ERR_UNSUPPORTED;
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_INVALID_ARG;
    if (layout != KDA_ROPE_HALF && layout != KDA_ROPE_INTERLEAVED) return KDA_ERR_INVALID_ARG;
    if (rot < 0 || rot > D) return KDA_ERR_INVALID_ARG;
    if (rot % 8) return KDA_ERR_UNSUPPORTED;
    if (T < 0 || T >= (int64_t)INT32_MAX - THREADS || Hq < 1 || Hkv < 1 || Hq > (1 << 20) || Hkv > (1 << 20))
        return KDA_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || eps > 1e30f || !(fabsf(amplitude) <= 1e30f)) return KDA_ERR_INVALID_ARG;
    const int per16 = dtype == KDA_BF16 ? 8 : 4;
    if (q_stride < (int64_t)Hq * D || k_stride < (int64_t)Hkv * D || q_out_stride < (int64_t)Hq * D) return KDA_ERR_INVALID_ARG;
    if (q_stride % per16 || k_stride % per16 || q_out_stride % per16) return KDA_ERR_INVALID_ARG;
    if (T > 0 && (!q || !k || !q_out || (rot > 0 && (!positions || !freq)))) return KDA_ERR_INVALID_ARG;
    for (const void *p : {q, k, q_out, (const void *)q_weight, (const void *)k_weight, (const void *)freq})
        if ((uintptr_t)p & 15u) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// Tokens of a block (their logarithm) and blocks of a token.
dim3 rope_grid(RopeArgs &a, int rows, int &log) {
    const int sms = device_sm_count();
    log = 0;
    a.rows_per_y = rows;
    int y = 1;
    if (a.T >= 16 * sms) {
        // Few rows: a unit works its token's angles out alone and waits for no other (20,000 tokens of 20 rows 41
        // us, of 24 46, of 6 16; eight tokens to a block 46, 47 and 26).  With 48 rows there are too few units
        // left to fill the last wave (81 us eight tokens to a block, 87 one to a unit).
        log = rows <= 24 ? EACH : MANY;
    } else if (a.T >= 4 * sms) {  // (1,280 tokens of 48 rows, bf16 and e4m3 caches: 8.3 and 9.6 us; 11.0 and 11.9 a block to each, 10.2 and 12.1 eight to a block)
        log = SOME;
    } else {
        // a block to a token, or several to one where there are few: a row for each unit
        while (y * UNITS < rows && (int64_t)a.T * y < sms) ++y;
        a.rows_per_y = (rows + y - 1) / y;
    }
    return dim3((unsigned)((a.T + (1 << log) - 1) >> log), (unsigned)y);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

int kda_rope_frequencies(int rot_dim, double base, int scaling, double factor, double original_len, double beta_fast,
                         double beta_slow, int64_t *freq, float *amplitude) {
    if (rot_dim < 8 || rot_dim > D) return KDA_ERR_INVALID_ARG;
    if (rot_dim % 8) return KDA_ERR_UNSUPPORTED;
    if (!(base > 1.0) || !std::isfinite(base) || !freq || !amplitude) return KDA_ERR_INVALID_ARG;
    if (scaling < KDA_ROPE_NONE || scaling > KDA_ROPE_YARN) return KDA_ERR_INVALID_ARG;
    if (scaling != KDA_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return KDA_ERR_INVALID_ARG;
    if (scaling == KDA_ROPE_YARN &&
        (!(original_len > 0.0) || !std::isfinite(original_len) || !(beta_slow >= 0.0) || !(beta_fast > beta_slow) ||
         !std::isfinite(beta_fast)))
        return KDA_ERR_INVALID_ARG;
    const double turn = 6.283185307179586476925;
    if (scaling == KDA_ROPE_NTK) base *= pow(factor, (double)rot_dim / (rot_dim - 2));
    if (!std::isfinite(base)) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / rot_dim);
        if (scaling == KDA_ROPE_LINEAR) f /= factor;
        if (scaling == KDA_ROPE_YARN) {
            double g = (original_len * f / turn - beta_slow) / (beta_fast - beta_slow);
            g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
            f = f * (g + (1.0 - g) / factor);
        }
        freq[i] = (int64_t)llrint(f / turn * 0x1p64);  // (f <= 1: under 2^62)
    }
    *amplitude = scaling == KDA_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    return KDA_OK;
}

int kda_qk_rope(const void *q, const void *k, const int32_t *positions, const int64_t *freq, float amplitude,
                const float *q_weight, const float *k_weight, float eps, int64_t T_total, int Hq, int Hkv, int Dm,
                int rot_dim, int layout, int dtype, int64_t q_stride, int64_t k_stride, void *q_out, void *k_out,
                int64_t q_out_stride, int64_t k_out_stride, kda_stream_t stream) {
    const int rc = check_rope(q, k, positions, freq, amplitude, q_weight, k_weight, eps, T_total, Hq, Hkv, Dm, rot_dim, layout,
                              dtype, q_stride, k_stride, q_out, q_out_stride);
    if (rc) return rc;
    if (k_out_stride < (int64_t)Hkv * D || k_out_stride % (dtype == KDA_BF16 ? 8 : 4) || ((uintptr_t)k_out & 15u) ||
        (T_total > 0 && !k_out))
        return KDA_ERR_INVALID_ARG;
    // in place only over the same rows: another row may be read after this one is written
    if (T_total == 0) return KDA_OK;
    if ((q_out == q && q_out_stride != q_stride) || (k_out == k && k_out_stride != k_stride) || q_out == k || k_out == q ||
        q_out == k_out)
        return KDA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    note_begin(s);
    RopeArgs a = {};
    a.q = q, a.k = k, a.q_out = q_out, a.k_out = k_out;
    a.positions = positions, a.freq = freq, a.q_weight = q_weight, a.k_weight = k_weight;
    a.q_stride = q_stride, a.k_stride = k_stride, a.q_out_stride = q_out_stride, a.k_out_stride = k_out_stride;
    a.T = (int)T_total, a.Hq = Hq, a.Hkv = Hkv, a.rot = rot_dim, a.amplitude = amplitude, a.eps = eps;
    int log;
    const dim3 grid = rope_grid(a, Hq + Hkv, log);
    // (without rotation a lane's channels lie side by side)
    const bool inter = layout == KDA_ROPE_INTERLEAVED || rot_dim == 0;
    if (dtype == KDA_BF16)
        launch_rope<__nv_bfloat16, TO_ROWS>(a, inter, log, grid, s);
    else
        launch_rope<float, TO_ROWS>(a, inter, log, grid, s);
    note_launch("qk_rope", s);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int kda_paged_rope_append(const void *q, const void *k, const void *v, const int32_t *positions,
                          const int64_t *slot_map, const int64_t *freq, float amplitude, const float *q_weight,
                          const float *k_weight, float eps, int64_t T_total, int Hq, int Hkv, int Dm, int rot_dim,
                          int layout, int dtype, int cache_dtype, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                          void *q_out, int64_t q_out_stride, const float *k_scale, const float *v_scale, void *k_cache,
                          void *v_cache, int n_pages, int page_size, int64_t page_stride, int32_t *error_word,
                          kda_stream_t stream) {
    int rc = check_rope(q, k, positions, freq, amplitude, q_weight, k_weight, eps, T_total, Hq, Hkv, Dm, rot_dim, layout, dtype,
                        q_stride, k_stride, q_out, q_out_stride);
    if (rc) return rc;
    rc = check_paged_cache(Hkv, Dm, dtype, cache_dtype, k_scale, v_scale, k_cache, v_cache, n_pages, page_size, page_stride);
    if (rc) return rc;
    if (v_stride < (int64_t)Hkv * D || v_stride % (dtype == KDA_BF16 ? 8 : 4) || ((uintptr_t)v & 15u)) return KDA_ERR_INVALID_ARG;
    if (T_total > 0 && (!v || !slot_map)) return KDA_ERR_INVALID_ARG;
    if (T_total == 0) return KDA_OK;
    if ((q_out == q && q_out_stride != q_stride) || q_out == k || q_out == v) return KDA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    note_begin(s);
    RopeArgs a = {};
    a.q = q, a.k = k, a.v = v, a.q_out = q_out, a.k_out = k_cache, a.v_cache = v_cache;
    a.positions = positions, a.freq = freq, a.slot_map = slot_map, a.q_weight = q_weight, a.k_weight = k_weight;
    a.k_scale = k_scale, a.v_scale = v_scale, a.err = error_word;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride, a.q_out_stride = q_out_stride;
    a.page_stride = page_stride, a.n_slots = (int64_t)n_pages * page_size;
    a.T = (int)T_total, a.Hq = Hq, a.Hkv = Hkv, a.rot = rot_dim, a.page_size = page_size;
    a.amplitude = amplitude, a.eps = eps;
    int log;
    const dim3 grid = rope_grid(a, Hq + 2 * Hkv, log);
    const bool inter = layout == KDA_ROPE_INTERLEAVED || rot_dim == 0;
    if (cache_dtype == KDA_E4M3)
        launch_rope<__nv_bfloat16, TO_E4M3>(a, inter, log, grid, s);
    else if (dtype == KDA_BF16)
        launch_rope<__nv_bfloat16, TO_PAGES>(a, inter, log, grid, s);
    else
        launch_rope<float, TO_PAGES>(a, inter, log, grid, s);
    note_launch("paged_rope_append", s);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
