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
// A block works the sines and cosines of its tokens out once, in shared memory, for all
// their heads.
#include <cuda_fp8.h>

#include <cmath>

#include "kda_internal.cuh"

namespace kda {

int check_paged_cache(int Hkv, int Dm, int dtype, int cache_dtype, const float *k_scale, const float *v_scale,
                      const void *k_cache, const void *v_cache, int n_pages, int page_size, int64_t page_stride);

namespace {

constexpr int THREADS = 256, UNITS = THREADS / 16;  // a unit of 16 lanes takes a row at a time
constexpr int AHEAD = 4;                            // rows of a unit in flight
constexpr int PAIRS = D / 2;

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
    int T, Hq, Hkv, rot, page_size, tok_log, rows_per_y;
    float amplitude, eps;
};

// Eight channels of a row: chunks of four, c0 and c1.
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
    __device__ __forceinline__ void get(float *x) const {
        const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float *x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
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
    __device__ __forceinline__ void get(float *x) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ __forceinline__ void set(const float *x) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
};

// x / scale in fp32, then one rounding to e4m3 (a true division: a product with 1 / scale
// would round twice and move values across a border)
__device__ __forceinline__ uint32_t e4m3_4(const float *x, float scale) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __nv_fp8x2_storage_t b = __nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale)), __NV_SATFINITE, __NV_E4M3);
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

template <typename T, int TO, bool INTER>
__global__ void __launch_bounds__(THREADS) rope_kernel(const RopeArgs a) {
    __shared__ float2 turn[UNITS][PAIRS];
    const int tid = threadIdx.x, l = tid & 15, unit = tid >> 4;
    const int per_tok = UNITS >> a.tok_log;  // units of one token
    const int mine = unit / per_tok, step0 = unit - mine * per_tok;
    const int t0 = blockIdx.x << a.tok_log, tok = t0 + mine;
    const int rows = a.Hq + (TO == TO_ROWS ? 1 : 2) * a.Hkv;
    const int r0 = blockIdx.y * a.rows_per_y, r1 = min(rows, r0 + a.rows_per_y);
    const bool live = tok < a.T;
    // this lane's chunks of four channels; lanes under `turning` hold pairs 4 l .. 4 l + 3
    const int turning = a.rot >> 3;
    const int c0 = INTER ? 2 * l : l < turning ? l : 2 * l, c1 = INTER ? c0 + 1 : l < turning ? l + turning : 2 * l + 1;

    auto source = [&](int r) -> const void * {
        const T *p = r < a.Hq ? (const T *)a.q + (int64_t)tok * a.q_stride + r * D
                     : r < a.Hq + a.Hkv ? (const T *)a.k + (int64_t)tok * a.k_stride + (r - a.Hq) * D
                                        : (const T *)a.v + (int64_t)tok * a.v_stride + (r - a.Hq - a.Hkv) * D;
        return p;
    };
    Eight<T> x[AHEAD];
    auto load = [&](int base) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int r = base + i * per_tok;
            if (live && r < r1) x[i].template load<INTER>(source(r), c0, c1);
        }
    };
    load(r0 + step0);
    // the tokens' angles, meanwhile
    const int pairs = a.rot >> 1;
    for (int i = tid; i < (pairs << a.tok_log); i += THREADS) {
        const int w = i / pairs, p = i - w * pairs;
        if (t0 + w < a.T) turn[w][p] = turn_of(a.positions[t0 + w], a.freq[p], a.amplitude);
    }
    int64_t page = -1;
    int off = 0;
    if (TO != TO_ROWS && live) {
        const int64_t slot = a.slot_map[tok];
        if (slot >= a.n_slots) {
            if (unit == mine * per_tok && l == 0 && blockIdx.y == 0 && a.err) atomicOr(a.err, KDA_DEVERR_PAGE);
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
    __syncthreads();
    if (!live) return;  // (a whole unit: shuffles stay among its 16 lanes)
    const uint32_t lanes = tid & 16 ? 0xffff0000u : 0x0000ffffu;
    float2 cs[4];
    if (l < turning) {
#pragma unroll
        for (int i = 0; i < 4; ++i) cs[i] = turn[mine][4 * l + i];
    }
    for (int base = r0 + step0; base < r1; base += AHEAD * per_tok) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int r = base + i * per_tok;
            if (r >= r1) break;
            const bool is_q = r < a.Hq, is_v = TO != TO_ROWS && r >= a.Hq + a.Hkv;
            float y[8];
            const float *w = is_q ? a.q_weight : a.k_weight;
            if (!is_v) {
                x[i].get(y);
                if (w) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
                    for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(lanes, ss, o);
                    const float f = rsqrtf(fmaf(ss, 1.f / D, a.eps));
                    const float4 wa = __ldg(reinterpret_cast<const float4 *>(w) + c0), wb = __ldg(reinterpret_cast<const float4 *>(w) + c1);
                    y[0] *= f * wa.x, y[1] *= f * wa.y, y[2] *= f * wa.z, y[3] *= f * wa.w;
                    y[4] *= f * wb.x, y[5] *= f * wb.y, y[6] *= f * wb.z, y[7] *= f * wb.w;
                }
                if (l < turning) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int u = INTER ? 2 * e : e, v = INTER ? 2 * e + 1 : e + 4;
                        const float p = y[u], q = y[v];
                        y[u] = p * cs[e].x - q * cs[e].y;
                        y[v] = p * cs[e].y + q * cs[e].x;
                    }
                }
            } else if (TO == TO_E4M3) {
                x[i].get(y);
            }
            if (is_q) {
                x[i].set(y);
                x[i].template store<INTER>((T *)a.q_out + (int64_t)tok * a.q_out_stride + r * D, c0, c1);
            } else if (TO == TO_ROWS) {
                x[i].set(y);
                x[i].template store<INTER>((T *)a.k_out + (int64_t)tok * a.k_out_stride + (r - a.Hq) * D, c0, c1);
            } else if (page >= 0) {
                const int h = r - a.Hq - (is_v ? a.Hkv : 0);
                const int64_t at = page * a.page_stride + ((int64_t)h * a.page_size + off) * D;
                if constexpr (TO == TO_E4M3) {
                    char *row = (char *)(is_v ? a.v_cache : a.k_out) + at;
                    const float sc = is_v ? a.v_scale[h] : a.k_scale[h];
                    const uint32_t lo = e4m3_4(y, sc), hi = e4m3_4(y + 4, sc);
                    if constexpr (INTER) {
                        *(reinterpret_cast<uint2 *>(row) + l) = make_uint2(lo, hi);
                    } else {
                        *(reinterpret_cast<uint32_t *>(row) + c0) = lo;
                        *(reinterpret_cast<uint32_t *>(row) + c1) = hi;
                    }
                } else {
                    if (!is_v) x[i].set(y);
                    x[i].template store<INTER>((T *)(is_v ? a.v_cache : a.k_out) + at, c0, c1);
                }
            }
        }
        load(base + AHEAD * per_tok);
    }
}

template <typename T, int TO>
void launch_rope(const RopeArgs &a, bool inter, dim3 grid, cudaStream_t s) {
    if (inter)
        rope_kernel<T, TO, true><<<grid, THREADS, 0, s>>>(a);
    else
        rope_kernel<T, TO, false><<<grid, THREADS, 0, s>>>(a);
}

// The shape of a call, and what both calls check.
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

// Tokens of a block and blocks of a token.
dim3 rope_grid(RopeArgs &a, int rows) {
    const int sms = device_sm_count();
    a.tok_log = 0;
    a.rows_per_y = rows;
    int y = 1;
    if ((int64_t)a.T * rows >= (int64_t)sms * 8 * UNITS * 12) {
        a.tok_log = 2;
    } else {
        // a block to a token, or several to one where there are few: a row for each unit
        while (y * UNITS < rows && (int64_t)a.T * y < sms) ++y;
        a.rows_per_y = (rows + y - 1) / y;
    }
    return dim3((unsigned)((a.T + (1 << a.tok_log) - 1) >> a.tok_log), (unsigned)y);
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
    const dim3 grid = rope_grid(a, Hq + Hkv);
    // (without rotation a lane's channels lie side by side)
    const bool inter = layout == KDA_ROPE_INTERLEAVED || rot_dim == 0;
    if (dtype == KDA_BF16)
        launch_rope<__nv_bfloat16, TO_ROWS>(a, inter, grid, s);
    else
        launch_rope<float, TO_ROWS>(a, inter, grid, s);
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
    const dim3 grid = rope_grid(a, Hq + 2 * Hkv);
    const bool inter = layout == KDA_ROPE_INTERLEAVED || rot_dim == 0;
    if (cache_dtype == KDA_E4M3)
        launch_rope<__nv_bfloat16, TO_E4M3>(a, inter, grid, s);
    else if (dtype == KDA_BF16)
        launch_rope<__nv_bfloat16, TO_PAGES>(a, inter, grid, s);
    else
        launch_rope<float, TO_PAGES>(a, inter, grid, s);
    note_launch("paged_rope_append", s);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
