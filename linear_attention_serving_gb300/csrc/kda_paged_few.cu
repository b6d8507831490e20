// kda_paged_few.cu -- paged attention on tcgen05 for few rows (single tokens,
// draft windows; bf16 and e4m3 caches): NR rows of one kv head at a time, 16 where no
// request of the call can have more, else 32 (e4m3 caches; bf16 with more heads to a kv
// head than a tile of the other kernel has rows).
// Each key and value is read for few rows, so the time is the pages' bytes over HBM;
// what the kernel has to do is keep copies in flight and stay out of their way.
//
// The products are taken the other way round than for many rows, so that the 128
// lanes of TMEM are keys (and channels) and only the NR columns in use cost
// anything:
//   S^T = K Q^T    128 keys x NR fp32 in TMEM, K from shared memory as it was loaded
//   P^T = exp2(S^T scale - ref): thread = key, NR values, stored as the [key][row]
//         operand of the second product (bf16; fp16 for e4m3 caches)
//   O^T += V^T P^T 128 channels x NR fp32 in TMEM, V from shared memory as loaded
// Two groups of four softmax warps take every other tile, each with its own buffers,
// references, sums and O, merged at the item's end: one group alone needs 2,000 cycles
// a tile, nearly all of it latency, more than an e4m3 tile takes to arrive.
// Products of S, issued by one warp, run up to two tiles ahead of those of O, issued by
// another, across items.
//
// `ref` follows a row's maximum only when that has grown by more than 2^8 (kept
// probabilities are then as precise in 16 bits, sums are fp32): most tiles need no
// maximum over their keys at all, which would go across lanes, and no rescaling; one
// barrier tells a group's warps whether any of them saw such growth.
//
// e4m3 caches: S^T multiplies K as it was loaded (8-bit products) by three e5m2 parts of
// q, three bits each, which hold a bf16 value's eight bits (two e4m3 parts do so only for
// values over 2^-9 of the row's largest; the third costs 1.6% on single tokens).  V is
// widened to fp16, which is exact, by warps beside the copies (K too would be too much:
// the conversions run at 16 a cycle and SM, some 500 cycles a tile).
//
// Probabilities are rounded to 16 bits because their product with V needs V's type (bf16)
// or one that holds V exactly (fp16); the sums take them unrounded.
//
// Measured: one token of 256 requests over up to 16,384 keys of 4 kv heads 343 to 349 us
// (6.7 TB/s, a copy's rate), of 64 requests over up to 65,536 e4m3 keys of 8 kv heads 420 us
// (6.5 TB/s), one request over 8,192 keys 13.8 us with the join, which is starts, first
// copies and the pieces' way through memory.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kda_paged_tc.cuh"

namespace kda {
namespace {
using namespace tc;

constexpr int BK = KEY_TILE;
constexpr int TILE = BK * D * 2;       // an operand tile: two 64-channel blocks of 128 rows x 128 B
constexpr int RAW = BK * D;            // an e4m3 tile as loaded
constexpr int SEGS = 4;                // segments ahead of the roles
// An item's cost besides its tiles, in tiles (1: 17 e4m3 requests of up to 7,629 keys 40 us
// for 34, 116 windows over short contexts 82 us for 78, no better where contexts are long;
// 3: the bf16 batch of 256 352 us for 349).
constexpr int HEAD = 2;
constexpr float GROW = 8.f, NOTHING = -1e30f;
// Warps: two softmax groups of four, then one each for the products of S, loads, the
// walk and the products of O, and those that widen V.
// Buffers: K tiles (e4m3: as loaded), V operand tiles, e4m3 V tiles as loaded.
template <bool E4, int NR> struct Cfg {
    static constexpr int SOFT = 8, W_S = 8, W_LOAD = 9, W_WALK = 10, W_O = 11, W_WIDEN = 12;
    static constexpr int WIDEN = !E4 ? 0 : NR == 16 ? 8 : 4;  // (512 threads leave 128 registers for NR = 32)
    static constexpr int KT = E4 ? RAW : TILE;                // bytes of a K tile
    static constexpr int KS = E4 ? (NR == 32 ? 3 : 4) : 3, VS = E4 ? 2 : 3, RS = E4 ? 4 : 0;
    static constexpr int PB = BK * NR * 2, QB = NR * 128 * (E4 ? 3 : 2);  // (three 8-bit parts, two 64-channel blocks)
    static constexpr int OFF_K = 0, OFF_V = OFF_K + KS * KT, OFF_R = OFF_V + VS * TILE, OFF_Q = OFF_R + RS * RAW,
                         OFF_P = OFF_Q + 2 * QB, OFF_REF = OFF_P + 2 * PB, OFF_FAC = OFF_REF + 2 * NR * 4,
                         OFF_MRG = OFF_FAC + 2 * NR * 4, OFF_SUM = OFF_MRG + 2 * NR * 4, OFF_SC = OFF_SUM + 8 * NR * 4, OFF_SEG = OFF_SC + SEGS * NR * 4,
                         OFF_DESC = OFF_SEG + SEGS * 64, OFF_BAR = OFF_DESC + 32;
    static constexpr int NBAR = 2 * (KS + VS + RS) + 4 + 8 + 3 + 3 * SEGS;
    static constexpr int OFF_MISC = (OFF_BAR + NBAR * 8 + 15) / 16 * 16, SMEM = OFF_MISC + 64;
    static constexpr int THREADS = (W_WIDEN + WIDEN) * 32;
    static constexpr int TCOLS = NR == 16 ? 128 : 256;        // S [2][NR], O [item parity][group][NR]
    static_assert(SMEM <= 232448 && OFF_SEG % 16 == 0 && OFF_BAR % 8 == 0 && RS <= 8 && OFF_V % 1024 == 0, "shared memory layout");
};

template <class C> struct Bars {
    uint64_t *k_full, *k_empty, *v_full, *v_empty, *r_full, *r_empty, *q_full, *q_empty, *s_full, *p_ready, *pv_done, *o_free,
        *last, *joint, *seg_full, *seg_ready, *seg_empty;
    __device__ explicit Bars(uint8_t *sm) {
        k_full = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR);
        k_empty = k_full + C::KS;
        v_full = k_empty + C::KS;
        v_empty = v_full + C::VS;
        r_full = v_empty + C::VS;  // V tiles as loaded
        r_empty = r_full + C::RS;
        q_full = r_empty + C::RS;  // [2] by item
        q_empty = q_full + 2;
        s_full = q_empty + 2;      // [2] by tile
        p_ready = s_full + 2;
        pv_done = p_ready + 2;
        o_free = pv_done + 2;      // [2] by item
        last = o_free + 2;
        joint = last + 2;          // (last: the products of S, of O)
        seg_full = joint + 1;      // (joint: the two groups at an item's end)
        seg_ready = seg_full + SEGS;  // its queries and their scales are there too
        seg_empty = seg_ready + SEGS;
    }
};

// ---------------------------------------------------------------- the line
// Row groups: th = floor(NR / G) whole tokens, or, with more heads than NR, one
// token's heads NR at a time (`parts` of them).
struct Rows {
    int th, parts;
    __device__ Rows(int G, int NR) : th(G <= NR ? NR / G : 1), parts(G <= NR ? 1 : (G + NR - 1) / NR) {}
};
struct Req {
    PagedReq r;
    int n, ng;
};
__device__ __forceinline__ Req few_req(const PagedAttn &a, int i, const Rows &w, int *err) {
    Req q;
    q.r = paged_req(a, i, err);
    q.n = q.r.rows / a.G;
    q.ng = (q.n + w.th - 1) / w.th;
    return q;
}
__device__ __forceinline__ int item_units(const PagedAttn &a, const Req &q, int g, const Rows &w) {
    const int j0 = g * w.th, j1 = min(q.n, j0 + w.th) - 1;
    int lo, hi, t0, t1;
    key_tiles(a, q.r, j0, j1, lo, hi, t0, t1);
    return HEAD + max(1, t1 - t0);
}
// Units of the row groups before g.
__device__ __forceinline__ int64_t units_before(const PagedAttn &a, const Req &q, int g, const Rows &w) {
    const int full = min(g, q.n / w.th), pos0 = q.r.pos0;
    int neg = pos0 < 0 ? -pos0 / w.th : 0;  // groups whose last query stands before position 0
    if (neg > full) neg = full;
    int64_t u = neg + (int64_t)HEAD * full;
    if (full > neg) {
        u += floor_sum(full - neg, BK, w.th, pos0 + (neg + 1) * w.th + BK - 1);
        if (a.window > 0) {
            const int d = window_from(a, pos0);  // lo > 0 from g th > d on
            int gw = d < 0 ? 0 : d / w.th + 1;
            if (gw < neg) gw = neg;
            if (gw < full) u -= floor_sum(full - gw, BK, w.th, gw * w.th - d);
        }
    }
    if (g > full) u += item_units(a, q, full, w);  // the last, shorter group
    return u;
}
__device__ __forceinline__ int64_t line_units(const PagedAttn &a, int i, const Rows &w, int *err) {
    const Req q = few_req(a, i, w, err);
    return q.r.rows == 0 ? 0 : (int64_t)a.Hkv * w.parts * units_before(a, q, q.ng, w);
}

// A block's segment of an item: rows r = 0 .. R - 1 are rr = r0 + r, token tok + rr / G,
// head h G + rr % G.
struct __align__(16) Seg {
    int tok, R, h, r0;
    int pos, lo, hi, t0;     // first token's position; keys seen, first key tile
    int nt, req, whole, slot;
    int c0, c1, pad0, pad1;
};
static_assert(sizeof(Seg) == 64, "segment size");

struct Walk {
    int64_t pos, end, per, A;
    int req, vh, g;          // vh = kv head x parts + part
    Req q;
    bool fresh;
    __device__ bool next(const PagedAttn &a, const Rows &w, int NR, int64_t P0, Seg &s) {
        while (pos < end) {
            if (fresh) {
                while (true) {
                    q = few_req(a, req, w, nullptr);
                    if (q.r.rows) break;
                    ++req;  // (the total says that a request with tiles follows)
                }
                fresh = false;
            }
            const int64_t B = A + item_units(a, q, g, w), stop = B < end ? B : end;
            const int j0 = g * w.th, j1 = min(q.n, j0 + w.th) - 1;
            int t0, t1;
            key_tiles(a, q.r, j0, j1, s.lo, s.hi, t0, t1);
            const int b = max(0, (int)(pos - A) - HEAD), e = min((int)(stop - A) - HEAD, t1 - t0);
            const bool some = stop - A > HEAD;
            const int part = vh % w.parts;
            s.h = vh / w.parts;
            s.r0 = part * NR;
            s.R = w.parts > 1 ? min(NR, a.G - s.r0) : (j1 - j0 + 1) * a.G;
            s.tok = q.r.tok0 + j0;
            s.pos = q.r.pos0 + j0;
            s.t0 = t0 + b;
            s.nt = max(0, e - b);
            s.req = req;
            s.whole = b == 0 && stop == B;
            s.slot = 2 * (int)blockIdx.x + (pos == P0 ? 0 : 1);
            s.c0 = A + HEAD >= P0 ? (int)blockIdx.x : -1;  // block of the item's first tile: this one, or one before
            s.c1 = (int)blockIdx.x;                       // block of its last
            if (B > end) s.c1 = (int)((B - 1) / per);
            pos = stop;
            if (stop == B) {
                A = B;
                if (++g == q.ng) {
                    g = 0;
                    if (++vh == a.Hkv * w.parts) {
                        vh = 0;
                        ++req;
                        fresh = true;
                    }
                }
            }
            if (some) return true;
        }
        return false;
    }
};

struct Shared {
    uint32_t tmem;
    int abort, req, vh, g, pad;
    int64_t A;
};

template <class C, class Gate>
__device__ __forceinline__ bool next_seg(uint8_t *sm, const Bars<C> &bar, int &i, const Gate &gate, Seg &s) {
    if (!gate(&bar.seg_full[i % SEGS], (i / SEGS) & 1)) return false;
    s = *reinterpret_cast<const Seg *>(sm + C::OFF_SEG + (i % SEGS) * 64);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bar.seg_empty[i % SEGS]);
    ++i;
    return s.nt >= 0;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_f16(float x, float y) {
    const __half2 p = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// ---------------------------------------------------------------- walk, queries
// One warp walks the line, tells the others of each segment (the loads begin on it) and
// puts its queries (rows past R zero) into the buffer of their turn.
template <bool E4, int NR, class Gate>
__device__ __forceinline__ void walk_role(const PagedAttn &a, uint8_t *sm, Walk w, int64_t P0, const Gate &gate) {
    using C = Cfg<E4, NR>;
    const int lane = threadIdx.x & 31;
    const Bars<C> bar(sm);
    const Rows rw(a.G, NR);
    int item = 0;  // items with tiles
    for (int i = 0;; ++i) {
        Seg s;
        const bool more = w.next(a, rw, NR, P0, s);
        if (!more) s.nt = -1;
        if (!gate(&bar.seg_empty[i % SEGS], ((i / SEGS) & 1) ^ 1)) return;
        if (lane == 0) {
            *reinterpret_cast<Seg *>(sm + C::OFF_SEG + (i % SEGS) * 64) = s;
            mbar_arrive(&bar.seg_full[i % SEGS]);
        }
        __syncwarp();
        if (s.nt > 0) {
            const int x = item & 1;
            if (!gate(&bar.q_empty[x], ((item >> 1) & 1) ^ 1)) return;
            ++item;
            uint8_t *qb = sm + C::OFF_Q + x * C::QB;
            float *sc = reinterpret_cast<float *>(sm + C::OFF_SC) + (i % SEGS) * NR;
            const float ks = E4 ? a.scale_log2 * a.k_scale[s.h] : a.scale_log2;
            const int c = lane & 15;  // 16-byte piece of a row; two rows at a time
#pragma unroll 4
            for (int r = lane >> 4; r < NR; r += 2) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r < s.R) {
                    const int rr = s.r0 + r, j = rr / a.G;
                    v = __ldg((const uint4 *)a.q + ((int64_t)(s.tok + j) * a.Hq + s.h * a.G + (rr - j * a.G)) * (D / 8) + c);
                }
                if (E4) {
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                    float y[8], top = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        y[2 * k] = bf_lo(u[k]);
                        y[2 * k + 1] = bf_hi(u[k]);
                        // (the parts are cut at the largest value: NaN says that there is no answer)
                        if (fabsf(y[2 * k]) == INFINITY) y[2 * k] = NAN;
                        if (fabsf(y[2 * k + 1]) == INFINITY) y[2 * k + 1] = NAN;
                        top = fmaxf(top, fmaxf(fabsf(y[2 * k]), fabsf(y[2 * k + 1])));
                    }
#pragma unroll
                    for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    // The row's largest value goes to 2^14 .. 2^15 (rows under 2^-110: 2^124 times
                    // theirs).  Parts go down to 2^-16, so values over 2^-23 of the largest are exact,
                    // and what smaller ones lose is 2^-31 of it, far below the sums' own rounding.
                    // (Two e4m3 parts end 2^-16 below the largest: with one channel 2^12 times the
                    // others, scores were off by 0.2.)
                    const int e = max((int)(__float_as_uint(top) >> 23) - 127, -110);
                    const float down = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
                    if (c == 0) sc[r] = ks * __uint_as_float((uint32_t)(127 + e - 14) << 23);
                    uint32_t w[3][2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
#pragma unroll
                        for (int p = 0; p < 3; ++p) w[p][k] = 0;
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            float2 z = make_float2(y[4 * k + 2 * g] * down, y[4 * k + 2 * g + 1] * down);
#pragma unroll
                            for (int p = 0; p < 3; ++p) {
                                const __nv_fp8x2_storage_t b = __nv_cvt_float2_to_fp8x2(z, __NV_SATFINITE, __NV_E5M2);
                                const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(b, __NV_E5M2);
                                const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&hr));
                                w[p][k] |= (uint32_t)b << (16 * g);
                                z.x -= back.x;
                                z.y -= back.y;
                            }
                        }
                    }
                    // three [row][channel] e5m2 operands, 128 bytes a row: this lane's 8 channels
                    uint8_t *at = qb + r * 128 + (((c >> 1) ^ (r & 7)) << 4) + 8 * (c & 1);
#pragma unroll
                    for (int p = 0; p < 3; ++p) *reinterpret_cast<uint2 *>(at + p * NR * 128) = make_uint2(w[p][0], w[p][1]);
                } else {
                    if (c == 0) sc[r] = ks;
                    *reinterpret_cast<uint4 *>(qb + (c >> 3) * NR * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.q_full[x]);
        }
        if (lane == 0) mbar_arrive(&bar.seg_ready[i % SEGS]);
        __syncwarp();
        if (!more) return;
    }
}

// ---------------------------------------------------------------- loads
// Tiles go in the order K0, K1, V0, K2, V1 .. through all items: K is used two tiles
// before V is.  e4m3's V goes into a ring of its own, with a word that says which rows
// hold seen keys.
template <bool E4, int NR, class Gate>
__device__ __forceinline__ void load_role(const PagedAttn &a, const PagedMaps &maps, uint8_t *sm, const Gate &gate) {
    using C = Cfg<E4, NR>;
    constexpr int ES = E4 ? 1 : 2, NV = E4 ? C::RS : C::VS;
    const int lane = threadIdx.x & 31;
    const Bars<C> bar(sm);
    const int box = a.box, lg = a.box_log, nbx = BK >> lg;
    uint64_t *vf = E4 ? bar.r_full : bar.v_full, *ve = E4 ? bar.r_empty : bar.v_empty;
    uint8_t *kb = sm + C::OFF_K, *vb = sm + (E4 ? C::OFF_R : C::OFF_V);
    int nk = 0, nv = 0;                                 // tiles of K and V so far
    int kslot = 0, kph = 1, vslot = 0, vph = 1;         // their places in the rings, and the parity to wait for
    // The block ends only when its copies have landed, also where a wait of another role runs
    // out after this one has issued its last.  v: tiles of V that may be in flight.
    auto drain = [&](int v) {
        for (int u = nk - 1; u >= 0 && u >= nk - C::KS; --u) mbar_wait(&bar.k_full[u % C::KS], (u / C::KS) & 1);
        for (int u = nv - 1; u >= 0 && u >= nv - v; --u) mbar_wait(&vf[u % NV], (u / NV) & 1);
        __syncwarp();
    };
    // boxes f .. e - 1 of a tile: this lane's page and row
    struct Tile {
        int f, e, page, y, z;  // z: first and one past the last row that holds a seen key (e4m3)
    };
    auto load = [&](const Tile &t, bool v) -> bool {
        const int slot = v ? vslot : kslot;
        if (!gate(v ? &ve[slot] : &bar.k_empty[slot], v ? vph : kph)) return false;
        uint8_t *dst = (v ? vb : kb) + slot * C::KT;
        uint64_t *full = v ? &vf[slot] : &bar.k_full[slot];
        if (E4 && v && lane == 0) reinterpret_cast<int *>(sm + C::OFF_DESC)[slot] = t.z;
        if (v) {
            ++nv;
            if (++vslot == NV) vslot = 0, vph ^= 1;
        } else {
            ++nk;
            if (++kslot == C::KS) kslot = 0, kph ^= 1;
        }
        if (lane == 0) mbar_expect_tx(full, (uint32_t)((t.e - t.f) << lg) * (D * ES));
        __syncwarp();
        if (lane >= t.f && lane < t.e) {
            const CUtensorMap *m = v ? &maps.v : &maps.k;
            tma_load_3d(dst + (lane << lg) * 128, m, 0, t.y, t.page, full);
            if (!E4) tma_load_3d(dst + TILE / 2 + (lane << lg) * 128, m, 64, t.y, t.page, full);
        }
        __syncwarp();
        return true;
    };
    Seg s;
    int iseg = 0;
    Tile prev{0, 0, 0, 0, 0};
    bool have = false;
    while (next_seg<C>(sm, bar, iseg, gate, s)) {
        if (s.nt == 0) {
            // The last item's V does not wait for the next K here: the walk goes SEGS segments ahead of
            // the softmax, so behind SEGS - 1 items without keys that K is told of only after this V
            // has been used.
            if (have && !load(prev, true)) return drain(NV);
            have = false;
            continue;
        }
        int cbase = 0, page = 0, off = 0;
        const int lob = s.lo & ~(box - 1);  // boxes before this one hold no seen key (their pages may be gone)
        for (int j = 0; j < s.nt; ++j) {
            const int key0 = (s.t0 + j) * BK, b0 = key0 >> lg;
            if (j == 0 || b0 + nbx > cbase + 32) {  // pages of the next 32 boxes, one per lane
                cbase = b0;
                const int key = (cbase + lane) << lg, blk = key / a.page_size;
                page = 0;
                off = s.h * a.page_size + key - blk * a.page_size;
                if (key >= lob && key < s.hi) {
                    page = a.table[(int64_t)s.req * a.max_blocks + blk];
                    if (page < 0 || page >= a.n_pages) {
                        if (a.err) atomicOr(a.err, KDA_DEVERR_PAGE);
                        page = 0;
                    }
                }
            }
            Tile t;
            t.f = max(0, (lob - key0) >> lg);
            t.e = min(nbx, (s.hi - key0 + box - 1) >> lg);
            t.page = __shfl_sync(0xffffffffu, page, (b0 - cbase + lane) & 31);
            t.y = __shfl_sync(0xffffffffu, off, (b0 - cbase + lane) & 31);
            t.z = max(0, s.lo - key0) | (min(BK, s.hi - key0) << 8);
            if (!load(t, false)) return drain(NV);
            if (have && !load(prev, true)) return drain(NV);
            prev = t;
            have = true;
        }
    }
    if (have && !*gate.abort && !load(prev, true)) return drain(NV);
    if (E4) {  // the end, for the widening warps
        if (!gate(&ve[vslot], vph)) return drain(NV);
        if (lane == 0) {
            reinterpret_cast<int *>(sm + C::OFF_DESC)[vslot] = -1;
            mbar_arrive(&vf[vslot]);
        }
        __syncwarp();
        return drain(NV - 1);  // (the tile that stood where the end does has been used)
    }
    drain(NV);
}

// ---------------------------------------------------------------- widening
// V from e4m3 to fp16, 32 WIDEN / 128 threads to a row.  Rows that no seen key stands in
// become zeros (0 x NaN is NaN).
template <int NR, class Gate>
__device__ __forceinline__ void widen_role(uint8_t *sm, const Gate &gate) {
    using C = Cfg<true, NR>;
    constexpr int W = 32 / C::WIDEN;  // 16-byte pieces of a row for one thread: 8 of them to a row
    const Bars<C> bar(sm);
    const int tid = threadIdx.x - C::W_WIDEN * 32, row = tid & 127, lane = tid & 31, x = row & 7, p0 = (tid >> 7) * W;
    const uint8_t *raw = sm + C::OFF_R + row * 128;
    uint8_t *out = sm + C::OFF_V + row * 128;
    const volatile int *desc = reinterpret_cast<const volatile int *>(sm + C::OFF_DESC);
    int slot = 0, ph = 0, os = 0, oph = 0;
    while (true) {
        if (!gate(&bar.r_full[slot], ph)) return;
        const int z = desc[slot];
        if (z < 0) return;
        const uint8_t *src = raw + slot * RAW;
        uint4 w[W];
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = *reinterpret_cast<const uint4 *>(src + (((p0 + i) ^ x) << 4));
        if (row < (z & 255) || row >= (z >> 8)) {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = make_uint4(0, 0, 0, 0);
        }
        if (!gate(&bar.v_empty[os], oph ^ 1)) return;
        uint8_t *dst = out + os * TILE;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint32_t y[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t h[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(y[k] & 0xffff), __NV_E4M3);
                const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(y[k] >> 16), __NV_E4M3);
                h[2 * k] = (uint32_t)lo.x | ((uint32_t)lo.y << 16);
                h[2 * k + 1] = (uint32_t)hi.x | ((uint32_t)hi.y << 16);
            }
            const int p = p0 + i;  // piece of 16 channels: two of the 16-bit row
            uint8_t *at = dst + (p >> 2) * (TILE / 2);
            *reinterpret_cast<uint4 *>(at + (((2 * (p & 3)) ^ x) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(at + (((2 * (p & 3) + 1) ^ x) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&bar.v_full[os]);
            mbar_arrive(&bar.r_empty[slot]);
        }
        if (++slot == C::RS) {
            slot = 0;
            ph ^= 1;
        }
        if (++os == C::VS) {
            os = 0;
            oph ^= 1;
        }
    }
}

// ---------------------------------------------------------------- products
// S^T = K Q^T: eight steps of 16 channels, 32 bytes on within a block of 64; the
// second blocks begin at k + 1024 and q2 (units of 16 bytes).
__device__ __forceinline__ void issue_s(uint32_t d, uint64_t k, uint64_t q, uint64_t q2, uint32_t idesc) {
    asm volatile(
        "{\n .reg .pred e, t, f;\n .reg .b64 a, b;\n"
        " setp.eq.u32 t, 0, 0;\n setp.ne.u32 f, 0, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, f;\n"
        " add.s64 a, %1, 2;\n add.s64 b, %2, 2;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        " add.s64 a, %1, 4;\n add.s64 b, %2, 4;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        " add.s64 a, %1, 6;\n add.s64 b, %2, 6;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        " add.s64 a, %1, 1024;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, %3, %4, t;\n"
        " add.s64 a, %1, 1026;\n add.s64 b, %3, 2;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        " add.s64 a, %1, 1028;\n add.s64 b, %3, 4;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        " add.s64 a, %1, 1030;\n add.s64 b, %3, 6;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
        "}\n" ::"r"(d),
        "l"(k), "l"(q), "l"(q2), "r"(idesc)
        : "memory");
}
// The same with 8-bit K and the three parts of Q: four steps of 32 channels each.
__device__ __forceinline__ void issue_s8(uint32_t d, uint64_t k, uint64_t q, uint64_t q2, uint64_t q3, uint32_t idesc) {
    asm volatile(
        "{\n .reg .pred e, t, f;\n .reg .b64 a, b;\n"
        " setp.eq.u32 t, 0, 0;\n setp.ne.u32 f, 0, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %5, f;\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %3, %5, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %4, %5, t;\n"
        " add.s64 a, %1, 2;\n add.s64 b, %2, 2;\n @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, t;\n"
        " add.s64 b, %3, 2;\n @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, t;\n"
        " add.s64 b, %4, 2;\n @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, t;\n"
        " add.s64 a, %1, 4;\n add.s64 b, %2, 4;\n @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, t;\n"
        " add.s64 b, %3, 4;\n @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, t;\n"
        " add.s64 b, %4, 4;\n @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, t;\n"
        " add.s64 a, %1, 6;\n add.s64 b, %2, 6;\n @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, t;\n"
        " add.s64 b, %3, 6;\n @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, t;\n"
        " add.s64 b, %4, 6;\n @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, t;\n"
        "}\n" ::"r"(d),
        "l"(k), "l"(q), "l"(q2), "l"(q3), "r"(idesc)
        : "memory");
}
// O^T (+)= V^T P^T: eight steps of 16 keys, V 2 KB on, P 512 bytes on.
__device__ __forceinline__ void issue_o(uint32_t d, uint64_t v, uint64_t p, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred e, t, f;\n .reg .b64 a, b;\n"
        " setp.eq.u32 t, 0, 0;\n setp.ne.u32 f, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n"
        " add.s64 a, %1, 128;\n add.s64 b, %2, 32;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        " add.s64 a, %1, 256;\n add.s64 b, %2, 64;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        " add.s64 a, %1, 384;\n add.s64 b, %2, 96;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        " add.s64 a, %1, 512;\n add.s64 b, %2, 128;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        " add.s64 a, %1, 640;\n add.s64 b, %2, 160;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        " add.s64 a, %1, 768;\n add.s64 b, %2, 192;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        " add.s64 a, %1, 896;\n add.s64 b, %2, 224;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        "}\n" ::"r"(d),
        "l"(v), "l"(p), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}

// types: e4m3 0 and e5m2 1 (8-bit products), fp16 0, bf16 1 (16-bit ones); K and Q are K-major,
// V^T and P^T run along M and N
template <bool E4, int NR>
constexpr uint32_t ID_S = (1u << 4) | (E4 ? 0u : 1u << 7) | (1u << 10) | ((uint32_t)(NR >> 3) << 17) | ((128u >> 4) << 24);
template <bool E4, int NR>
constexpr uint32_t ID_O = (1u << 4) | (E4 ? 0u : (1u << 7) | (1u << 10)) | (1u << 15) | (1u << 16) | ((uint32_t)(NR >> 3) << 17) | ((128u >> 4) << 24);

// Before TMEM is given back and the block ends, whichever wait ran out or none.
template <class C>
__device__ __forceinline__ void drain_products(const Bars<C> &bar, int i) {
    mma_commit_w(bar.last + i);
    mbar_wait(bar.last + i, 0);
    __syncwarp();
}

template <bool E4, int NR, class Gate>
__device__ __forceinline__ void s_role(uint8_t *sm, uint32_t tmem, const Gate &gate) {
    using C = Cfg<E4, NR>;
    const Bars<C> bar(sm);
    const uint64_t dk = sdesc_sw128(smem_u32(sm) + C::OFF_K), dq = sdesc_sw128(smem_u32(sm) + C::OFF_Q);
    int n = 0, slot = 0, ph = 0, item = 0, iseg = 0;
    Seg s;
    while (next_seg<C>(sm, bar, iseg, gate, s)) {
        if (s.nt == 0) continue;
        const int x = item & 1, nt = s.nt;
        bool ok = gate(&bar.q_full[x], (item >> 1) & 1);
        const uint64_t q = dq + (uint32_t)x * (C::QB >> 4);
        for (int j = 0; ok && j < nt; ++j, ++n) {
            const int b = n & 1;
            ok = gate(&bar.k_full[slot], ph);
            if (n >= 2) ok = gate(&bar.p_ready[b], ((n >> 1) - 1) & 1) && ok;  // the S before last has been read
            if (!ok) break;
            tc_fence_after();
            const uint64_t k = dk + (uint32_t)slot * (C::KT >> 4);
            if constexpr (E4)
                issue_s8(tmem + b * NR, k, q, q + (NR * 128 >> 4), q + (2 * NR * 128 >> 4), ID_S<E4, NR>);
            else
                issue_s(tmem + b * NR, k, q, q + (NR * 128 >> 4), ID_S<E4, NR>);
            mma_commit_w(&bar.s_full[b]);
            mma_commit_w(&bar.k_empty[slot]);
            if (++slot == C::KS) {
                slot = 0;
                ph ^= 1;
            }
        }
        if (!ok) break;
        mma_commit_w(&bar.q_empty[x]);
        ++item;
    }
    drain_products<C>(bar, 0);
}
template <bool E4, int NR, class Gate>
__device__ __forceinline__ void o_role(uint8_t *sm, uint32_t tmem, const Gate &gate) {
    using C = Cfg<E4, NR>;
    const Bars<C> bar(sm);
    const uint64_t dv = sdesc_mn(smem_u32(sm) + C::OFF_V, TILE / 2, 1024, SWZ_128B),
                   dp = sdesc_mn(smem_u32(sm) + C::OFF_P, BK * 32, 256, SWZ_32B);
    int n = 0, slot = 0, ph = 0, item = 0, iseg = 0;
    Seg s;
    while (next_seg<C>(sm, bar, iseg, gate, s)) {
        if (s.nt == 0) continue;
        const int nt = s.nt;
        bool ok = gate(&bar.o_free[item & 1], ((item >> 1) & 1) ^ 1);  // the item before last has left this O
        const uint32_t to = tmem + 2 * NR + (item & 1) * 2 * NR;
        for (int j = 0; ok && j < nt; ++j, ++n) {
            const int b = n & 1;
            ok = gate(&bar.v_full[slot], ph);
            ok = gate(&bar.p_ready[b], (n >> 1) & 1) && ok;
            if (!ok) break;
            tc_fence_after();
            issue_o(to + b * NR, dv + (uint32_t)slot * (TILE >> 4), dp + (uint32_t)b * (C::PB >> 4), ID_O<E4, NR>, j > 1);
            mma_commit_w(&bar.pv_done[b]);
            mma_commit_w(&bar.v_empty[slot]);
            if (++slot == C::VS) {
                slot = 0;
                ph ^= 1;
            }
        }
        if (!ok) break;
        ++item;
    }
    drain_products<C>(bar, 1);
}

// ---------------------------------------------------------------- softmax
// Every lane brings NR = 16 or 32 values; afterwards lane's v[0] is the maximum (or sum)
// over the lanes of value first_of(lane): each step hands half of the values to the lane
// across.
template <int NR, bool MAX>
__device__ __forceinline__ void across(float (&v)[NR], int lane) {
    int n = NR;
#pragma unroll
    for (int s = 16; s; s >>= 1) {
        if (n > 1) {
            n >>= 1;
#pragma unroll
            for (int i = 0; i < NR / 2; ++i) {
                if (i < n) {
                    const bool up = lane & s;
                    const float keep = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
                    const float got = __shfl_xor_sync(0xffffffffu, give, s);
                    v[i] = MAX ? fmaxf(keep, got) : keep + got;
                }
            }
        } else {
            const float got = __shfl_xor_sync(0xffffffffu, v[0], s);
            v[0] = MAX ? fmaxf(v[0], got) : v[0] + got;
        }
    }
}
template <int NR> __device__ __forceinline__ int first_of(int lane) { return NR == 32 ? lane : lane >> 1; }

// NR columns of this thread's lane
template <int NR>
__device__ __forceinline__ void tmem_row(uint32_t taddr, float *o) {
    if constexpr (NR == 16) {
        tmem_ld16(taddr, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) asm volatile("" : "+f"(o[i]));
    } else {
#pragma unroll
        for (int c = 0; c < NR; c += 32) tmem_ld32(taddr + c, o + c);
#pragma unroll
        for (int c = 0; c < NR; c += 32) tmem_arrived(o + c);
    }
}

// Thread = key of a tile, and channel of O; group g has the tiles of its parity.  A wait
// that runs out is passed on at the group's next meeting (every segment begins with one,
// every meeting looks for it), so that a group's warps leave together; the groups wait
// for each other with bounded waits only.
template <bool E4, int NR, class Gate>
__device__ __forceinline__ void softmax_role(const PagedAttn &a, uint8_t *sm, uint32_t tmem, const Gate &gate) {
    using C = Cfg<E4, NR>;
    const Bars<C> bar(sm);
    const int g = threadIdx.x >> 7, tid = threadIdx.x & 127, warp = tid >> 5, lane = tid & 31, id = 1 + g;
    const uint32_t lanes = (uint32_t)warp << 21, ts = tmem + lanes + g * NR;  // 32 warp << 16
    float *refs = reinterpret_cast<float *>(sm + C::OFF_REF), *ref = refs + g * NR;  // this group's references
    float *fac = reinterpret_cast<float *>(sm + C::OFF_FAC) + g * NR;                // and factors
    float *sums = reinterpret_cast<float *>(sm + C::OFF_SUM);                        // [group][warp][NR]
    uint8_t *pb = sm + C::OFF_P + g * C::PB;
    const int G = a.G;
    int n = 0, k = 0, item = 0, joint = 0;  // tiles, this group's, items with tiles, joint meetings so far
    bool failed = false;
    auto together = [&]() {  // the two groups
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.joint);
        if (!gate(bar.joint, joint & 1)) failed = true;
        ++joint;
    };
    for (int iseg = 0;; ++iseg) {
        if (!gate(&bar.seg_ready[iseg % SEGS], (iseg / SEGS) & 1)) failed = true;
        if (meet_count<128>(id, failed) >= 32) return;
        const Seg *sg = reinterpret_cast<const Seg *>(sm + C::OFF_SEG + (iseg % SEGS) * 64);
        const int nt = sg->nt;
        if (nt < 0) return;
        const float *sc = reinterpret_cast<const float *>(sm + C::OFF_SC) + (iseg % SEGS) * NR;
        const int lo = sg->lo, hi = sg->hi, t0 = sg->t0, pos = sg->pos, R = sg->R, r0 = sg->r0;
        const uint32_t to = tmem + lanes + 2 * NR + (item & 1) * 2 * NR;  // + NR g
        float l[NR], top = -INFINITY;  // sums of this thread's keys; row tid's maximum at the last change of ref
#pragma unroll
        for (int r = 0; r < NR; ++r) l[r] = 0.f;
        int mine = 0;
        for (int j = (n & 1) ^ g; j < nt; j += 2, ++k, ++mine) {
            const int key0 = (t0 + j) * BK, key = key0 + tid;
            if (!gate(&bar.s_full[g], k & 1)) failed = true;
            tc_fence_after();
            float t[NR];
            // scores; -inf where a row does not see this key (rows that do: [first, last))
            auto scores = [&]() {
                tmem_row<NR>(ts, t);
                if (key0 + BK - 1 > pos || key0 + BK > hi || a.window > 0) {
                    const int d = min(max(key - pos, 0), NR + 1), u = a.window > 0 ? min(max(key - pos + a.window, 0), NR + 1) : NR + 1;
                    const int first = key < hi ? d * G - r0 : NR, last = u > NR ? NR : u * G - r0;
#pragma unroll
                    for (int r = 0; r < NR; ++r) t[r] = r >= first && r < last ? t[r] : -INFINITY;
                }
            };
            // the exponents: t sc - ref
            auto exponents = [&]() {
#pragma unroll
                for (int r = 0; r < NR; r += 4) {
                    const float4 y = *reinterpret_cast<const float4 *>(ref + r);
                    const float4 f = E4 ? *reinterpret_cast<const float4 *>(sc + r)
                                        : make_float4(a.scale_log2, a.scale_log2, a.scale_log2, a.scale_log2);
                    t[r] = fmaf(t[r], f.x, -y.x);
                    t[r + 1] = fmaf(t[r + 1], f.y, -y.y);
                    t[r + 2] = fmaf(t[r + 2], f.z, -y.z);
                    t[r + 3] = fmaf(t[r + 3], f.w, -y.w);
                }
            };
            scores();
            bool grow = mine == 0;
            if (mine > 0) {
                exponents();
                float m0 = max3(t[0], t[1], t[2]), m1 = t[3];
#pragma unroll
                for (int r = 4; r < NR; r += 4) {
                    m0 = max3(m0, t[r], t[r + 1]);
                    m1 = max3(m1, t[r + 2], t[r + 3]);
                }
                grow = fmaxf(m0, m1) > GROW;
            }
            grow = __any_sync(0xffffffffu, grow);
            if (k > 0 && !gate(&bar.pv_done[g], (k - 1) & 1)) failed = true;  // P's buffer, O: the last product is done
            // a warp that gave up counts 32, one that saw a maximum grow 1
            const int said = meet_count<128>(id, failed || (grow && lane == 0));
            if (said >= 32) return;
            if (said) {
                if (mine > 0) scores();
                // largest score of each row over the tile (the warps' maxima meet in P's buffer)
                {
                    float m[NR];
#pragma unroll
                    for (int r = 0; r < NR; ++r) m[r] = t[r] * (E4 ? sc[r] : a.scale_log2);
                    across<NR, true>(m, lane);
                    reinterpret_cast<float *>(pb)[warp * NR + first_of<NR>(lane)] = m[0];
                }
                if (meet_count<128>(id, failed) >= 32) return;
                if (tid < NR) {
                    const float was = mine == 0 ? -INFINITY : top, old = ref[tid];
                    float m = was;
#pragma unroll
                    for (int w = 0; w < 4; ++w) m = fmaxf(m, reinterpret_cast<const float *>(pb)[w * NR + tid]);
                    // a row that had seen nothing has zeros in O and in its sums, and a reference
                    // that its first score will be far above
                    const float next = m == -INFINITY ? NOTHING : was == -INFINITY ? m : fmaxf(m, old);
                    fac[tid] = was == -INFINITY ? 0.f : ex2(old - next);
                    ref[tid] = next;
                    top = m;
                }
                if (meet_count<128>(id, failed) >= 32) return;
                if (mine > 0) {
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < NR; c += 16) {
                        float o[16];
                        uint32_t w[16];
                        tmem_ld16(to + g * NR + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            asm volatile("" : "+f"(o[i]));
                            w[i] = __float_as_uint(o[i] * fac[c + i]);
                        }
                        tmem_st16(to + g * NR + c, w);
                    }
                    tmem_st_wait();
#pragma unroll
                    for (int r = 0; r < NR; ++r) l[r] *= fac[r];
                }
                exponents();
            }
            uint32_t p[NR / 2];
#pragma unroll
            for (int r = 0; r < NR; r += 2) {
                const float e0 = ex2(t[r]), e1 = ex2(t[r + 1]);
                l[r] += e0;
                l[r + 1] += e1;
                p[r / 2] = E4 ? pack_f16(e0, e1) : pack_bf16(e0, e1);
            }
            // [key][row], blocks of 16 rows, the two 16-byte halves swapped on every other group of four keys
#pragma unroll
            for (int c = 0; c < NR / 8; ++c)
                *reinterpret_cast<uint4 *>(pb + (c >> 1) * BK * 32 + tid * 32 + (((c & 1) ^ ((tid >> 2) & 1)) << 4)) =
                    make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
            if (!E4) {
                // a row of V that no seen key stands in may hold anything: zero it (0 x NaN is NaN)
                const bool none = key >= hi || key < lo;
                if (__any_sync(0xffffffffu, none)) {
                    const int v = n + j;
                    if (!gate(&bar.v_full[v % C::VS], (v / C::VS) & 1)) failed = true;
                    uint8_t *vt = sm + C::OFF_V + (v % C::VS) * TILE + tid * 128;
                    if (none) {
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            *reinterpret_cast<uint4 *>(vt + (c >> 3) * (TILE / 2) + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
                    }
                }
            }
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.p_ready[g]);
        }
        n += nt;

        // ---- the segment's end: the groups' sums and O merged, normalised or as a piece
        const bool whole = sg->whole;
        const int h = sg->h;
        float *slot = paged_slot(a, sg->slot);
        float *f0 = reinterpret_cast<float *>(sm + C::OFF_MRG), *f1 = f0 + NR;
        const int64_t out0 = (int64_t)sg->tok * a.Hq + h * G;  // row rr = r0 + r of the token's heads, the next token Hq on
        if (nt > 0) {
            if (mine > 0 && !gate(&bar.pv_done[g], (k - 1) & 1)) failed = true;
            across<NR, false>(l, lane);
            sums[(g * 4 + warp) * NR + first_of<NR>(lane)] = l[0];
            tc_fence_before();
            together();
            tc_fence_after();
            if (g == 0 && tid < NR) {
                float L0 = 0.f, L1 = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    L0 += sums[w * NR + tid];
                    L1 += sums[(4 + w) * NR + tid];
                }
                const float m0 = L0 == 0.f ? -INFINITY : refs[tid], m1 = L1 == 0.f ? -INFINITY : refs[NR + tid];
                const float m = fmaxf(m0, m1), base = m == -INFINITY ? 0.f : m;
                const float e0 = L0 == 0.f ? 0.f : ex2(m0 - base), e1 = L1 == 0.f ? 0.f : ex2(m1 - base);
                const float L = e0 * L0 + e1 * L1, s = L == 0.f ? 0.f : whole ? (E4 ? a.v_scale[h] : 1.f) / L : 1.f;
                f0[tid] = e0 * s;
                f1[tid] = e1 * s;
                if (tid < R) {
                    if (!whole) {
                        reinterpret_cast<float2 *>(slot)[tid] = make_float2(L == 0.f ? -INFINITY : base, L);
                    } else if (a.lse) {
                        const int rr = r0 + tid, jt = rr / G;
                        a.lse[out0 + (int64_t)jt * a.Hq + rr - jt * G] =
                            L == 0.f ? -INFINITY : (base + log2f(L)) * 0.6931471805599453f;
                    }
                }
            }
            together();
        } else if (g == 0 && tid < R) {
            if (!whole) {
                reinterpret_cast<float2 *>(slot)[tid] = make_float2(-INFINITY, 0.f);
            } else if (a.lse) {
                const int rr = r0 + tid, jt = rr / G;
                a.lse[out0 + (int64_t)jt * a.Hq + rr - jt * G] = -INFINITY;
            }
        }
        {  // a thread has one channel of every row; group g writes the rows from NR / 2 g on
            const int rb = g * (NR / 2), j0 = (r0 + rb) / G;
            int hh = r0 + rb - j0 * G;  // head within the token's group
            int64_t at = (out0 + (int64_t)j0 * a.Hq + hh) * D + tid;
            float o[16], q[16];  // the groups' O (where a group had no tile its factor is zero)
            const int c = NR == 32 ? rb : 0;
            tmem_ld16(to + c, o);
            tmem_ld16(to + NR + c, q);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                asm volatile("" : "+f"(o[i]));
                asm volatile("" : "+f"(q[i]));
            }
#pragma unroll
            for (int i = 0; i < NR / 2; ++i) {
                const int r = rb + i;
                if (r >= R) break;
                const float u = NR == 16 && g ? o[(i + 8) & 15] : o[i], w = NR == 16 && g ? q[(i + 8) & 15] : q[i];
                float y = 0.f;
                if (nt > 0) {
                    if (f0[r] != 0.f) y = u * f0[r];  // (nothing seen: zero whatever O holds)
                    if (f1[r] != 0.f) y += w * f1[r];
                }
                if (whole) {
                    reinterpret_cast<__nv_bfloat16 *>(a.o)[at] = __float2bfloat16_rn(y);
                    at += D;
                    if (++hh == G) {
                        hh = 0;
                        at += (int64_t)(a.Hq - G) * D;
                    }
                } else {
                    slot[2 * a.slot_rows + r * D + tid] = y;
                }
            }
        }
        if (threadIdx.x == 0 && !whole && sg->c0 == (int)blockIdx.x) {
            a.lead[2 * blockIdx.x] = make_int4(sg->tok, h, sg->r0, sg->R);
            a.lead[2 * blockIdx.x + 1] = make_int4(sg->slot, sg->c0, sg->c1, 1);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if (nt > 0) mbar_arrive(&bar.o_free[item & 1]);
            mbar_arrive(&bar.seg_empty[iseg % SEGS]);
        }
        if (nt > 0) ++item;
    }
}

template <bool E4, int NR, bool SHORT>
__global__ void __launch_bounds__(Cfg<E4, NR>::THREADS, 1)
    paged_few_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ PagedAttn a, int min_per) {
    using C = Cfg<E4, NR>;
    extern __shared__ __align__(1024) uint8_t sm[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Shared *sh = reinterpret_cast<Shared *>(sm + C::OFF_MISC);
    int64_t *scratch = reinterpret_cast<int64_t *>(sm + C::OFF_SEG);
    const Bars<C> bar(sm);
    const Rows rw(a.G, NR);
    if (tid == 0) {
        for (int i = 0; i < C::KS; ++i) {
            mbar_init(&bar.k_full[i], 1);
            mbar_init(&bar.k_empty[i], 1);
        }
        for (int i = 0; i < C::VS; ++i) {
            mbar_init(&bar.v_full[i], E4 ? C::WIDEN : 1);
            mbar_init(&bar.v_empty[i], 1);
        }
        for (int i = 0; i < C::RS; ++i) {
            mbar_init(&bar.r_full[i], 1);
            mbar_init(&bar.r_empty[i], C::WIDEN);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.q_full[i], 1);
            mbar_init(&bar.q_empty[i], 1);
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_ready[i], C::SOFT / 2);
            mbar_init(&bar.pv_done[i], 1);
            mbar_init(&bar.o_free[i], C::SOFT);
        }
        for (int i = 0; i < SEGS; ++i) {
            mbar_init(&bar.seg_full[i], 1);
            mbar_init(&bar.seg_ready[i], 1);
            mbar_init(&bar.seg_empty[i], C::SOFT + 3);
        }
        mbar_init(bar.last, 1);
        mbar_init(bar.last + 1, 1);
        mbar_init(bar.joint, C::SOFT);
        mbar_fence_init();
        sh->abort = 0;
        a.lead[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
    }
    auto units = [&](int i, int *err) { return line_units(a, i, rw, err); };
    const PagedLine line = paged_line<C::THREADS>(a, scratch, min_per, units, [](int64_t) { return 1; });
    if (line.P0 >= line.P1) return;
    if (warp == 0) {  // virtual head and row group of the block's first unit
        const Req q = few_req(a, line.req, rw, nullptr);
        const int64_t head = line.units / (a.Hkv * rw.parts), in = line.P0 - line.before;
        const int vh = (int)(in / head);
        const int64_t rem = in - vh * head;
        // the last row group that begins at or before rem, 32 candidates at a time
        int lo = 0, n = q.ng;
        while (n > 1) {
            const int step = (n + 31) / 32, g = lo + lane * step;
            const bool at = lane * step < n && units_before(a, q, g, rw) <= rem;
            const int k = 31 - __clz(__ballot_sync(0xffffffffu, at));
            lo += k * step;
            n = min(step, n - k * step);
        }
        if (lane == 0) {
            sh->req = line.req;
            sh->vh = vh;
            sh->g = lo;
            sh->A = line.before + vh * head + units_before(a, q, lo, rw);
        }
    }
    if (warp == C::W_S) tmem_alloc(&sh->tmem, C::TCOLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    const Waits<SHORT> gate{&sh->abort, a.err, a.wait_budget};
    if (warp < C::SOFT) {
        softmax_role<E4, NR>(a, sm, tmem, gate);
    } else if (warp == C::W_S) {
        s_role<E4, NR>(sm, tmem, gate);
    } else if (warp == C::W_O) {
        o_role<E4, NR>(sm, tmem, gate);
    } else if (warp == C::W_LOAD) {
        load_role<E4, NR>(a, maps, sm, gate);
    } else if (warp == C::W_WALK) {
        Walk w;
        w.pos = line.P0;
        w.end = line.P1;
        w.per = line.per;
        w.A = sh->A;
        w.req = sh->req;
        w.vh = sh->vh;
        w.g = sh->g;
        w.fresh = true;
        walk_role<E4, NR>(a, sm, w, line.P0, gate);
    } else {
        if constexpr (E4) widen_role<NR>(sm, gate);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::W_S) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TCOLS);
    }
}

template <bool E4, int NR, bool SHORT>
int launch_for(const PagedAttn &a, const PagedMaps &maps, cudaStream_t s) {
    using C = Cfg<E4, NR>;
    const int rc = prepare_kernel((const void *)paged_few_kernel<E4, NR, SHORT>, C::SMEM, C::THREADS, nullptr);
    if (rc) return rc;
    paged_few_kernel<E4, NR, SHORT><<<paged_few_blocks(), C::THREADS, C::SMEM, s>>>(maps, a, 3);
    note_launch("paged_few", s);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
template <bool E4, int NR>
int launch(const PagedAttn &a, const PagedMaps &maps, cudaStream_t s) {
    return a.wait_budget < SHORT_BUDGET ? launch_for<E4, NR, true>(a, maps, s) : launch_for<E4, NR, false>(a, maps, s);
}

}  // namespace

int paged_few_blocks() { return device_sm_count(); }

int launch_paged_few(PagedAttn a, int cache_dtype, const void *k, const void *v, int64_t page_stride, int64_t max_rows,
                     cudaStream_t s) {
    int box = 16;
    while (box < BK && a.page_size % (2 * box) == 0) box *= 2;
    a.box = box;
    a.box_log = __builtin_ctz(box);
    PagedMaps maps;
    const int rc = make_paged_maps(k, v, cache_dtype, a.Hkv, a.page_size, a.n_pages, page_stride, box, &maps);
    if (rc) return rc;
    const bool e4 = cache_dtype == KDA_E4M3;
    if (max_rows <= 16) return e4 ? launch<true, 16>(a, maps, s) : launch<false, 16>(a, maps, s);
    return e4 ? launch<true, 32>(a, maps, s) : launch<false, 32>(a, maps, s);
}

}  // namespace kda
