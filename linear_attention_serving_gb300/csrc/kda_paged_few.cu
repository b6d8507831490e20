// kda_paged_few.cu -- paged attention on tcgen05 for few rows (single tokens,
// draft windows, short chunks; bf16 and e4m3 caches): up to NR = 16, 32 or 64 rows
// of one kv head at a time.  Each key and value is read for few rows, so the time is
// the pages' bytes over HBM; what the kernel has to do is keep copies in flight and
// stay out of their way.
//
// The products are taken the other way round than for many rows, so that the 128
// lanes of TMEM are keys (and channels) and only the NR columns in use cost
// anything:
//   S^T = K Q^T    128 keys x NR fp32 in TMEM, K from shared memory as it was loaded
//   P^T = exp2(S^T scale - ref): thread = key, NR values, stored as the [key][row]
//         operand of the second product (bf16; fp16 for e4m3 caches)
//   O^T += V^T P^T 128 channels x NR fp32 in TMEM, V from shared memory as loaded
// Products of S run two tiles ahead of those of O, across items.
//
// `ref` follows a row's maximum only when that has grown by more than 2^8 (kept
// probabilities are then as precise in 16 bits, sums are fp32): most tiles need no
// maximum over their keys at all, which would go across lanes, and no rescaling; one
// barrier tells the four softmax warps whether any of them saw such growth.
//
// e4m3 caches: the copies bring 16 KB tiles, eight warps widen them to fp16, which is
// exact, into the operands' buffers; q is scaled by a power of two per row so that
// fp16 holds it as precisely as bf16 did.
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
constexpr int HEAD = 1;                // an item's cost besides its tiles, in tiles
constexpr float GROW = 8.f, NOTHING = -1e30f;
constexpr int SOFT = 4;                // softmax warps (0..3), then products, loads, walk, idle, and the widening warps
constexpr int W_MMA = 4, W_LOAD = 5, W_WALK = 6, W_WIDEN = 8, WIDEN = 8;

// Buffers: K and V operand tiles, raw e4m3 tiles.
template <bool E4, int NR> struct Cfg {
    static constexpr int KS = E4 ? 1 : NR == 64 ? 2 : 3, VS = E4 ? 2 : 3, RS = E4 ? (NR == 64 ? 4 : NR == 32 ? 6 : 7) : 0;
    static constexpr int PB = BK * NR * 2, QB = NR * D * 2;
    static constexpr int OFF_K = 0, OFF_V = OFF_K + KS * TILE, OFF_R = OFF_V + VS * TILE, OFF_Q = OFF_R + RS * RAW,
                         OFF_P = OFF_Q + 2 * QB, OFF_REF = OFF_P + 2 * PB, OFF_CORR = OFF_REF + NR * 4,
                         OFF_SC = OFF_CORR + NR * 4, OFF_SEG = OFF_SC + SEGS * NR * 4, OFF_DESC = OFF_SEG + SEGS * 64,
                         OFF_BAR = OFF_DESC + 128;
    static constexpr int NBAR = 2 * (KS + VS + RS) + 4 + 8 + 1 + 2 * SEGS;
    static constexpr int OFF_MISC = (OFF_BAR + NBAR * 8 + 15) / 16 * 16, SMEM = OFF_MISC + 64;
    static constexpr int THREADS = (W_WIDEN + (E4 ? WIDEN : 0)) * 32;
    static constexpr int TCOLS = 4 * NR;
    static_assert(SMEM <= 232448 && OFF_SEG % 16 == 0 && OFF_BAR % 8 == 0, "shared memory layout");
};

template <class C> struct Bars {
    uint64_t *k_full, *k_empty, *v_full, *v_empty, *r_full, *r_empty, *q_full, *q_empty, *s_full, *p_ready, *pv_done, *o_free,
        *last, *seg_full, *seg_empty;
    __device__ explicit Bars(uint8_t *sm) {
        k_full = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR);
        k_empty = k_full + C::KS;
        v_full = k_empty + C::KS;
        v_empty = v_full + C::VS;
        r_full = v_empty + C::VS;
        r_empty = r_full + C::RS;
        q_full = r_empty + C::RS;  // [2] by item
        q_empty = q_full + 2;
        s_full = q_empty + 2;      // [2] by tile
        p_ready = s_full + 2;
        pv_done = p_ready + 2;
        o_free = pv_done + 2;      // [2] by item
        last = o_free + 2;
        seg_full = last + 1;
        seg_empty = seg_full + SEGS;
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
            const int d = a.window - 1 - pos0;  // lo > 0 from g th > d on
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
            s.c0 = (int)((A + HEAD) / per);
            s.c1 = (int)((B - 1) / per);
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

template <class C>
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
// One warp walks the line and puts each item's queries (rows past R zero) into the
// buffer of its turn before it tells the others of the segment.
template <bool E4, int NR>
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
                    uint32_t u[4] = {v.x, v.y, v.z, v.w};
                    float top = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) top = fmaxf(top, fmaxf(fabsf(bf_lo(u[k])), fabsf(bf_hi(u[k]))));
#pragma unroll
                    for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    // 2^-e with e the exponent of the row's largest value (none for 0, inf and the ends of the range)
                    const int e = (int)(__float_as_uint(top) >> 23) - 127;
                    const bool ok = e > -120 && e < 120;
                    const float down = ok ? __uint_as_float((uint32_t)(127 - e) << 23) : 1.f;
                    if (c == 0) sc[r] = ks * (ok ? __uint_as_float((uint32_t)(127 + e) << 23) : 1.f);
#pragma unroll
                    for (int k = 0; k < 4; ++k) u[k] = pack_f16(bf_lo(u[k]) * down, bf_hi(u[k]) * down);
                    v = make_uint4(u[0], u[1], u[2], u[3]);
                } else if (c == 0) {
                    sc[r] = ks;
                }
                *reinterpret_cast<uint4 *>(qb + (c >> 3) * NR * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.q_full[x]);
        }
        if (lane == 0) {
            *reinterpret_cast<Seg *>(sm + C::OFF_SEG + (i % SEGS) * 64) = s;
            mbar_arrive(&bar.seg_full[i % SEGS]);
        }
        __syncwarp();
        if (!more) return;
    }
}

// ---------------------------------------------------------------- loads
// Tiles go in the order K0, K1, V0, K2, V1 .. through all items: K is used two tiles
// before V is.  bf16: straight into the operands' buffers.  e4m3: into the ring of
// raw tiles, with a word that says what it is.
template <bool E4, int NR>
__device__ __forceinline__ void load_role(const PagedAttn &a, const PagedMaps &maps, uint8_t *sm, const Gate &gate) {
    using C = Cfg<E4, NR>;
    constexpr int ES = E4 ? 1 : 2, RING = E4 ? C::RS : 1;
    const int lane = threadIdx.x & 31;
    const Bars<C> bar(sm);
    const int box = a.box, nbx = BK / box;
    int nk = 0, nv = 0, nr = 0;  // tiles of K, V, raw so far
    auto drain = [&]() {         // a wait ran out: let the copies in flight land before the block ends
        if (E4) {
            for (int u = nr - 1; u >= 0 && u >= nr - RING; --u) mbar_wait(&bar.r_full[u % RING], (u / RING) & 1);
        } else {
            for (int u = nk - 1; u >= 0 && u >= nk - C::KS; --u) mbar_wait(&bar.k_full[u % C::KS], (u / C::KS) & 1);
            for (int u = nv - 1; u >= 0 && u >= nv - C::VS; --u) mbar_wait(&bar.v_full[u % C::VS], (u / C::VS) & 1);
        }
        __syncwarp();
    };
    // boxes f .. e - 1 of a tile: this lane's page and row
    struct Tile {
        int f, e, page, y, z;  // z: first and one past the last row that holds a key (e4m3)
    };
    auto load = [&](const Tile &t, bool v) -> bool {
        uint8_t *dst;
        uint64_t *full;
        if (E4) {
            const int slot = nr % RING;
            if (!gate(&bar.r_empty[slot], ((nr / RING) & 1) ^ 1)) return false;
            dst = sm + C::OFF_R + slot * RAW;
            full = &bar.r_full[slot];
            if (lane == 0) reinterpret_cast<int *>(sm + C::OFF_DESC)[slot] = t.z | (v ? 1 << 16 : 0);
            ++nr;
        } else if (v) {
            const int slot = nv % C::VS;
            if (!gate(&bar.v_empty[slot], ((nv / C::VS) & 1) ^ 1)) return false;
            dst = sm + C::OFF_V + slot * TILE;
            full = &bar.v_full[slot];
            ++nv;
        } else {
            const int slot = nk % C::KS;
            if (!gate(&bar.k_empty[slot], ((nk / C::KS) & 1) ^ 1)) return false;
            dst = sm + C::OFF_K + slot * TILE;
            full = &bar.k_full[slot];
            ++nk;
        }
        if (lane == 0) mbar_expect_tx(full, (uint32_t)((t.e - t.f) * box * D * ES));
        __syncwarp();
        if (lane >= t.f && lane < t.e) {
            const CUtensorMap *m = v ? &maps.v : &maps.k;
            tma_load_3d(dst + lane * box * 128, m, 0, t.y, t.page, full);
            if (!E4) tma_load_3d(dst + TILE / 2 + lane * box * 128, m, 64, t.y, t.page, full);
        }
        __syncwarp();
        return true;
    };
    Seg s;
    int iseg = 0;
    Tile prev{0, 0, 0, 0, 0};
    bool have = false;
    while (next_seg<C>(sm, bar, iseg, gate, s)) {
        if (s.nt == 0) continue;
        int cbase = 0, page = 0;
        const int lob = s.lo & ~(box - 1);  // boxes before this one hold no seen key (their pages may be gone)
        for (int j = 0; j < s.nt; ++j) {
            const int key0 = (s.t0 + j) * BK, b0 = key0 / box;
            if (j == 0 || b0 + nbx > cbase + 32) {  // pages of the next 32 boxes, one per lane
                cbase = b0;
                const int key = (cbase + lane) * box;
                page = 0;
                if (key >= lob && key < s.hi) {
                    page = a.table[(int64_t)s.req * a.max_blocks + key / a.page_size];
                    if (page < 0 || page >= a.n_pages) {
                        if (a.err) atomicOr(a.err, KDA_DEVERR_PAGE);
                        page = 0;
                    }
                }
            }
            Tile t;
            t.f = max(0, (lob - key0) / box);
            t.e = min(nbx, (s.hi - key0 + box - 1) / box);
            t.page = __shfl_sync(0xffffffffu, page, (b0 - cbase + lane) & 31);
            t.y = s.h * a.page_size + (key0 + lane * box) % a.page_size;
            t.z = max(0, lob - key0) | (min(BK, s.hi - key0) << 8);
            if (!load(t, false)) return drain();
            if (have && !load(prev, true)) return drain();
            prev = t;
            have = true;
        }
    }
    if (have && !*gate.abort && !load(prev, true)) return drain();
    if (E4) {
        const int slot = nr % RING;
        if (!gate(&bar.r_empty[slot], ((nr / RING) & 1) ^ 1)) return drain();
        if (lane == 0) {
            reinterpret_cast<int *>(sm + C::OFF_DESC)[slot] = -1;
            mbar_arrive(&bar.r_full[slot]);
        }
        __syncwarp();
    }
    if (*gate.abort) drain();
}

// ---------------------------------------------------------------- widening
// e4m3 to fp16, 256 threads: a thread takes 64 of a row's 128 channels.  Rows that no
// key stands in become zeros (V: 0 x NaN is NaN).
template <int NR>
__device__ __forceinline__ void widen_role(uint8_t *sm, const Gate &gate) {
    using C = Cfg<true, NR>;
    const Bars<C> bar(sm);
    const int tid = threadIdx.x - W_WIDEN * 32, lane = tid & 31, row = tid & 127, hf = tid >> 7;
    int nk = 0, nv = 0;
    for (int n = 0;; ++n) {
        const int slot = n % C::RS;
        if (!gate(&bar.r_full[slot], (n / C::RS) & 1)) return;
        const int z = reinterpret_cast<const volatile int *>(sm + C::OFF_DESC)[slot];
        if (z < 0) return;
        const bool v = z >> 16;
        const uint8_t *src = sm + C::OFF_R + slot * RAW + row * 128;
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint4 *>(src + (((4 * hf + i) ^ (row & 7)) << 4));
        const bool live = row >= (z & 255) && row < ((z >> 8) & 255);
        uint8_t *dst;
        if (v) {
            const int s = nv % C::VS;
            if (!gate(&bar.v_empty[s], ((nv / C::VS) & 1) ^ 1)) return;
            dst = sm + C::OFF_V + s * TILE;
        } else {
            const int s = nk % C::KS;
            if (!gate(&bar.k_empty[s], ((nk / C::KS) & 1) ^ 1)) return;
            dst = sm + C::OFF_K + s * TILE;
        }
        dst += hf * (TILE / 2) + row * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t h[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x[k] & 0xffff), __NV_E4M3);
                const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x[k] >> 16), __NV_E4M3);
                h[2 * k] = live ? (uint32_t)lo.x | ((uint32_t)lo.y << 16) : 0u;
                h[2 * k + 1] = live ? (uint32_t)hi.x | ((uint32_t)hi.y << 16) : 0u;
            }
            *reinterpret_cast<uint4 *>(dst + (((2 * i) ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(dst + (((2 * i + 1) ^ (row & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&bar.r_empty[slot]);
            mbar_arrive(v ? &bar.v_full[nv % C::VS] : &bar.k_full[nk % C::KS]);
        }
        if (v) ++nv;
        else ++nk;
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

template <bool E4, int NR>
__device__ __forceinline__ void mma_role(uint8_t *sm, uint32_t tmem, const Gate &gate) {
    using C = Cfg<E4, NR>;
    const Bars<C> bar(sm);
    // fp16 operands have type 0 where bf16 has 1; K and Q are K-major, V^T and P^T run along M and N
    constexpr uint32_t TYPES = E4 ? 0u : (1u << 7) | (1u << 10);
    constexpr uint32_t ID_S = (1u << 4) | TYPES | ((uint32_t)(NR >> 3) << 17) | ((128u >> 4) << 24);
    constexpr uint32_t ID_O = ID_S | (1u << 15) | (1u << 16);
    const uint32_t base = smem_u32(sm);
    const uint64_t dk = sdesc_sw128(base + C::OFF_K), dq = sdesc_sw128(base + C::OFF_Q),
                   dv = sdesc_mn(base + C::OFF_V, TILE / 2, 1024, SWZ_128B), dp = sdesc_mn(base + C::OFF_P, BK * 32, 256, SWZ_32B);
    int nk = 0, nv = 0;              // S and O products issued
    int nt = 0, j = 0, item = -1, iseg = 0;
    int first0 = 0, first1 = 0, ob0 = 0, ob1 = 0;  // of the two tiles ahead: does it begin its item, whose O
    bool ok = true, more = true;
    auto ahead = [&]() {             // the next tile's S
        while (more && j == nt) {
            Seg s;
            if (!next_seg<C>(sm, bar, iseg, gate, s)) {
                more = false;
                ok = ok && !*gate.abort;
                return;
            }
            if (s.nt == 0) continue;
            nt = s.nt;
            j = 0;
            ++item;
            ok = gate(&bar.q_full[item & 1], (item >> 1) & 1) && ok;
        }
        if (!more || !ok) return;
        const int b = nk & 1, slot = nk % C::KS, x = item & 1;
        ok = gate(&bar.k_full[slot], (nk / C::KS) & 1);
        if (!ok) return;
        tc_fence_after();
        const uint64_t q = dq + (uint32_t)x * (C::QB >> 4);
        issue_s(tmem + b * NR, dk + (uint32_t)slot * (TILE >> 4), q, q + (NR * 128 >> 4), ID_S);
        mma_commit_w(&bar.s_full[b]);
        mma_commit_w(&bar.k_empty[slot]);
        if (j == nt - 1) mma_commit_w(&bar.q_empty[x]);
        if (b) first1 = j == 0, ob1 = x;
        else first0 = j == 0, ob0 = x;
        ++j;
        ++nk;
    };
    int items = 0;  // whose O has begun
    ahead();
    ahead();
    while (ok && nv < nk) {
        const int b = nv & 1, slot = nv % C::VS, first = b ? first1 : first0, ob = b ? ob1 : ob0;
        ok = gate(&bar.v_full[slot], (nv / C::VS) & 1);
        if (first) {  // the item before last must have left this O
            ok = gate(&bar.o_free[ob], ((items >> 1) & 1) ^ 1) && ok;
            ++items;
        }
        ok = gate(&bar.p_ready[b], (nv >> 1) & 1) && ok;
        if (!ok) break;
        tc_fence_after();
        issue_o(tmem + 2 * NR + ob * NR, dv + (uint32_t)slot * (TILE >> 4), dp + (uint32_t)b * (C::PB >> 4), ID_O, !first);
        mma_commit_w(&bar.pv_done[b]);
        mma_commit_w(&bar.v_empty[slot]);
        ++nv;
        ahead();
    }
    if (!ok || *gate.abort) {  // let the products in flight end before TMEM is given back
        mma_commit_w(bar.last);
        mbar_wait(bar.last, 0);
        __syncwarp();
    }
}

// ---------------------------------------------------------------- softmax
__device__ __forceinline__ int ordered(float x) {  // the same order among integers
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

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

// Thread = key of a tile, and channel of O.  A wait that runs out is passed on at the
// next meeting, so that all four warps leave together.
template <bool E4, int NR>
__device__ __forceinline__ void softmax_role(const PagedAttn &a, uint8_t *sm, uint32_t tmem, const Gate &gate) {
    using C = Cfg<E4, NR>;
    const Bars<C> bar(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t lanes = (uint32_t)warp << 21;  // 32 warp << 16
    float *refs = reinterpret_cast<float *>(sm + C::OFF_REF), *corrs = reinterpret_cast<float *>(sm + C::OFF_CORR);
    const int G = a.G;
    int n = 0, item = 0;  // tiles, items with tiles so far
    bool failed = false;
    for (int iseg = 0;; ++iseg) {
        if (!gate(&bar.seg_full[iseg % SEGS], (iseg / SEGS) & 1)) {
            meet_count<SOFT * 32>(1, true);
            return;
        }
        const Seg *sg = reinterpret_cast<const Seg *>(sm + C::OFF_SEG + (iseg % SEGS) * 64);
        const int nt = sg->nt;
        if (nt < 0) {
            meet_count<SOFT * 32>(1, false);
            return;
        }
        const float *sc = reinterpret_cast<const float *>(sm + C::OFF_SC) + (iseg % SEGS) * NR;
        const int lo = sg->lo, hi = sg->hi, t0 = sg->t0, pos = sg->pos, R = sg->R, r0 = sg->r0;
        const uint32_t to = tmem + lanes + 2 * NR + (item & 1) * NR;
        float l[NR], top = -INFINITY;  // sums of this thread's keys; row tid's maximum at the last change of ref
#pragma unroll
        for (int r = 0; r < NR; ++r) l[r] = 0.f;
        for (int j = 0; j < nt; ++j, ++n) {
            const int b = n & 1, key0 = (t0 + j) * BK, key = key0 + tid;
            if (!gate(&bar.s_full[b], (n >> 1) & 1)) failed = true;
            tc_fence_after();
            float t[NR];
            tmem_row<NR>(tmem + lanes + b * NR, t);
            // rows that see this key: [first, last)
            const int d = min(max(key - pos, 0), NR + 1), u = a.window > 0 ? min(max(key - pos + a.window, 0), NR + 1) : NR + 1;
            const int first = key < hi ? d * G - r0 : NR, last = u > NR ? NR : u * G - r0;
            if (__any_sync(0xffffffffu, first > 0 || last < R)) {
#pragma unroll
                for (int r = 0; r < NR; ++r) t[r] = r >= first && r < last ? t[r] : -INFINITY;
            }
            bool grow = j == 0;
            if (j > 0) {
                float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                for (int r = 0; r < NR; r += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(sc + r), g = *reinterpret_cast<const float4 *>(refs + r);
                    m0 = max3(m0, fmaf(t[r], f.x, -g.x), fmaf(t[r + 1], f.y, -g.y));
                    m1 = max3(m1, fmaf(t[r + 2], f.z, -g.z), fmaf(t[r + 3], f.w, -g.w));
                }
                grow = fmaxf(m0, m1) > GROW;
            }
            grow = __any_sync(0xffffffffu, grow);
            // a warp that gave up counts 32, one that saw a maximum grow 1
            const int said = meet_count<SOFT * 32>(1, failed || (grow && lane == 0));
            if (said >= 32) return;
            uint8_t *pb = sm + C::OFF_P + b * C::PB;
            if (said) {
                // largest score of each row over the tile (P's buffer is free: it holds the warps' maxima)
                float *wm = reinterpret_cast<float *>(pb) + warp * NR;
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const int m = __reduce_max_sync(0xffffffffu, ordered(t[r] * sc[r]));
                    if (lane == (r & 31)) wm[r] = unordered(m);
                }
                meet_count<SOFT * 32>(1, false);
                if (tid < NR) {
                    const float *all = reinterpret_cast<const float *>(pb);
                    const float was = j == 0 ? -INFINITY : top, ref = refs[tid];
                    float m = was;
#pragma unroll
                    for (int w = 0; w < SOFT; ++w) m = fmaxf(m, all[w * NR + tid]);
                    // a row that had seen nothing has zeros in O and in its sums, and a reference
                    // that its first score will be far above
                    const float next = m == -INFINITY ? NOTHING : was == -INFINITY ? m : fmaxf(m, ref);
                    corrs[tid] = was == -INFINITY ? 0.f : ex2(ref - next);
                    refs[tid] = next;
                    top = m;
                }
                meet_count<SOFT * 32>(1, false);
                if (j > 0) {
                    if (!gate(&bar.pv_done[b ^ 1], ((n - 1) >> 1) & 1)) failed = true;  // the last product must have left O
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < NR; c += 16) {
                        float o[16];
                        uint32_t w[16];
                        tmem_ld16(to + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            asm volatile("" : "+f"(o[i]));
                            w[i] = __float_as_uint(o[i] * corrs[c + i]);
                        }
                        tmem_st16(to + c, w);
                    }
                    tmem_st_wait();
#pragma unroll
                    for (int r = 0; r < NR; ++r) l[r] *= corrs[r];
                }
            }
            uint32_t p[NR / 2];
#pragma unroll
            for (int r = 0; r < NR; r += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(sc + r), g = *reinterpret_cast<const float4 *>(refs + r);
                const float e0 = ex2(fmaf(t[r], f.x, -g.x)), e1 = ex2(fmaf(t[r + 1], f.y, -g.y));
                const float e2 = ex2(fmaf(t[r + 2], f.z, -g.z)), e3 = ex2(fmaf(t[r + 3], f.w, -g.w));
                l[r] += e0;
                l[r + 1] += e1;
                l[r + 2] += e2;
                l[r + 3] += e3;
                p[r / 2] = E4 ? pack_f16(e0, e1) : pack_bf16(e0, e1);
                p[r / 2 + 1] = E4 ? pack_f16(e2, e3) : pack_bf16(e2, e3);
            }
            // [key][row], blocks of 16 rows, the two 16-byte halves swapped on every other group of four keys
#pragma unroll
            for (int c = 0; c < NR / 8; ++c)
                *reinterpret_cast<uint4 *>(pb + (c >> 1) * BK * 32 + tid * 32 + (((c & 1) ^ ((tid >> 2) & 1)) << 4)) =
                    make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
            if (!E4) {
                // a row of V that no key stands in may hold anything: zero it (0 x NaN is NaN)
                const bool none = key >= hi || key < (lo & ~(a.box - 1));
                if (__any_sync(0xffffffffu, none)) {
                    if (!gate(&bar.v_full[n % C::VS], (n / C::VS) & 1)) failed = true;
                    uint8_t *vt = sm + C::OFF_V + (n % C::VS) * TILE + tid * 128;
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
            if (lane == 0) mbar_arrive(&bar.p_ready[b]);
        }

        // ---- the segment's end: sums over the keys, then O, normalised or as a piece
        const bool whole = sg->whole;
        const int64_t tok = sg->tok;
        const int head0 = sg->h * G;
        float *slot = paged_slot(a, sg->slot);
        float *sums = reinterpret_cast<float *>(sm + C::OFF_P);  // [NR][128]: both P buffers, their products done
        if (nt > 0) {
            if (!gate(&bar.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1)) failed = true;
            tc_fence_after();
#pragma unroll
            for (int r = 0; r < NR; ++r) sums[r * 128 + tid] = l[r];
            if (meet_count<SOFT * 32>(1, failed) >= 32) return;
#pragma unroll 4
            for (int r = warp; r < NR; r += SOFT) {
                const float4 x = *reinterpret_cast<const float4 *>(sums + r * 128 + 4 * lane);
                float y = (x.x + x.y) + (x.z + x.w);
#pragma unroll
                for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                if (lane == 0) corrs[r] = y;
            }
            meet_count<SOFT * 32>(1, false);
            const float vs = E4 ? a.v_scale[sg->h] : 1.f;
#pragma unroll 1
            for (int c = 0; c < NR; c += 16) {
                if (c >= R) break;
                float o[16];
                tmem_ld16(to + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    asm volatile("" : "+f"(o[i]));
                    const int r = c + i;
                    if (r >= R) continue;
                    const float L = corrs[r];
                    if (whole) {
                        const int rr = r0 + r, jt = rr / G;
                        const float y = L == 0.f ? 0.f : o[i] * (vs / L);
                        reinterpret_cast<__nv_bfloat16 *>(a.o)[((tok + jt) * a.Hq + head0 + rr - jt * G) * D + tid] = __float2bfloat16_rn(y);
                    } else {
                        slot[2 * a.slot_rows + r * D + tid] = o[i];
                    }
                }
            }
        } else if (whole) {
            for (int r = 0; r < R; ++r) {
                const int rr = r0 + r, jt = rr / G;
                reinterpret_cast<__nv_bfloat16 *>(a.o)[((tok + jt) * a.Hq + head0 + rr - jt * G) * D + tid] = __float2bfloat16_rn(0.f);
            }
        } else {
            for (int r = 0; r < R; ++r) slot[2 * a.slot_rows + r * D + tid] = 0.f;
        }
        if (tid < R) {
            const float L = nt > 0 ? corrs[tid] : 0.f, ref = nt > 0 ? refs[tid] : 0.f;
            if (!whole) {
                reinterpret_cast<float2 *>(slot)[tid] = make_float2(L == 0.f ? -INFINITY : ref, L);
            } else if (a.lse) {
                const int rr = r0 + tid, jt = rr / G;
                a.lse[(tok + jt) * a.Hq + head0 + rr - jt * G] = L == 0.f ? -INFINITY : (ref + log2f(L)) * 0.6931471805599453f;
            }
        }
        if (tid == 0 && !whole && sg->c0 == (int)blockIdx.x) {
            a.lead[2 * blockIdx.x] = make_int4((int)tok, sg->h, r0, R);
            a.lead[2 * blockIdx.x + 1] = make_int4(sg->slot, sg->c0, sg->c1, 1);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if (nt > 0) mbar_arrive(&bar.o_free[item & 1]);
            mbar_arrive(&bar.seg_empty[iseg % SEGS]);
        }
        // (refs, corrs and the sums are written again only past the next tile's meeting)
        if (nt > 0) ++item;
    }
}

template <bool E4, int NR>
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
            mbar_init(&bar.k_full[i], E4 ? WIDEN : 1);
            mbar_init(&bar.k_empty[i], 1);
        }
        for (int i = 0; i < C::VS; ++i) {
            mbar_init(&bar.v_full[i], E4 ? WIDEN : 1);
            mbar_init(&bar.v_empty[i], 1);
        }
        for (int i = 0; i < C::RS; ++i) {
            mbar_init(&bar.r_full[i], 1);
            mbar_init(&bar.r_empty[i], WIDEN);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.q_full[i], 1);
            mbar_init(&bar.q_empty[i], 1);
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_ready[i], SOFT);
            mbar_init(&bar.pv_done[i], 1);
            mbar_init(&bar.o_free[i], SOFT);
        }
        for (int i = 0; i < SEGS; ++i) {
            mbar_init(&bar.seg_full[i], 1);
            mbar_init(&bar.seg_empty[i], SOFT + 2);
        }
        mbar_init(bar.last, 1);
        mbar_fence_init();
        sh->abort = 0;
        a.lead[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
    }
    auto units = [&](int i, int *err) { return line_units(a, i, rw, err); };
    const PagedLine line = paged_line<C::THREADS>(a, scratch, min_per, 1, units);
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
    if (warp == W_MMA) tmem_alloc(&sh->tmem, C::TCOLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    const Gate gate{&sh->abort, a.err};
    // e4m3 with 64 rows: 128 registers a thread at launch (512 x 128 = 65,536), 200 for
    // the softmax warps' 64 scores and sums, 104 for the others: 128 x 200 + 384 x 104
    constexpr bool SPLIT = E4 && NR == 64;
    if (warp < SOFT) {
        if constexpr (SPLIT) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        softmax_role<E4, NR>(a, sm, tmem, gate);
    } else {
        if constexpr (SPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    }
    if (warp == W_MMA) {
        mma_role<E4, NR>(sm, tmem, gate);
    } else if (warp == W_LOAD) {
        load_role<E4, NR>(a, maps, sm, gate);
    } else if (warp == W_WALK) {
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
    } else if (E4 && warp >= W_WIDEN) {
        if constexpr (E4) widen_role<NR>(sm, gate);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TCOLS);
    }
}

template <bool E4, int NR>
int launch(const PagedAttn &a, const PagedMaps &maps, cudaStream_t s) {
    using C = Cfg<E4, NR>;
    const int rc = prepare_kernel((const void *)paged_few_kernel<E4, NR>, C::SMEM, C::THREADS, nullptr);
    if (rc) return rc;
    paged_few_kernel<E4, NR><<<paged_few_blocks(), C::THREADS, C::SMEM, s>>>(maps, a, 3);
    note_launch("paged_few", s);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

int paged_few_blocks() { return device_sm_count(); }

int launch_paged_few(PagedAttn a, int cache_dtype, const void *k, const void *v, int64_t page_stride, int64_t max_rows,
                     cudaStream_t s) {
    int box = 16;
    while (box < BK && a.page_size % (2 * box) == 0) box *= 2;
    a.box = box;
    PagedMaps maps;
    const int rc = make_paged_maps(k, v, cache_dtype, a.Hkv, a.page_size, a.n_pages, page_stride, box, &maps);
    if (rc) return rc;
    const bool e4 = cache_dtype == KDA_E4M3;
    if (max_rows <= 16) return e4 ? launch<true, 16>(a, maps, s) : launch<false, 16>(a, maps, s);
    if (max_rows <= 32) return e4 ? launch<true, 32>(a, maps, s) : launch<false, 32>(a, maps, s);
    return e4 ? launch<true, 64>(a, maps, s) : launch<false, 64>(a, maps, s);
}

}  // namespace kda
