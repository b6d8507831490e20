// kda_paged_tile.cu -- paged attention on tcgen05 tensor cores, for bf16 caches
// and requests with more rows than the rows kernel takes.
//
// One block per SM: eight softmax warps (two groups of 128 threads, a thread to
// a row), one warp that issues the products, one that has the tensor memory
// accelerator load Q, K and V.  An item is up to two halves of 128 rows (whole
// tokens: floor(128 / G) of them times G heads) of one kv head; key tiles are
// 128 keys.
//   S_w = Q_w K^T   128 x 128 fp32 in TMEM
//   P_w = exp2(S_w scale - ref) as bf16 over S_w's own columns (the softmax
//         group reads a row of S into registers, so nothing of S is needed)
//   O_w += P_w V    128 x 128 fp32 in TMEM, P_w read from TMEM
// The two groups w take turns: while one works out probabilities, the tensor
// cores run the other's products.  With over 128 rows the groups are the two
// halves of the rows and share each key tile; with fewer they take every other
// key tile of the same rows and are merged at the end (each group then has its
// own maximum, sum and O).
//
// The reference `ref` of a row's exponents follows its maximum only when that
// has grown by more than 2^8: until then probabilities up to 256 are as precise
// in bf16 and the sums stay in fp32, and O needs no rescaling (which would mean
// reading and writing 128 columns of TMEM between two products).
#include "kda_paged.cuh"

namespace kda {
namespace {
using namespace tc;

constexpr int BK = 128;                        // keys per tile
constexpr int BM = 128;                        // rows per half
constexpr int SLOTS = 5;                       // ring of K / V tiles
constexpr int SLOT = BK * D * 2;               // 32 KB: two 64-channel blocks of 128 rows x 128 B
constexpr int QHALF = BM * D * 2;
constexpr int OFF_Q = 0;
constexpr int OFF_KV = 2 * QHALF;
constexpr int OFF_ML = OFF_KV + SLOTS * SLOT;  // [2][128] float2
constexpr int OFF_BAR = OFF_ML + 2 * BM * 8;
constexpr int NBAR = 2 * SLOTS + 14 + 2 * 4;
constexpr int SEGS = 4;                        // ring of segments ahead of the roles
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;   // TMEM address, abort flag, start of the block's line
constexpr int OFF_SEG = OFF_MISC + 64;
constexpr int SMEM = OFF_SEG + SEGS * 64;
constexpr int SOFT = 8;                        // softmax warps
constexpr int THREADS = (SOFT + 4) * 32;       // (registers are given out by four warps: the last one has nothing to do)
// registers a thread: 168 at launch (384 x 168 = 64,512), then 208 for the softmax
// warps, which hold a row of S, and 88 for the others: 256 x 208 + 128 x 88 = 64,512
constexpr int REGS_SOFT = 208, REGS_AUX = 88;
static_assert(SOFT * 32 * REGS_SOFT + 128 * REGS_AUX <= THREADS * 168, "register split");
constexpr int TCOLS = 512;
constexpr uint32_t COL_S = 0, COL_O = 256;     // + 128 w
constexpr float GROW = 8.f;                    // log2 growth of a maximum that ref follows

struct Bars {
    uint64_t *kv_full, *kv_empty, *q_full, *q_empty, *s_full, *p_ready, *pv_done, *o_free, *meet, *seg_full, *seg_empty;
    __device__ explicit Bars(uint8_t *sm) {
        uint64_t *b = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
        kv_full = b;
        kv_empty = b + SLOTS;
        q_full = b + 2 * SLOTS;      // [2]
        q_empty = q_full + 2;        // [2]
        s_full = q_empty + 2;        // [2]
        p_ready = s_full + 2;        // [2]
        pv_done = p_ready + 2;       // [2]
        o_free = pv_done + 2;        // [2]
        meet = o_free + 2;           // [1], then one for products in flight when a wait ran out
        seg_full = meet + 2;
        seg_empty = seg_full + SEGS;
    }
};

// sum_{i < n} floor((a i + b) / m) for a, b >= 0: whole parts of a / m and b / m
// first; then, with K = floor((a (n - 1) + b) / m), counting the points below the
// line by rows instead of columns gives
//   K (n - 1) - sum_{j < K} floor((m j + m - b - 1) / a),
// the same kind of sum on smaller numbers (Euclid's steps on a and m).
__device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
    int64_t s = 0, sign = 1;
    while (n > 0) {
        const int64_t qa = a / m, qb = b / m;
        s += sign * (qa * (n * (n - 1) / 2) + qb * n);
        a -= qa * m;
        b -= qb * m;
        const int64_t K = (a * (n - 1) + b) / m;
        if (K == 0) break;
        s += sign * K * (n - 1);
        sign = -sign;
        b = m - b - 1;
        n = K;
        const int64_t t = m;
        m = a;
        a = t;
    }
    return s;
}

// One request's row tiles: TT = 2 th tokens each (th = floor(128 / G)).
struct TileReq {
    PagedReq r;
    int n, ng;
};
__device__ __forceinline__ TileReq tile_req(const PagedAttn &a, int i, int th, int *err) {
    TileReq q;
    q.r = paged_req(a, i, err);
    q.n = q.r.rows / a.G;
    q.ng = (q.n + 2 * th - 1) / (2 * th);
    return q;
}
// Key tiles [t0, t1) of the tokens j0 .. j1 of a request (none: t1 = t0).
__device__ __forceinline__ void key_tiles(const PagedAttn &a, const PagedReq &r, int j0, int j1, int &lo, int &hi, int &t0, int &t1) {
    hi = r.pos0 + j1 + 1;
    lo = a.window > 0 ? max(0, r.pos0 + j0 - a.window + 1) : 0;
    if (hi <= 0) {
        t0 = t1 = 0;
        return;
    }
    t0 = lo / BK;
    t1 = (hi + BK - 1) / BK;
}
// Length of an item in the line: two units a tile (one product pair per half), one
// where the groups split the tiles, always even so that every cut falls on a tile
// of either kind; an item without keys takes the place of one tile.
__device__ __forceinline__ int item_units(const PagedAttn &a, const TileReq &q, int g, int th) {
    const int j0 = g * 2 * th, j1 = min(q.n, j0 + 2 * th) - 1;
    int lo, hi, t0, t1;
    key_tiles(a, q.r, j0, j1, lo, hi, t0, t1);
    const int nt = max(1, t1 - t0);
    return j1 - j0 + 1 > th ? 2 * nt : (nt + 1) & ~1;
}
// Units of the row tiles before g (closed form: a long request has thousands).
__device__ __forceinline__ int64_t units_before(const PagedAttn &a, const TileReq &q, int g, int th) {
    const int TT = 2 * th, full = min(g, q.n / TT);
    const int64_t pos0 = q.r.pos0;
    int64_t neg = pos0 < 0 ? -pos0 / TT : 0;  // tiles whose last query stands before position 0
    if (neg > full) neg = full;
    int64_t tiles = neg + floor_sum(full - neg, BK, TT, pos0 + (neg + 1) * TT + BK - 1);
    if (a.window > 0) {
        const int64_t d = a.window - 1 - pos0;  // lo > 0 from g TT > d on
        int64_t gw = d < 0 ? 0 : d / TT + 1;
        if (gw < neg) gw = neg;
        if (gw < full) tiles -= floor_sum(full - gw, BK, TT, gw * TT - d);
    }
    int64_t u = 2 * tiles;
    if (g > full) u += item_units(a, q, full, th);  // the last, shorter row tile
    return u;
}
__device__ __forceinline__ int64_t line_units(const PagedAttn &a, int i, int th, int *err) {
    const TileReq q = tile_req(a, i, th, err);
    return q.r.rows == 0 ? 0 : (int64_t)a.Hkv * units_before(a, q, q.ng, th);
}

// A block's segment of an item.
struct __align__(16) Seg {
    int tok, ntok;           // first token, tokens
    int h, pos;              // kv head, first token's position
    int lo, hi, t0, nt;      // keys seen, first key tile of the segment, its tiles (0: nothing to read)
    int req, alt, whole, slot, c0, c1, pad;
};
static_assert(sizeof(Seg) == 64, "segment size");

// The line's items from the block's start on.
struct Walk {
    int64_t pos, end, per, before, A;
    int req, h, g;
    TileReq q;
    bool fresh;
    __device__ bool next(const PagedAttn &a, int th, int64_t P0, Seg &s) {
        if (pos >= end) return false;
        if (fresh) {
            while (true) {
                q = tile_req(a, req, th, nullptr);
                if (q.r.rows) break;
                ++req;  // (the total says that a request with tiles follows)
            }
            fresh = false;
        }
        const int units = item_units(a, q, g, th);
        const int64_t B = A + units, stop = B < end ? B : end;
        const int j0 = g * 2 * th, j1 = min(q.n, j0 + 2 * th) - 1;
        int t0, t1;
        key_tiles(a, q.r, j0, j1, s.lo, s.hi, t0, t1);
        s.alt = j1 - j0 + 1 <= th;
        const int sh = s.alt ? 0 : 1;
        const int b = (int)(pos - A) >> sh, e = min((int)(stop - A) >> sh, t1 - t0);
        s.t0 = t0 + b;
        s.nt = max(0, e - b);
        s.tok = q.r.tok0 + j0;
        s.ntok = j1 - j0 + 1;
        s.h = h;
        s.pos = q.r.pos0 + j0;
        s.req = req;
        s.whole = pos == A && stop == B;
        s.slot = 2 * (int)blockIdx.x + (pos == P0 ? 0 : 1);
        s.c0 = (int)(A / per);
        s.c1 = (int)((B - 1) / per);
        pos = stop;
        if (stop == B) {
            A = B;
            if (++g == q.ng) {
                g = 0;
                if (++h == a.Hkv) {
                    h = 0;
                    ++req;
                    fresh = true;
                }
            }
        }
        return true;
    }
};

// Place of K_j and V_j in the order of loading, counted from the item's first:
// shared tiles K0 V0 K1 V1 ..; alternating K0 K1 V0 K2 V1 .. (two K tiles are
// multiplied before the first V).
__device__ __forceinline__ int seq_k(bool alt, int j) { return alt ? (j == 0 ? 0 : 2 * j - 1) : 2 * j; }
__device__ __forceinline__ int seq_v(bool alt, int j, int nt) { return alt ? (j == nt - 1 ? 2 * nt - 1 : 2 * j + 2) : 2 * j + 1; }

__device__ __forceinline__ void mma_ta_w(uint32_t d, uint32_t ta, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(ta), "l"(b), "r"(idesc), "r"((uint32_t)acc));
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *o) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
          "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *o) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]), "r"(o[8]), "r"(o[9]), "r"(o[10]),
        "r"(o[11]), "r"(o[12]), "r"(o[13]), "r"(o[14]), "r"(o[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

struct Shared {
    uint32_t tmem;
    int abort;
    int req, h, g;
    int pad;
    int64_t A;
};

struct Gate {  // bounded waits that stop the whole block when one runs out
    volatile int *abort;
    int32_t *err;
    __device__ bool operator()(uint64_t *bar, int parity) const {
        const bool ok = __all_sync(0xffffffffu, mbar_wait_ab(bar, parity, abort));
        if (!ok && (threadIdx.x & 31) == 0) {
            *abort = 1;
            if (err) atomicOr(err, KDA_DEVERR_TIMEOUT);
        }
        return ok;
    }
};

// One warp walks the line ahead of the others; a segment with nt < 0 ends it.
__device__ __forceinline__ void walk_role(const PagedAttn &a, uint8_t *sm, Walk w, int th, int64_t P0, const Gate &gate) {
    const int lane = threadIdx.x & 31;
    const Bars bar(sm);
    for (int i = 0;; ++i) {
        Seg s;
        const bool more = w.next(a, th, P0, s);
        if (!more) s.nt = -1;
        if (!gate(&bar.seg_empty[i % SEGS], ((i / SEGS) & 1) ^ 1)) return;
        if (lane == 0) {
            *reinterpret_cast<Seg *>(sm + OFF_SEG + (i % SEGS) * 64) = s;
            mbar_arrive(&bar.seg_full[i % SEGS]);
        }
        __syncwarp();
        if (!more) return;
    }
}
// The next segment, for a whole warp; false at the line's end.
__device__ __forceinline__ bool next_seg(uint8_t *sm, const Bars &bar, int &i, const Gate &gate, Seg &s) {
    if (!gate(&bar.seg_full[i % SEGS], (i / SEGS) & 1)) return false;
    s = *reinterpret_cast<const Seg *>(sm + OFF_SEG + (i % SEGS) * 64);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bar.seg_empty[i % SEGS]);
    ++i;
    return s.nt >= 0;
}

// ---------------------------------------------------------------- loads
__device__ __forceinline__ void load_role(const PagedAttn &a, const PagedMaps &maps, const CUtensorMap &qmap, uint8_t *sm,
                                          int th, const Gate &gate) {
    const int lane = threadIdx.x & 31;
    const Bars bar(sm);
    const int box = a.box, nbx = BK / box;
    int64_t seq = 0;   // K / V tiles so far
    int qn[2] = {0, 0};
    auto drain = [&]() {  // a wait ran out: let the copies in flight land before the block ends
        for (int64_t u = seq - 1; u >= 0 && u >= seq - SLOTS; --u) mbar_wait(&bar.kv_full[u % SLOTS], (u / SLOTS) & 1);
        for (int x = 0; x < 2; ++x)
            if (qn[x]) mbar_wait(&bar.q_full[x], (qn[x] - 1) & 1);
        __syncwarp();
    };
    Seg s;
    int iseg = 0;
    while (next_seg(sm, bar, iseg, gate, s)) {
        if (s.nt == 0) continue;
        const int nh = s.ntok > th ? 2 : 1;
        int cbase = -64, page = 0;
        const int lob = s.lo & ~(box - 1);  // boxes before this one hold no seen key (their pages may be gone)
        // one K or V tile
        auto tile = [&](int j, bool v) -> bool {
            const int key0 = (s.t0 + j) * BK, b0 = key0 / box;
            if (cbase < 0 || b0 < cbase || b0 + nbx > cbase + 32) {  // pages of the next 32 boxes, one per lane
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
            const int slot = (int)(seq % SLOTS);
            if (!gate(&bar.kv_empty[slot], (int)((seq / SLOTS) & 1) ^ 1)) return false;
            const int f = max(0, (lob - key0) / box), e = min(nbx, (s.hi - key0 + box - 1) / box);
            if (lane == 0) mbar_expect_tx(&bar.kv_full[slot], (uint32_t)((e - f) * box * D * 2));
            __syncwarp();
            const int pg = __shfl_sync(0xffffffffu, page, (b0 - cbase + lane) & 31);
            if (lane >= f && lane < e) {
                const int key = key0 + lane * box, y = s.h * a.page_size + key % a.page_size;
                uint8_t *dst = sm + OFF_KV + slot * SLOT + lane * box * 128;
                const CUtensorMap *m = v ? &maps.v : &maps.k;
                tma_load_3d(dst, m, 0, y, pg, &bar.kv_full[slot]);
                tma_load_3d(dst + SLOT / 2, m, 64, y, pg, &bar.kv_full[slot]);
            }
            __syncwarp();
            ++seq;
            return true;
        };
        for (int x = 0; x < nh; ++x) {
            if (!gate(&bar.q_empty[x], (qn[x] & 1) ^ 1)) return drain();
            if (lane == 0) {
                mbar_expect_tx(&bar.q_full[x], (uint32_t)(2 * th * a.G * 128));
                uint8_t *dst = sm + OFF_Q + x * QHALF;
                tma_load_3d(dst, &qmap, 0, s.h * a.G, s.tok + x * th, &bar.q_full[x]);
                tma_load_3d(dst + QHALF / 2, &qmap, 64, s.h * a.G, s.tok + x * th, &bar.q_full[x]);
            }
            __syncwarp();
            ++qn[x];
        }
        for (int j = 0; j < s.nt; ++j) {
            if (!s.alt) {
                if (!tile(j, false) || !tile(j, true)) return drain();
            } else {
                if (j == 0 && !tile(0, false)) return drain();
                if (j + 1 < s.nt && !tile(j + 1, false)) return drain();
                if (!tile(j, true)) return drain();
            }
        }
    }
}

// ---------------------------------------------------------------- products
__device__ __forceinline__ void mma_role(const PagedAttn &a, uint8_t *sm, uint32_t tmem, int th, const Gate &gate) {
    const Bars bar(sm);
    constexpr uint32_t ID_QK = idesc_bf16_f32(BM, BK), ID_PV = idesc_bf16_f32_bmn(BM, D);
    const uint32_t base = smem_u32(sm);
    int64_t seq0 = 0;
    int qn[2] = {0, 0}, np[2] = {0, 0}, ni[2] = {0, 0};  // halves of Q, products P V, items, by group
    Seg s;
    int iseg = 0;
    while (next_seg(sm, bar, iseg, gate, s)) {
        if (s.nt == 0) continue;
        const bool alt = s.alt;
        const int ne = alt ? s.nt : 2 * s.nt;  // events: one S and one P V of one group
        auto kv_ready = [&](int64_t q) { return gate(&bar.kv_full[q % SLOTS], (int)((q / SLOTS) & 1)); };
        auto qk = [&](int e) -> bool {
            const int x = e & 1, j = alt ? e : e >> 1;
            const int64_t q = seq0 + seq_k(alt, j);
            const int half = alt ? 0 : x;
            if (e == 0 || (!alt && e == 1))
                if (!gate(&bar.q_full[half], qn[half] & 1)) return false;
            if ((alt || x == 0) && !kv_ready(q)) return false;
            tc_fence_after();
            const uint32_t qa = base + OFF_Q + half * QHALF, ka = base + OFF_KV + (uint32_t)(q % SLOTS) * SLOT;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = (uint32_t)(k >> 2) * (SLOT / 2) + (uint32_t)(k & 3) * 32;
                mma_bf16_w(tmem + COL_S + x * 128, sdesc_sw128(qa + off), sdesc_sw128(ka + off), ID_QK, k > 0);
            }
            mma_commit_w(&bar.s_full[x]);
            if (alt || x == 1) mma_commit_w(&bar.kv_empty[q % SLOTS]);
            if (alt ? e == ne - 1 : e >= ne - 2) {
                mma_commit_w(&bar.q_empty[half]);
                ++qn[half];
            }
            return true;
        };
        auto pv = [&](int e) -> bool {
            const int x = e & 1, j = alt ? e : e >> 1;
            const int64_t q = seq0 + seq_v(alt, j, s.nt);
            if ((alt || x == 0) && !kv_ready(q)) return false;
            if (!gate(&bar.p_ready[x], np[x] & 1)) return false;
            if (e < 2) {  // the group's last item must have left O
                if (!gate(&bar.o_free[x], (ni[x] & 1) ^ 1)) return false;
                ++ni[x];
            }
            tc_fence_after();
            const uint32_t va = base + OFF_KV + (uint32_t)(q % SLOTS) * SLOT;
#pragma unroll
            for (int k = 0; k < BK / 16; ++k)
                mma_ta_w(tmem + COL_O + x * 128, tmem + COL_S + x * 128 + k * 8, sdesc_mn(va + k * 2048, SLOT / 2, 1024, SWZ_128B),
                         ID_PV, e >= 2 || k > 0);
            mma_commit_w(&bar.pv_done[x]);
            ++np[x];
            if (alt || x == 1) mma_commit_w(&bar.kv_empty[q % SLOTS]);
            return true;
        };
        bool ok = qk(0) && (ne < 2 || qk(1));
        for (int e = 0; ok && e < ne; ++e) ok = pv(e) && (e + 2 >= ne || qk(e + 2));
        if (!ok) {  // let the products in flight end before TMEM is given back
            uint64_t *last = bar.meet + 1;
            mma_commit_w(last);
            mbar_wait(last, 0);
            __syncwarp();
            return;
        }
        seq0 += 2 * s.nt;
    }
}

// ---------------------------------------------------------------- softmax
__device__ __forceinline__ void softmax_role(const PagedAttn &a, uint8_t *sm, uint32_t tmem, int th, const Gate &gate) {
    const Bars bar(sm);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, x = warp >> 2;  // group
    const int row = threadIdx.x & 127;                                         // row of the half = TMEM lane
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;                         // 32 (warp % 4) << 16
    const uint32_t ts = tmem + lanes + COL_S + x * 128, to = tmem + lanes + COL_O + x * 128;
    float2 *ml = reinterpret_cast<float2 *>(sm + OFF_ML);
    const float sc = a.scale_log2;
    const int box = a.box;
    int nev = 0, meets = 0;  // events of this group so far
    int64_t seq0 = 0;
    Seg s;
    int iseg = 0;
    while (next_seg(sm, bar, iseg, gate, s)) {
        const bool alt = s.alt;
        const int half = alt ? 0 : x;
        const int hrows = min(th, s.ntok - half * th) * a.G;  // rows of this half
        const int jt = row / a.G, pos = s.pos + half * th + jt;
        const int first_key = a.window > 0 ? pos - a.window + 1 : 0;  // keys first_key .. pos, all below hi
        float ref = 0.f, l = 0.f, top = -INFINITY;
        int mine = 0;  // events of this item
        for (int j = alt ? x : 0; j < s.nt; j += alt ? 2 : 1) {
            const int key0 = (s.t0 + j) * BK;
            if (!gate(&bar.s_full[x], nev & 1)) return;
            tc_fence_after();
            float v[BK];
#pragma unroll
            for (int c = 0; c < BK; c += 32) tmem_ld32(ts + c, v + c);
            tmem_ld_wait();
            // keys of the tile that this row sees: [c0, c1)
            const int c1 = min(pos + 1, s.hi) - key0, c0 = first_key - key0;
            if (__any_sync(0xffffffffu, c1 < BK || c0 > 0)) {
#pragma unroll
                for (int c = 0; c < BK; ++c) v[c] = c < c1 && c >= c0 ? v[c] : -INFINITY;
            }
            float m0 = v[0], m1 = v[1], m2 = v[2], m3 = v[3];
#pragma unroll
            for (int c = 4; c < BK; c += 4) {
                m0 = fmaxf(m0, v[c]);
                m1 = fmaxf(m1, v[c + 1]);
                m2 = fmaxf(m2, v[c + 2]);
                m3 = fmaxf(m3, v[c + 3]);
            }
            const float mt = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * sc;
            float corr = 1.f;
            if (mine == 0) {
                top = mt;
                ref = mt == -INFINITY ? 0.f : mt;
            } else {
                const bool grow = mt > (top == -INFINITY ? -INFINITY : ref + GROW);
                if (__any_sync(0xffffffffu, grow)) {
                    const float m = fmaxf(top, mt), nref = m == -INFINITY ? 0.f : fmaxf(m, top == -INFINITY ? m : ref);
                    corr = top == -INFINITY ? 0.f : ex2(ref - nref);  // (nothing summed yet: whatever O holds is zero)
                    ref = nref;
                    l *= corr;
                    // the group's last product must have left O
                    if (!gate(&bar.pv_done[x], (nev - 1) & 1)) return;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < D; c += 16) {
                        float o[16];
                        tmem_ld16(to + c, o);
                        tmem_ld_wait();
                        uint32_t u[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(o[i] * corr);
                        tmem_st16(to + c, u);
                    }
                    tmem_st_wait();
                }
                top = fmaxf(top, mt);
            }
            // probabilities, 32 at a time over S's own columns
            float l0 = 0.f, l1 = 0.f;
#pragma unroll
            for (int c = 0; c < BK; c += 32) {
                uint32_t p[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float e0 = ex2(fmaf(v[c + 2 * i], sc, -ref)), e1 = ex2(fmaf(v[c + 2 * i + 1], sc, -ref));
                    l0 += e0;
                    l1 += e1;
                    const __nv_bfloat162 b = __floats2bfloat162_rn(e0, e1);
                    p[i] = *reinterpret_cast<const uint32_t *>(&b);
                }
                tmem_st16(ts + c / 2, p);
            }
            l += l0 + l1;
            // rows of V that no key of this item stands in may hold anything: zero
            // them (0 x NaN is NaN); the group whose product comes first does it
            const int z0 = max(0, (s.lo & ~(box - 1)) - key0), z1 = min(BK, s.hi - key0);
            if ((z0 > 0 || z1 < BK) && (alt || x == 0)) {
                const int64_t q = seq0 + seq_v(alt, j, s.nt);
                if (!gate(&bar.kv_full[q % SLOTS], (int)((q / SLOTS) & 1))) return;
                uint8_t *vt = sm + OFF_KV + (q % SLOTS) * SLOT;
                for (int u = row; u < BK * 16; u += BM) {
                    const int r = u >> 4, c = u & 15;
                    if (r < z0 || r >= z1)
                        *reinterpret_cast<uint4 *>(vt + (c >> 3) * (SLOT / 2) + r * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.p_ready[x]);
            ++nev;
            ++mine;
        }
        seq0 += 2 * s.nt;

        // ---- the segment's end: O, normalised or as a piece
        const int G = a.G;
        // row `row` of this half -> local row of the item
        const int local = half * th * G + row;
        const bool live = row < hrows;
        const int64_t tok = s.tok + half * th + jt;
        const int head = s.h * G + (row - jt * G);
        if (!alt) {
            if (s.nt > 0) {
                if (!gate(&bar.pv_done[x], (nev - 1) & 1)) return;
                tc_fence_after();
            }
            float *slot = paged_slot(a, s.slot);
            const float f = l > 0.f || l != l ? (s.whole ? 1.f / l : 1.f) : 0.f;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float o[32];
                if (s.nt > 0) {
                    tmem_ld32(to + c, o);
                    tmem_ld_wait();
                }
                if (live) {
                    const bool dead = s.nt == 0 || l == 0.f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = dead ? 0.f : o[i] * f;
                    if (s.whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.o + (tok * a.Hq + head) * D + c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t u[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const __nv_bfloat162 b = __floats2bfloat162_rn(o[8 * i + 2 * k], o[8 * i + 2 * k + 1]);
                                u[k] = *reinterpret_cast<const uint32_t *>(&b);
                            }
                            dst[i] = make_uint4(u[0], u[1], u[2], u[3]);
                        }
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(slot + 2 * a.slot_rows + (size_t)local * D + c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
            }
            if (live) {
                if (s.whole) {
                    if (a.lse) a.lse[tok * a.Hq + head] = l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
                } else {
                    reinterpret_cast<float2 *>(slot)[local] = make_float2(l == 0.f ? -INFINITY : ref, l);
                }
            }
            if (s.nt > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.o_free[x]);
            }
        } else {
            // both groups hold every row: exchange (reference, sum), then each group
            // writes half of the channels of the merged row
            if (mine == 0) l = 0.f, top = -INFINITY;
            ml[x * BM + row] = make_float2(l == 0.f ? -INFINITY : ref, l);
            __syncwarp();
            if (mine > 0) {
                if (!gate(&bar.pv_done[x], (nev - 1) & 1)) return;
            }
            // (this warp has seen its own group's last product end; the meeting
            // passes that on to the other group's warps)
            tc_fence_before();
            if (lane == 0) mbar_arrive(bar.meet);
            if (!gate(bar.meet, meets & 1)) return;
            ++meets;
            tc_fence_after();
            const float2 y0 = ml[row], y1 = ml[BM + row];
            const float m = fmaxf(y0.x, y1.x), rf = m == -INFINITY ? 0.f : m;
            const float f0 = y0.y == 0.f ? 0.f : ex2(y0.x - rf), f1 = y1.y == 0.f ? 0.f : ex2(y1.x - rf);
            const float L = f0 * y0.y + f1 * y1.y;
            float *slot = paged_slot(a, s.slot);
            const bool dead = L == 0.f;
            const float inv = s.whole && !dead ? 1.f / L : 1.f;
            const uint32_t o0 = tmem + lanes + COL_O;
#pragma unroll 1
            for (int c = x * 64; c < x * 64 + 64; c += 32) {
                float o[32], p[32];
                if (s.nt > 0) {
                    tmem_ld32(o0 + c, o);
                    if (s.nt > 1) tmem_ld32(o0 + 128 + c, p);
                    tmem_ld_wait();
                }
                if (live) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float z = 0.f;
                        if (s.nt > 0 && f0 != 0.f) z = f0 * o[i];
                        if (s.nt > 1 && f1 != 0.f) z += f1 * p[i];
                        o[i] = dead ? 0.f : z * inv;
                    }
                    if (s.whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.o + (tok * a.Hq + head) * D + c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t u[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const __nv_bfloat162 b = __floats2bfloat162_rn(o[8 * i + 2 * k], o[8 * i + 2 * k + 1]);
                                u[k] = *reinterpret_cast<const uint32_t *>(&b);
                            }
                            dst[i] = make_uint4(u[0], u[1], u[2], u[3]);
                        }
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(slot + 2 * a.slot_rows + (size_t)local * D + c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
            }
            if (live && x == 0) {
                if (s.whole) {
                    if (a.lse) a.lse[tok * a.Hq + head] = dead ? -INFINITY : (rf + log2f(L)) * 0.6931471805599453f;
                } else {
                    reinterpret_cast<float2 *>(slot)[local] = make_float2(dead ? -INFINITY : rf, L);
                }
            }
            // O of both groups is read by both: second meeting, then each frees its own
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.meet);
            if (!gate(bar.meet, meets & 1)) return;
            ++meets;
            if (mine > 0 && lane == 0) mbar_arrive(&bar.o_free[x]);
        }
        if (!s.whole && s.c0 == (int)blockIdx.x && threadIdx.x == 0) {
            a.lead[2 * blockIdx.x] = make_int4(s.tok, s.h, 0, s.ntok * a.G);
            a.lead[2 * blockIdx.x + 1] = make_int4(s.slot, s.c0, s.c1, 1);
        }
    }
}

__global__ void __launch_bounds__(THREADS, 1)
    paged_tile_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ CUtensorMap qmap, const PagedAttn a, int th,
                      int min_per) {
    extern __shared__ __align__(1024) uint8_t sm[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Shared *sh = reinterpret_cast<Shared *>(sm + OFF_MISC);
    int64_t *scratch = reinterpret_cast<int64_t *>(sm + OFF_ML);
    const Bars bar(sm);
    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&bar.kv_full[i], 1);
            mbar_init(&bar.kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.q_full[i], 1);
            mbar_init(&bar.q_empty[i], 1);
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_ready[i], 4);
            mbar_init(&bar.pv_done[i], 1);
            mbar_init(&bar.o_free[i], 4);
        }
        for (int i = 0; i < SEGS; ++i) {
            mbar_init(&bar.seg_full[i], 1);
            mbar_init(&bar.seg_empty[i], SOFT + 2);
        }
        mbar_init(bar.meet, SOFT);
        mbar_init(bar.meet + 1, 1);
        mbar_fence_init();
        sh->abort = 0;
        a.lead[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
    }
    auto units = [&](int i, int *err) { return line_units(a, i, th, err); };
    const int64_t total = paged_total<THREADS>(a, scratch, units);
    int64_t per = (total + gridDim.x - 1) / gridDim.x;
    if (per < min_per) per = min_per;
    per = (per + 1) & ~(int64_t)1;
    const int64_t P0 = (int64_t)blockIdx.x * per, P1 = P0 + per < total ? P0 + per : total;
    if (P0 >= P1) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    int req;
    int64_t before;
    paged_find<THREADS>(a, P0, scratch, req, before, units);
    if (warp == 0) {  // kv head and row tile of the block's first unit
        const TileReq q = tile_req(a, req, th, nullptr);
        const int64_t head = units_before(a, q, q.ng, th);
        const int h = (int)((P0 - before) / head);
        const int64_t rem = P0 - before - h * head;
        // the last row tile that begins at or before rem, 32 candidates at a time
        int lo = 0, n = q.ng;
        while (n > 1) {
            const int step = (n + 31) / 32, g = lo + lane * step;
            const bool at = lane * step < n && units_before(a, q, g, th) <= rem;
            const int k = 31 - __clz(__ballot_sync(0xffffffffu, at));
            lo += k * step;
            n = min(step, n - k * step);
        }
        if (lane == 0) {
            sh->req = req;
            sh->h = h;
            sh->g = lo;
            sh->A = before + h * head + units_before(a, q, lo, th);
        }
    }
    if (warp == SOFT) tmem_alloc(&sh->tmem, TCOLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    Walk w;
    w.pos = P0;
    w.end = P1;
    w.per = per;
    w.A = sh->A;
    w.req = sh->req;
    w.h = sh->h;
    w.g = sh->g;
    w.fresh = true;
    const Gate gate{&sh->abort, a.err};
    if (warp < SOFT) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFT));
        softmax_role(a, sm, tmem, th, gate);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_AUX));
        if (warp == SOFT)
            mma_role(a, sm, tmem, th, gate);
        else if (warp == SOFT + 1)
            load_role(a, maps, qmap, sm, th, gate);
        else if (warp == SOFT + 2)
            walk_role(a, sm, w, th, P0, gate);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == SOFT) {
        tc_fence_after();
        tmem_dealloc(tmem, TCOLS);
    }
    // the join waits for this grid; this grid may run beside the rows kernel, so it
    // ends only after that one
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace

int paged_tile_blocks() { return device_sm_count(); }

int launch_paged_tile(PagedAttn a, const void *k, const void *v, int64_t page_stride, bool after_rows, cudaStream_t s) {
    int box = 16;
    while (box < BK && a.page_size % (2 * box) == 0) box *= 2;
    a.box = box;
    const int th = BM / a.G;
    PagedMaps maps;
    CUtensorMap qmap;
    int rc = make_paged_maps(k, v, KDA_BF16, a.Hkv, a.page_size, a.n_pages, page_stride, box, &maps);
    if (rc) return rc;
    if ((rc = make_paged_q_map(a.q, a.T, a.Hq, a.G, th, &qmap))) return rc;
    const void *f = (const void *)paged_tile_kernel;
    if ((rc = prepare_kernel(f, SMEM, THREADS, nullptr))) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(paged_tile_blocks());
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = after_rows ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_tile_kernel, maps, qmap, a, th, 8);
    note_launch("paged_tile", s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace kda
