// kda_paged_tile.cu -- paged attention on tcgen05 tensor cores, for bf16 caches
// and requests with more rows than the kernel for few rows takes.
//
// One block per SM: sixteen softmax warps (two groups of 256 threads, two threads
// to a row, each with half of its keys), a warp that issues each group's products,
// one that has the tensor memory accelerator load K and V, and one that walks the
// block's items and has Q loaded.  An item is up to two halves of 128 rows (whole
// tokens: floor(128 / G) of them times G heads) of one kv head; key tiles are
// 128 keys.
//   S_w = Q_w K^T   128 x 128 fp32 in TMEM
//   P_w = exp2(S_w scale - ref) as bf16 over S_w's own columns (the softmax
//         group reads a row of S into registers, so nothing of S is needed)
//   O_w += P_w V    128 x 128 fp32 in TMEM, P_w read from TMEM
// The two groups w are the two halves of the rows and share each key tile; an item
// of one half has the first group alone.  Each group takes a tile in two steps of 64
// keys, whose S stand side by side: while it works out the probabilities of one, the
// tensor cores run the other's P V and, over the same columns, the next S.  (Whole
// tiles, one S a group: prompt 242 us, windows 311 us; the groups made to take turns:
// 234 and 292 us.  Registers given out by role: 229 and 268 us, when it was 223 and 262
// without.)
//
// The reference `ref` of a row's exponents follows its maximum only when that
// has grown by more than 2^8: until then probabilities up to 256 are as precise
// in bf16 and the sums stay in fp32, and O needs no rescaling (which would mean
// reading and writing 128 columns of TMEM between two products).  Probabilities are
// bf16 because a product's operands have one type, and V is bf16; the sums take them
// unrounded.
//
// Measured: a prompt of 8,192 tokens, 16 heads over two kv heads, 224 us (1,225
// TFLOP/s of the pairs that the mask leaves; some tiles more are multiplied where it
// crosses them); 2,048 tokens, 32 heads, over 65,536 keys 1,501 to 1,541 us (1,405 to
// 1,442 TFLOP/s, by the box: the clock falls under the load); 256 windows of 60 rows 258 us (5.8 TB/s).  Bound by the
// products (S for 64 keys reads its operands, by their bytes, at three quarters of the
// rate) and by what the way from S to P leaves between them.  (A share of the
// exponentials by a polynomial made it slower, 250 to 276 us for 242 us: the special
// function unit is not what it waits for.)
#include "kda_paged_tc.cuh"

namespace kda {
namespace {
using namespace tc;

constexpr int BK = KEY_TILE;                   // keys per tile
constexpr int BM = 128;                        // rows per half
constexpr int SLOTS = 5;                       // ring of K / V tiles
constexpr int SLOT = BK * D * 2;               // 32 KB: two 64-channel blocks of 128 rows x 128 B
constexpr int QHALF = BM * D * 2;
constexpr int HALF_K = (BK / 2 * 128) >> 4;    // from a K or V tile's first 64 keys to the others, in descriptor units
constexpr int OFF_Q = 0;
constexpr int OFF_KV = 2 * QHALF;
constexpr int OFF_SCAN = OFF_KV + SLOTS * SLOT;  // the start's sums
constexpr int OFF_BAR = OFF_SCAN + 256;
constexpr int SEGS = 4;                        // ring of segments ahead of the roles
constexpr int NBAR = 2 * SLOTS + 20 + 2 * SEGS;
constexpr int OFF_MISC = (OFF_BAR + NBAR * 8 + 63) / 64 * 64;  // TMEM address, abort flag
constexpr int OFF_SEG = OFF_MISC + 64;
constexpr int OFF_MX = OFF_SEG + SEGS * 64;    // [group][half of the keys][row] maximum, sum
constexpr int SMEM = OFF_MX + 4 * BM * 4;
static_assert(OFF_SCAN % 16 == 0 && OFF_BAR % 8 == 0 && OFF_SEG % 64 == 0 && SMEM <= 232448, "shared memory layout");
constexpr int SOFT = 16;                       // softmax warps
constexpr int THREADS = (SOFT + 4) * 32;
constexpr int TCOLS = 512;
constexpr uint32_t COL_S = 0, COL_O = 256;     // + 128 w
constexpr float GROW = 8.f;                    // log2 growth of a maximum that ref follows

struct Bars {
    uint64_t *kv_full, *kv_empty, *q_full, *q_empty, *s_full, *p_ready, *pv_done, *o_free, *last, *seg_full, *seg_empty;
    __device__ explicit Bars(uint8_t *sm) {
        uint64_t *b = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
        kv_full = b;
        kv_empty = b + SLOTS;
        q_full = b + 2 * SLOTS;      // [2]
        q_empty = q_full + 2;        // [2]
        s_full = q_empty + 2;        // [group][half of a tile's keys]
        p_ready = s_full + 4;        // the same
        pv_done = p_ready + 4;       // the same
        o_free = pv_done + 4;        // [2]
        last = o_free + 2;           // [2] a warp's products
        seg_full = last + 2;
        seg_empty = seg_full + SEGS;
    }
};

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
// Length of an item in the line: first some units for what an item costs besides
// its tiles (the first S, O on its way out), then one for each tile, of one half or
// two: alone, a half is no sooner through its way from S to P V.  (Heads of 1 and 2,
// 2 and 2, 2 and 4, 3 and 4 tiles: each slower on windows or on prompts by 2 to 8%.)
// An item without keys takes the place of one tile.  A cut inside the fixed part
// leaves the item to the next block.
__host__ __device__ constexpr int item_head(bool alt) { return alt ? 1 : 3; }
__device__ __forceinline__ int item_units(const PagedAttn &a, const TileReq &q, int g, int th) {
    const int j0 = g * 2 * th, j1 = min(q.n, j0 + 2 * th) - 1;
    int lo, hi, t0, t1;
    key_tiles(a, q.r, j0, j1, lo, hi, t0, t1);
    const int nt = max(1, t1 - t0);
    const bool alt = j1 - j0 + 1 <= th;
    return item_head(alt) + nt;
}
// Units of the row tiles before g (closed form: a long request has thousands).
__device__ __forceinline__ int64_t units_before(const PagedAttn &a, const TileReq &q, int g, int th) {
    const int TT = 2 * th, full = min(g, q.n / TT);
    const int pos0 = q.r.pos0;
    int neg = pos0 < 0 ? -pos0 / TT : 0;  // tiles whose last query stands before position 0
    if (neg > full) neg = full;
    int64_t tiles = neg + floor_sum(full - neg, BK, TT, pos0 + (neg + 1) * TT + BK - 1);
    if (a.window > 0) {
        const int d = window_from(a, pos0);  // lo > 0 from g TT > d on
        int gw = d < 0 ? 0 : d / TT + 1;
        if (gw < neg) gw = neg;
        if (gw < full) tiles -= floor_sum(full - gw, BK, TT, gw * TT - d);
    }
    int64_t u = tiles + (int64_t)item_head(false) * full;
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
    int req, alt, whole, slot, c0, c1, half;  // half of Q's buffer (alt)
};
static_assert(sizeof(Seg) == 64, "segment size");

// The line's items from the block's start on.
struct Walk {
    int64_t pos, end, per, A;
    int vb;                  // number of the part: its lead and slots
    int req, h, g, alts;
    TileReq q;
    bool fresh;
    __device__ bool next(const PagedAttn &a, int th, int64_t P0, Seg &s) {
      while (true) {
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
        const int head = item_head(s.alt);
        const int b = max(0, (int)(pos - A) - head), e = min(max(0, (int)(stop - A) - head), t1 - t0);
        const bool some = stop - A > head;
        s.t0 = t0 + b;
        s.nt = max(0, e - b);
        s.tok = q.r.tok0 + j0;
        s.ntok = j1 - j0 + 1;
        s.h = h;
        s.pos = q.r.pos0 + j0;
        s.req = req;
        s.whole = b == 0 && stop == B;
        s.slot = 2 * vb + (pos == P0 ? 0 : 1);
        s.c0 = A + head >= P0 ? vb : -1;  // part with the item's first tile: this one, or one before
        s.c1 = vb;                        // part with its last
        if (B > end) s.c1 = (int)((B - 1) / per);
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
        if (!some) continue;
        s.half = 0;
        if (s.alt && s.nt > 0) s.half = alts++ & 1;
        return true;
      }
    }
};

// Sets the walk to P0, in request `req` of `units` units that `before` precede; a whole
// warp.
__device__ __forceinline__ void walk_from(const PagedAttn &a, Walk &w, int th, int64_t P0, int req, int64_t before, int64_t units) {
    const int lane = threadIdx.x & 31;
    const TileReq q = tile_req(a, req, th, nullptr);
    const int64_t head = units / a.Hkv;
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
    w.A = before + h * head + units_before(a, q, lo, th);
    w.req = req;
    w.h = h;
    w.g = lo;
    w.fresh = true;
    w.pos = P0;
}
// The same with the request to be found yet.
__device__ __forceinline__ void walk_to(const PagedAttn &a, Walk &w, int th, int64_t P0) {
    const int lane = threadIdx.x & 31;
    int64_t carry = 0;
    for (int base = 0; base < a.n_seqs; base += 32) {
        const int64_t t = base + lane < a.n_seqs ? line_units(a, base + lane, th, nullptr) : 0;
        const int64_t inc = paged_warp_scan(t, lane);
        const uint32_t at = __ballot_sync(0xffffffffu, P0 >= carry + inc - t && P0 < carry + inc);
        if (at) {
            const int k = __ffs(at) - 1;
            const int64_t before = carry + __shfl_sync(0xffffffffu, inc - t, k), units = __shfl_sync(0xffffffffu, t, k);
            walk_from(a, w, th, P0, base + k, before, units);
            return;
        }
        carry += __shfl_sync(0xffffffffu, inc, 31);
    }
}

// The products are issued by a whole converged warp, one elected lane of which
// does it, in batches of straight code: the issuing warp is on the path of every
// tile (with a descriptor built and a lane elected for each product it took some
// 2,200 cycles a tile and half, more than the products themselves).
//
// S = Q K^T for 64 keys: eight steps of 16 channels; q, k are the descriptors of the
// first step, each step 32 bytes on, the second 64 channels one block on.
__device__ __forceinline__ void issue_qk(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc) {
    asm volatile(
        "{\n .reg .pred e, t, f;\n .reg .b64 a, b;\n"
        " setp.eq.u32 t, 0, 0;\n setp.ne.u32 f, 0, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n"
        " add.s64 a, %1, 2;\n add.s64 b, %2, 2;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        " add.s64 a, %1, 4;\n add.s64 b, %2, 4;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        " add.s64 a, %1, 6;\n add.s64 b, %2, 6;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        " add.s64 a, %1, 1024;\n add.s64 b, %2, 1024;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        " add.s64 a, %1, 1026;\n add.s64 b, %2, 1026;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        " add.s64 a, %1, 1028;\n add.s64 b, %2, 1028;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        " add.s64 a, %1, 1030;\n add.s64 b, %2, 1030;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
        "}\n" ::"r"(d),
        "l"(q), "l"(k), "r"(idesc)
        : "memory");
}
// O (+)= P V for 64 keys: four steps of 16 keys, V 2 KB on; P stands in the first 16 of
// each 32 columns of S.
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t p, uint64_t v, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred e, t, f;\n .reg .b32 a;\n .reg .b64 b;\n"
        " setp.eq.u32 t, 0, 0;\n setp.ne.u32 f, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n"
        " add.u32 a, %1, 8;\n add.s64 b, %2, 128;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
        " add.u32 a, %1, 32;\n add.s64 b, %2, 256;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
        " add.u32 a, %1, 40;\n add.s64 b, %2, 384;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
        "}\n" ::"r"(d),
        "r"(p), "l"(v), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
struct Shared {
    uint32_t tmem;
    int abort;
};

// One warp walks the line ahead of the others, and has each segment's queries
// loaded; a segment with nt < 0 ends it.  Items of one half take the two halves of
// the buffer in turn, so the next one's queries arrive while this one is worked on.
template <class Gate>
__device__ __forceinline__ void walk_role(const PagedAttn &a, const CUtensorMap &qmap, uint8_t *sm, Walk w, int th, int64_t P0,
                                          int64_t total, const Gate &gate) {
    const int lane = threadIdx.x & 31;
    const Bars bar(sm);
    int n0 = 0, n1 = 0;  // loads of each half of Q
    auto landed = [&]() {  // the block ends only when its copies have
        if (n0) mbar_wait(&bar.q_full[0], (n0 - 1) & 1);
        if (n1) mbar_wait(&bar.q_full[1], (n1 - 1) & 1);
        __syncwarp();
    };
    for (int i = 0;; ++i) {
        Seg s;
        bool more = w.next(a, th, P0, s);
        while (!more) {  // the block's next part, if there is one
            P0 += gridDim.x * w.per;
            if (P0 >= total) break;
            w.vb += gridDim.x;
            w.end = P0 + w.per < total ? P0 + w.per : total;
            walk_to(a, w, th, P0);
            more = w.next(a, th, P0, s);
        }
        if (!more) s.nt = -1;
        bool ok = gate(&bar.seg_empty[i % SEGS], ((i / SEGS) & 1) ^ 1);
        if (ok && lane == 0) {
            *reinterpret_cast<Seg *>(sm + OFF_SEG + (i % SEGS) * 64) = s;
            mbar_arrive(&bar.seg_full[i % SEGS]);
        }
        __syncwarp();
        if (ok && !more) return landed();
        for (int x = 0; ok && s.nt > 0 && x < 2; ++x) {
            if (s.alt && x != s.half) continue;
            ok = gate(&bar.q_empty[x], ((x ? n1 : n0) & 1) ^ 1);
            if (ok && lane == 0) {
                mbar_expect_tx(&bar.q_full[x], (uint32_t)(2 * th * a.G * 128));
                uint8_t *dst = sm + OFF_Q + x * QHALF;
                const int tok = s.tok + (s.alt ? 0 : x * th);
                tma_load_3d(dst, &qmap, 0, s.h * a.G, tok, &bar.q_full[x]);
                tma_load_3d(dst + QHALF / 2, &qmap, 64, s.h * a.G, tok, &bar.q_full[x]);
            }
            __syncwarp();
            if (!ok) break;
            if (x) ++n1;
            else ++n0;
        }
        if (!ok) return landed();
    }
}
// The next segment, for a whole warp; false at the line's end.
template <class Gate>
__device__ __forceinline__ bool next_seg(uint8_t *sm, const Bars &bar, int &i, const Gate &gate, Seg &s) {
    if (!gate(&bar.seg_full[i % SEGS], (i / SEGS) & 1)) return false;
    s = *reinterpret_cast<const Seg *>(sm + OFF_SEG + (i % SEGS) * 64);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bar.seg_empty[i % SEGS]);
    ++i;
    return s.nt >= 0;
}

// ---------------------------------------------------------------- loads
// Keys and values.
template <class Gate>
__device__ __forceinline__ void load_role(const PagedAttn &a, const PagedMaps &maps, uint8_t *sm, const Gate &gate) {
    const int lane = threadIdx.x & 31;
    const Bars bar(sm);
    const int box = a.box, lg = a.box_log, nbx = BK >> lg;
    int ring = 0, ringp = 0;
    uint32_t seq = 0;  // K / V tiles so far
    // the block ends only when its copies have landed, also where a wait of another role runs out
    // after this one has issued its last
    auto drain = [&]() {
        for (uint32_t i = 1; i <= SLOTS && i <= seq; ++i) mbar_wait(&bar.kv_full[(seq - i) % SLOTS], ((seq - i) / SLOTS) & 1);
        __syncwarp();
    };
    Seg s;
    int iseg = 0;
    while (next_seg(sm, bar, iseg, gate, s)) {
        if (s.nt == 0) continue;
        int cbase = -64, page = 0, off = 0;
        const int lob = s.lo & ~(box - 1);  // boxes before this one hold no seen key (their pages may be gone)
        // one K or V tile
        auto tile = [&](int j, bool v) -> bool {
            const int key0 = (s.t0 + j) * BK, b0 = key0 >> lg;
            if (cbase < 0 || b0 < cbase || b0 + nbx > cbase + 32) {  // pages of the next 32 boxes, one per lane
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
            const int slot = ring;
            if (!gate(&bar.kv_empty[slot], ringp ^ 1)) return false;
            const int f = max(0, (lob - key0) >> lg), e = min(nbx, (s.hi - key0 + box - 1) >> lg);
            if (lane == 0) mbar_expect_tx(&bar.kv_full[slot], (uint32_t)((e - f) << lg) * (D * 2));
            __syncwarp();
            const int pg = __shfl_sync(0xffffffffu, page, (b0 - cbase + lane) & 31);
            const int y = __shfl_sync(0xffffffffu, off, (b0 - cbase + lane) & 31);
            if (lane >= f && lane < e) {
                uint8_t *dst = sm + OFF_KV + slot * SLOT + (lane << lg) * 128;
                const CUtensorMap *m = v ? &maps.v : &maps.k;
                tma_load_3d(dst, m, 0, y, pg, &bar.kv_full[slot]);
                tma_load_3d(dst + SLOT / 2, m, 64, y, pg, &bar.kv_full[slot]);
            }
            __syncwarp();
            ++seq;
            if (++ring == SLOTS) {
                ring = 0;
                ringp ^= 1;
            }
            return true;
        };
        for (int j = 0; j < s.nt; ++j) {
            if (!tile(j, false) || !tile(j, true)) return drain();
        }
    }
    drain();
}

// ---------------------------------------------------------------- products
// One warp for each group's products (an item of one half is the first warp's
// alone): what one of them spends on waits and on issuing hides behind the other's
// products.  Both see every K, V and Q tile, so that no barrier's phase passes one
// of them by: whoever has no product on a tile gives it back as soon as it came.
template <class Gate>
__device__ __forceinline__ void mma_role(uint8_t *sm, uint32_t tmem, int x, const Gate &gate) {
    const Bars bar(sm);
    constexpr uint32_t ID_QK = idesc_bf16_f32(BM, BK / 2), ID_PV = idesc_bf16_f32_bmn(BM, D);
    const int lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(sm), to = tmem + COL_O + x * 128;
    const uint64_t dq = sdesc_sw128(base + OFF_Q), dk = sdesc_sw128(base + OFF_KV),
                   dv = sdesc_mn(base + OFF_KV, SLOT / 2, 1024, SWZ_128B);
    // tiles are first used in the order in which they are loaded
    int ring = 0, ringp = 0;
    auto take = [&](int &slot) -> bool {
        slot = ring;
        const bool ok = gate(&bar.kv_full[ring], ringp);
        if (++ring == SLOTS) {
            ring = 0;
            ringp ^= 1;
        }
        return ok;
    };
    auto give = [&](uint64_t *b) {
        if (lane == 0) mbar_arrive(b);
        __syncwarp();
    };
    uint32_t par = 0;  // parity bits: 0, 1 halves of Q; 2, 3 P by half of the tile; 5 O
    bool ok = true;
    Seg s;
    int iseg = 0;
    while (ok && next_seg(sm, bar, iseg, gate, s)) {
        if (s.nt == 0) continue;
        const bool alt = s.alt;
        const int nt = s.nt, half = alt ? s.half : x;
        auto query = [&](int h) -> bool {
            const bool got = gate(&bar.q_full[h], (par >> h) & 1);
            par ^= 1u << h;
            return got;
        };
        if (alt && x) {  // the other warp's item
            ok = query(half);
            give(&bar.q_empty[half]);
            for (int i = 0; ok && i < 2 * nt; ++i) {
                int slot;
                ok = take(slot);
                give(&bar.kv_empty[slot]);
            }
            continue;
        }
        int kslot = 0, vslot = 0;
        ok = query(half);
        if (!alt) {  // the other half's queries
            ok = query(half ^ 1) && ok;
            give(&bar.q_empty[half ^ 1]);
        }
        const uint64_t q = dq + (uint32_t)half * (QHALF >> 4);
        // S of half a tile's keys
        const uint32_t sb = tmem + COL_S + x * 128;
        auto qk = [&](int u) {
            issue_qk(sb + u * 64, q, dk + (uint32_t)(kslot * (SLOT >> 4) + u * HALF_K), ID_QK);
            mma_commit_w(&bar.s_full[2 * x + u]);  // (first: it is waited for; a commit covers all before it)
        };
        auto k_done = [&](int j) {
            mma_commit_w(&bar.kv_empty[kslot]);
            if (j == nt - 1) mma_commit_w(&bar.q_empty[half]);
        };
        ok = take(kslot) && ok;
        tc_fence_after();
        if (ok) {
            qk(0);
            qk(1);
            k_done(0);
        }
        for (int j = 0; ok && j < nt; ++j) {
            ok = take(vslot);
            if (j == 0) {  // the group's last item must have left O
                ok = gate(&bar.o_free[x], ((par >> 5) & 1) ^ 1) && ok;
                par ^= 1u << 5;
            }
            // P V of each half, and after it S of the next tile's half over the same columns
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                ok = gate(&bar.p_ready[2 * x + u], (par >> (2 + u)) & 1) && ok;
                par ^= 1u << (2 + u);
                if (!ok) break;
                tc_fence_after();
                issue_pv(to, sb + u * 64, dv + (uint32_t)(vslot * (SLOT >> 4) + u * HALF_K), ID_PV, j + u > 0);
                mma_commit_w(&bar.pv_done[2 * x + u]);
                if (u) mma_commit_w(&bar.kv_empty[vslot]);
                if (j + 1 < nt) {
                    if (u == 0) {
                        ok = take(kslot);
                        tc_fence_after();
                        if (!ok) break;
                    }
                    qk(u);
                    if (u) k_done(j + 1);
                }
            }
        }
    }
    // TMEM is given back only after the products, whichever wait ran out or none
    mma_commit_w(bar.last + x);
    mbar_wait(bar.last + x, 0);
    __syncwarp();
}

// ---------------------------------------------------------------- softmax
// 32 channels of one row, 32 bytes at a time: a row is one thread's, so narrower
// stores would each touch 32 lines for less
__device__ __forceinline__ void store_bf16(const PagedAttn &a, int64_t row, int c, const float (&o)[32]) {
    char *dst = (char *)a.o + (row * D + c) * 2;
    if ((uintptr_t)a.o & 31u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(o[8 * i + 2 * k], o[8 * i + 2 * k + 1]);
                u[k] = *reinterpret_cast<const uint32_t *>(&b);
            }
            reinterpret_cast<uint4 *>(dst)[i] = make_uint4(u[0], u[1], u[2], u[3]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(o[16 * i + 2 * k], o[16 * i + 2 * k + 1]);
            u[k] = *reinterpret_cast<const uint32_t *>(&b);
        }
        store32(dst + 32 * i, u);
    }
}
__device__ __forceinline__ void store_f32(float *dst, const float (&o)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(o[8 * i + k]);
        store32(dst + 8 * i, u);
    }
}

// The segment's end of one group: half of O's channels, normalised or as a piece.
__device__ __forceinline__ void finish(const PagedAttn &a, uint32_t to, int th, const volatile Seg *s, int x, int hf, int row,
                                       float ref, float l) {
    const int G = a.G, half = s->alt ? 0 : x, nt = s->nt;
    const int jt = row / G, local = half * th * G + row;  // token within the half, row of the item
    const bool live = row < min(th, s->ntok - half * th) * G, whole = s->whole;
    const int64_t out = (int64_t)(s->tok + half * th + jt) * a.Hq + s->h * G + (row - jt * G);
    float *slot = paged_slot(a, s->slot);
    const bool dead = nt == 0 || l == 0.f;  // (NaN passes through)
    const float f = whole ? 1.f / l : 1.f;
#pragma unroll 1
    for (int c = 64 * hf; c < 64 * hf + 64; c += 32) {
        float o[32];
        tmem_ld32(to + c, o);
        tmem_arrived(o);
        if (live) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = dead ? 0.f : o[i] * f;
            if (whole)
                store_bf16(a, out, c, o);
            else
                store_f32(slot + 2 * a.slot_rows + (size_t)local * D + c, o);
        }
    }
    if (live && hf == 0) {
        if (!whole)
            reinterpret_cast<float2 *>(slot)[local] = make_float2(dead ? -INFINITY : ref, dead ? 0.f : l);
        else if (a.lse)
            a.lse[out] = dead ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
    }
    if (threadIdx.x == 0 && !whole && s->c0 >= 0) {  // the item's first piece is here
        a.lead[2 * s->c0] = make_int4(s->tok, s->h, 0, s->ntok * G);
        a.lead[2 * s->c0 + 1] = make_int4(s->slot, s->c0, s->c1, 1);
    }
}

// Two threads, of two warps that meet at a barrier of their own, share a row.  A
// wait that runs out is passed on at the next meeting, so both leave together.
template <class Gate>
__device__ __forceinline__ void softmax_role(const PagedAttn &a, uint8_t *sm, uint32_t tmem, int th, const Gate &gate) {
    constexpr int HK = BK / 4;  // keys of one thread: a half of half a tile
    const Bars bar(sm);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, x = warp >> 3, hf = (warp >> 2) & 1;
    const int row = (warp & 3) * 32 + lane;             // row of the half = TMEM lane
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // 32 (warp % 4) << 16
    const uint32_t to = tmem + lanes + COL_O + x * 128;
    const int id = 1 + x * 4 + (warp & 3);
    float *mx = reinterpret_cast<float *>(sm + OFF_MX) + x * 2 * BM + row;  // + BM hf
    const float sc = a.scale_log2;
    int n = 0;       // this group's tiles before this segment's
    uint32_t seq0 = 0;  // K / V tiles before this segment's
    bool failed = false;
    for (int iseg = 0;; ++iseg) {
        if (!gate(&bar.seg_full[iseg % SEGS], (iseg / SEGS) & 1)) {
            meet_count<64>(id, true);
            return;
        }
        const Seg *seg = reinterpret_cast<const Seg *>(sm + OFF_SEG + (iseg % SEGS) * 64);
        struct {
            int lo, hi, t0, nt;
        } s{seg->lo, seg->hi, seg->t0, seg->nt};
        if (s.nt < 0) {
            meet_count<64>(id, false);
            return;
        }
        const bool alt = seg->alt;
        const int pos = seg->pos + (alt ? 0 : x) * th + row / a.G;
        const int first_key = first_seen(a, pos);  // keys first_key .. pos, all below hi
        float ref = 0.f, l = 0.f, top = -INFINITY;  // (top: of all the row's keys at the last change of ref, then of this half's)
        // ref follows the maximum once that has passed this (never for the half's rows past the
        // item's tokens: they hold the next request's queries, or what was there before)
        float bound = row < min(th, seg->ntok - (alt ? 0 : x) * th) * a.G ? -INFINITY : INFINITY;
        const int ne = alt && x ? 0 : 2 * s.nt;  // halves of tiles
        uint64_t *prev = nullptr;  // the group's last product
        int prevp = 0;
        for (int e = 0; e < ne; ++e) {
            const int j = e >> 1, u = e & 1, b = 2 * x + u, ph = (n + j) & 1;
            const uint32_t ts = tmem + lanes + COL_S + x * 128 + u * 64 + HK * hf;  // this thread's scores, and P
            const int key0 = (s.t0 + j) * BK + u * (BK / 2);
            if (!gate(&bar.s_full[b], ph)) failed = true;
            tc_fence_after();
            float v[HK];
            tmem_ld32(ts, v);
            tmem_arrived(v);
            // of this thread's keys, the row sees [c0, c1)
            const int c1 = min(pos + 1, s.hi) - key0 - HK * hf, c0 = first_key - key0 - HK * hf;
            if (__any_sync(0xffffffffu, c1 < HK || c0 > 0)) {
#pragma unroll
                for (int c = 0; c < HK; ++c) v[c] = c < c1 && c >= c0 ? v[c] : -INFINITY;
            }
            float m0 = max3(v[0], v[1], v[2]), m1 = max3(v[3], v[4], v[5]), m2 = max3(v[6], v[7], v[8]), m3 = max3(v[9], v[10], v[11]);
#pragma unroll
            for (int c = 12; c + 8 <= HK; c += 8) {
                m0 = max3(m0, v[c], v[c + 1]);
                m1 = max3(m1, v[c + 2], v[c + 3]);
                m2 = max3(m2, v[c + 4], v[c + 5]);
                m3 = max3(m3, v[c + 6], v[c + 7]);
            }
            m0 = max3(m0, v[HK - 4], v[HK - 3]);
            m1 = max3(m1, v[HK - 2], v[HK - 1]);
            const float mt = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * sc;
            // Meet: does ref have to follow?  (a warp that gave up counts 32, one that asks
            // for it 1)
            const bool grow = __any_sync(0xffffffffu, mt > bound);
            const int said = meet_count<64>(id, failed || (grow && lane == 0));
            if (said >= 32) return;
            if (said) {
                mx[BM * hf] = mt;
                meet_count<64>(id, false);
                const float both = fmaxf(fmaxf(mt, mx[BM * (1 - hf)]), top);
                const float nref = both == -INFINITY ? 0.f : top == -INFINITY ? both : fmaxf(both, ref);
                const float corr = top == -INFINITY ? 0.f : ex2(ref - nref);  // (nothing summed yet: what O holds is zero)
                top = both;
                ref = nref;
                l *= corr;
                if (bound != INFINITY && both != -INFINITY) bound = nref + GROW;
                if (prev) {  // the group's last product must have left O
                    if (!gate(prev, prevp)) failed = true;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 64 * hf; c < 64 * hf + 64; c += 16) {
                        float o[16];
                        tmem_ld16(to + c, o);
                        tmem_ld_wait();
                        uint32_t u[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            asm volatile("" : "+f"(o[i]));
                            u[i] = __float_as_uint(o[i] * corr);
                        }
                        tmem_st16(to + c, u);
                    }
                }
            }
            // rows of V that no key seen by this item stands in may hold anything: zero
            // them (0 x NaN is NaN); each group before its own product
            const int z0 = max(0, s.lo - key0), z1 = min(BK, s.hi - key0);
            if (u == 0 && (z0 > 0 || z1 < BK)) {
                const uint32_t q = seq0 + 2 * j + 1;
                if (!gate(&bar.kv_full[q % SLOTS], (int)((q / SLOTS) & 1))) failed = true;
                uint8_t *vt = sm + OFF_KV + (q % SLOTS) * SLOT;
                for (int w = threadIdx.x & (2 * BM - 1); w < BK * 16; w += 2 * BM) {
                    const int r = w >> 4, c = w & 15;
                    if (r < z0 || r >= z1)
                        *reinterpret_cast<uint4 *>(vt + (c >> 3) * (SLOT / 2) + r * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
            }
            // probabilities, over the scores that they come from
            const uint64_t sc2 = pack2(sc, sc), ref2 = pack2(-ref, -ref);
            uint64_t sum2 = 0;
            uint32_t p[HK / 2];
#pragma unroll
            for (int i = 0; i < HK / 2; ++i) {
                float e0, e1;
                unpack2(fma2(pack2(v[2 * i], v[2 * i + 1]), sc2, ref2), e0, e1);
                e0 = ex2(e0);
                e1 = ex2(e1);
                sum2 = add2(sum2, pack2(e0, e1));
                const __nv_bfloat162 w = __floats2bfloat162_rn(e0, e1);
                p[i] = *reinterpret_cast<const uint32_t *>(&w);
            }
            tmem_st16(ts, p);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.p_ready[b]);
            float l0, l1;
            unpack2(sum2, l0, l1);
            l += l0 + l1;
            prev = &bar.pv_done[b];
            prevp = ph;
        }
        seq0 += 2 * s.nt;
        if (!alt || x == 0) n += s.nt;
        if (!(alt && x)) {
            float sum = 0.f;
            if (prev) {
                if (!gate(prev, prevp)) failed = true;
                tc_fence_after();
                mx[BM * hf] = l;  // (both are past the maxima that stood there: P V has been)
                if (meet_count<64>(id, failed) >= 32) return;
                sum = mx[0] + mx[BM];
            }
            finish(a, to, th, seg, x, hf, row, ref, sum);
            tc_fence_before();
            __syncwarp();
            if (prev && lane == 0) mbar_arrive(&bar.o_free[x]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.seg_empty[iseg % SEGS]);
    }
}

template <bool SHORT>
__global__ void __launch_bounds__(THREADS, 1)
    paged_tile_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ PagedAttn a, int th,
                      int min_per, int max_parts) {
    extern __shared__ __align__(1024) uint8_t sm[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Shared *sh = reinterpret_cast<Shared *>(sm + OFF_MISC);
    int64_t *scratch = reinterpret_cast<int64_t *>(sm + OFF_SCAN);
    const Bars bar(sm);
    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&bar.kv_full[i], 1);
            mbar_init(&bar.kv_empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.q_full[i], 1);
            mbar_init(&bar.q_empty[i], 2);
            mbar_init(&bar.o_free[i], 8);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_ready[i], 8);
            mbar_init(&bar.pv_done[i], 1);
        }
        for (int i = 0; i < SEGS; ++i) {
            mbar_init(&bar.seg_full[i], 1);
            mbar_init(&bar.seg_empty[i], SOFT + 3);
        }
        mbar_init(bar.last, 1);
        mbar_init(bar.last + 1, 1);
        mbar_fence_init();
        sh->abort = 0;
        for (int i = 0; i < max_parts; ++i) a.lead[2 * (blockIdx.x + i * gridDim.x) + 1] = make_int4(0, 0, 0, 0);
    }
    auto units = [&](int i, int *err) { return line_units(a, i, th, err); };
    int64_t kv_tiles = 0;
    if (max_parts > 1) {
        int64_t n = 0;
        for (int i = tid; i < a.n_seqs; i += THREADS) {
            const PagedReq r = paged_req(a, i, nullptr);
            if (r.rows) n += (int64_t)a.Hkv * ((r.kend - r.k0 + BK - 1) / BK);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        if (lane == 0) scratch[warp] = n;
        __syncthreads();
        for (int w = 0; w < THREADS / 32; ++w) kv_tiles += scratch[w];
        __syncthreads();
    }
    // Keys and values over 64 MB are taken in parts, so that those that the blocks read
    // at any time stay in the L2 cache (2,048 tokens over 65,536 keys of 8 heads, 268 MB:
    // read 23 times from HBM otherwise); each part should be worth the pieces that its
    // borders cost.
    auto parts = [&](int64_t total) -> int {
        const int64_t by_size = (kv_tiles * (2 * SLOT) + (64 << 20) - 1) >> 26, by_work = total / (gridDim.x * 128);
        const int64_t n = by_size < by_work ? by_size : by_work;
        return n < 1 ? 1 : n > max_parts ? max_parts : (int)n;
    };
    const PagedLine line = paged_line<THREADS>(a, scratch, min_per, units, parts);
    const int64_t P0 = line.P0, P1 = line.P1;
    if (P0 >= P1) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    if (warp == SOFT) tmem_alloc(&sh->tmem, TCOLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    const Waits<SHORT> gate{&sh->abort, a.err, a.wait_budget};
    if (warp < SOFT) {
        softmax_role(a, sm, tmem, th, gate);
    } else {
        if (warp < SOFT + 2)
            mma_role(sm, tmem, warp - SOFT, gate);
        else if (warp == SOFT + 2)
            load_role(a, maps, sm, gate);
        else {
            Walk w;
            w.end = P1;
            w.per = line.per;
            w.vb = blockIdx.x;
            w.alts = 0;
            walk_from(a, w, th, P0, line.req, line.before, line.units);
            walk_role(a, qmap, sm, w, th, P0, line.total, gate);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == SOFT) {
        tc_fence_after();
        tmem_dealloc(tmem, TCOLS);
    }
    // the join waits for this grid; this grid may run beside the kernel for few rows, so it
    // ends only after that one
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace

int paged_tile_blocks() { return device_sm_count(); }

int launch_paged_tile(PagedAttn a, const void *k, const void *v, int64_t page_stride, int max_parts, bool after_rows, cudaStream_t s) {
    int box = 16;
    while (box < BK && a.page_size % (2 * box) == 0) box *= 2;
    a.box = box;
    a.box_log = __builtin_ctz(box);
    const int th = BM / a.G;
    PagedMaps maps;
    CUtensorMap qmap;
    int rc = make_paged_maps(k, v, KDA_BF16, a.Hkv, a.page_size, a.n_pages, page_stride, box, &maps);
    if (rc) return rc;
    if ((rc = make_paged_q_map(a.q, a.T, a.Hq, a.G, th, &qmap))) return rc;
    const auto kernel = a.wait_budget < SHORT_BUDGET ? paged_tile_kernel<true> : paged_tile_kernel<false>;
    if ((rc = prepare_kernel((const void *)kernel, SMEM, THREADS, nullptr))) return rc;
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, maps, qmap, a, th, 4, max_parts);
    note_launch("paged_tile", s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace kda
