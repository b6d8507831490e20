// kda_paged_rows.cu -- paged attention in fp32.
//
// A block has eight consumer warps (four, where a call has few rows) and one producer warp.  The producer walks the
// block's line of key tiles (16 keys: 8 KB of K and 8 KB of V), looks pages up in
// the block table, and has the tensor memory accelerator fill a ring of four tiles,
// two blocks on an SM: 128 KB in flight.  A consumer warp holds up to 8 rows.  Few
// rows (<= 8): the warps take every eighth tile, each with its own running maximum
// and sum, merged in shared memory at the item's end.  More rows: two, four or eight
// warps take a share each of up to 16, 32 or 64, and the others other tiles.
//
// Products are plain fp32 multiply-adds: tf32 parts would lose digits that the fp32
// path of this library keeps (three products of two parts each left 2.5e-6 where this
// leaves 3.2e-7).  A lane holds half a key's channels for the scores and four channels
// of all keys for the output, so a warp reads each key and value once from shared
// memory whatever its rows are.
//
// Measured: one token of 16 requests, 16 heads of up to 3,000 keys, 5.1 TB/s (42 us), where
// the copies in flight and the start and the join bound it.  Many rows are bound by loads
// from shared memory and the shuffles between the products (8 requests of 40 rows over 2,040
// keys of 8 heads: 16 TFLOP/s, 162 us, and of 320 rows 27 TFLOP/s, 800 us; four warps of 16
// rows 246 and 1,358 us).
#include "kda_paged.cuh"

namespace kda {
namespace {
using namespace tc;

constexpr int RW = 8;                        // rows a warp holds at most
constexpr int STAGES = 4;
constexpr int HALF = 8192;                   // bytes of K (and of V) of one tile
constexpr int STAGE = 2 * HALF;
// CONS: consumer warps, eight, or four in calls of up to 8 rows (45 us instead of 48 then for
// one token of 16 requests: fewer pieces to merge, fewer warps to give a tile back)
template <int CONS_, bool SHORT_> struct Cfg {
    static constexpr bool SHORT = SHORT_;
    static constexpr int CONS = CONS_, THREADS = (CONS + 1) * 32;
    static constexpr int OFF_RED = STAGES * STAGE;                 // [CONS][RW][128] fp32
    static constexpr int OFF_P = OFF_RED + CONS * RW * D * 4;      // probabilities [CONS][RW][16]
    static constexpr int OFF_ML = OFF_P + CONS * RW * 16 * 4;
    static constexpr int OFF_DESC = OFF_ML + CONS * RW * 8;
    static constexpr int OFF_BAR = OFF_DESC + STAGES * 64;
    static constexpr int OFF_MEET = OFF_BAR + 2 * STAGES * 8;      // the consumer warps' meeting at an item's end
    static constexpr int OFF_ABORT = OFF_MEET + 8;
    static constexpr int SMEM = OFF_ABORT + 16;
    static_assert(OFF_RED % 1024 == 0 && OFF_ML % 16 == 0 && OFF_DESC % 16 == 0 && OFF_BAR % 8 == 0, "shared memory layout");
};

constexpr int TK = 16;                       // keys of a tile
// What an item costs besides its tiles (queries in, pieces merged, output), in tiles: short
// items are spread over the blocks by it (4 requests of up to 40 tokens over up to 66 keys,
// 64 heads: 28 us, without it 98; 3, 4 and 6 are within 3% on long ones).
constexpr int HEAD = 6;
constexpr int NSUB = D * 4 / 128;            // 128-byte pieces of a row, each a block of its own

// what the producer says about a tile
struct __align__(16) Desc {
    int flags, ord, wr, key0, kvalid, tok0, h, r0, R, pos0, slot, c0, c1, rpw;  // rpw: rows of a warp
    int kfirst, pad;         // the tile's rows [kfirst, kvalid) hold keys that the item sees
};
static_assert(sizeof(Desc) == 64, "descriptor size");
constexpr int FIRST = 1, LAST = 2, WHOLE = 4, END = 8, MASK = 16;

template <class C> __device__ __forceinline__ int row_group(int rows) {
    return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 || C::CONS == 4 ? 32 : 64;
}

__device__ __forceinline__ int req_tiles(const PagedReq &r) {
    const int keys = r.kend - r.k0;
    return keys > 0 ? (keys + TK - 1) / TK : 1;
}
template <class C> __device__ __forceinline__ int64_t line_tiles(const PagedAttn &a, int i, int *err) {
    const PagedReq r = paged_req(a, i, err);
    if (r.rows == 0) return 0;
    const int grp = row_group<C>(r.rows);
    return (int64_t)a.Hkv * ((r.rows + grp - 1) / grp) * (HEAD + req_tiles(r));
}

// A bounded wait of a whole warp that also gives up once *abort is set.  SHORT: as for the
// tensor-core kernels, the launch's budget, and no try that sleeps.
template <class C>
__device__ __forceinline__ bool wait_for(const PagedAttn &a, uint64_t *bar, uint32_t parity, const volatile int *abort) {
    bool ok;
    if constexpr (C::SHORT) {
        const long long t0 = clock64();
        while (!(ok = mbar_test_wait(bar, parity)) && !*abort && clock64() - t0 <= a.wait_budget) {
        }
    } else {
        ok = mbar_wait_ab(bar, parity, abort);
    }
    return __all_sync(0xffffffffu, ok);
}

// ---------------------------------------------------------------- producer
// One tile (16 keys of one head of one page) in one copy: the map's third dimension is
// the row's four 128-byte pieces, which land in blocks of their own.
__device__ __forceinline__ void load_tile(void *dst, const void *map, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(0), "r"(y), "r"(0), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
template <class C>
__device__ __forceinline__ void produce(const PagedAttn &a, const PagedMaps &maps, uint8_t *sm, int64_t P0, int64_t P1,
                                        int64_t per, int req, int64_t before) {
    const int lane = threadIdx.x & 31;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR), *empty = full + STAGES;
    volatile int *abort = reinterpret_cast<volatile int *>(sm + C::OFF_ABORT);
    int stage = 0, phase = 0, issued = 0;
    // the block ends only when its copies have landed, also where a wait of the consumers runs
    // out after the last was issued
    auto drain = [&]() {
        for (int i = 1; i <= STAGES && i <= issued; ++i) {
            const int u = issued - i;
            mbar_wait(&full[u % STAGES], (u / STAGES) & 1);
        }
        __syncwarp();
    };
    auto next_stage = [&]() -> bool {
        if (!wait_for<C>(a, &empty[stage], phase ^ 1, abort)) {
            if (lane == 0) {
                *abort = 1;
                if (a.err) atomicOr(a.err, KDA_DEVERR_TIMEOUT);
            }
            __syncwarp();
            drain();
            return false;
        }
        ++issued;
        return true;
    };
    auto advance = [&]() {
        if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
        }
    };

    int64_t pos = P0;
    while (pos < P1) {
        const PagedReq r = paged_req(a, req, nullptr);
        if (r.rows == 0) {
            ++req;  // (the totals say that a request with tiles follows)
            continue;
        }
        const int nt = req_tiles(r), grp = row_group<C>(r.rows), ngrp = (r.rows + grp - 1) / grp;
        const int64_t in = pos - before, item = in / (HEAD + nt);
        const int h = (int)(item / ngrp), g = (int)(item - (int64_t)h * ngrp);
        const int64_t A = before + item * (HEAD + nt), B = A + HEAD + nt;
        const int64_t seg_end = B < P1 ? B : P1;
        const int t_begin = max(0, (int)(pos - A) - HEAD), t_end = (int)(seg_end - A) - HEAD;
        if (t_end <= 0) break;  // a cut before the first tile leaves the item to the next block
        const int r0 = g * grp, R = min(grp, r.rows - r0);
        const int posf = r.pos0 + r0 / a.G, posl = r.pos0 + (r0 + R - 1) / a.G;
        const int lo = first_seen(a, posf), hi = posl + 1;  // keys that the group sees
        int tb = t_begin, te = t_end;
        if (hi <= lo) {
            te = tb;
        } else {
            tb = max(tb, (lo - r.k0) / TK);
            te = min(te, (hi - r.k0 + TK - 1) / TK);
        }
        Desc d;
        d.wr = grp / RW;
        d.rpw = (R + d.wr - 1) / d.wr;  // (the same for each, or one waits for the others)
        d.tok0 = r.tok0;
        d.h = h;
        d.r0 = r0;
        d.R = R;
        d.pos0 = r.pos0;
        d.c0 = (int)((A + HEAD) / per);
        d.c1 = (int)((B - 1) / per);
        d.slot = 2 * (int)blockIdx.x + (pos == P0 ? 0 : 1);
        const int whole = t_begin == 0 && seg_end == B ? WHOLE : 0;
        if (te <= tb) {  // nothing to read: one empty tile so that the segment is finished all the same
            if (!next_stage()) return;
            if (lane == 0) {
                d.flags = FIRST | LAST | MASK | whole;
                d.ord = 0;
                d.key0 = 0;
                d.kvalid = d.kfirst = 0;
                *reinterpret_cast<Desc *>(sm + C::OFF_DESC + stage * 64) = d;
                mbar_arrive(&full[stage]);
            }
            advance();
        }
        int cbase = 0, page = 0, off = 0;
        for (int t = tb; t < te; ++t) {
            if (t == tb || t >= cbase + 32) {  // pages of the next 32 tiles, one per lane
                cbase = t;
                const int key = r.k0 + (cbase + lane) * TK, blk = key / a.page_size;
                page = 0;
                off = h * a.page_size + key - blk * a.page_size;
                if (key < hi) {
                    page = a.table[(int64_t)req * a.max_blocks + blk];
                    if (page < 0 || page >= a.n_pages) {
                        if (a.err) atomicOr(a.err, KDA_DEVERR_PAGE);
                        page = 0;
                    }
                }
            }
            const int key0 = r.k0 + t * TK, kvalid = min(TK, hi - key0);
            const int pg = __shfl_sync(0xffffffffu, page, t - cbase), y = __shfl_sync(0xffffffffu, off, t - cbase);
            if (!next_stage()) return;
            if (lane == 0) {
                d.flags = (t == tb ? FIRST : 0) | (t == te - 1 ? LAST : 0) | whole;
                if (kvalid < TK || key0 + TK - 1 > posf || (a.window > 0 && key0 <= posl - a.window)) d.flags |= MASK;
                d.ord = t - tb;
                d.key0 = key0;
                d.kvalid = kvalid;
                d.kfirst = max(0, lo - key0);
                *reinterpret_cast<Desc *>(sm + C::OFF_DESC + stage * 64) = d;
                mbar_expect_tx(&full[stage], 2 * HALF);
                load_tile(sm + stage * STAGE, &maps.k, y, pg, &full[stage]);
                load_tile(sm + stage * STAGE + HALF, &maps.v, y, pg, &full[stage]);
            }
            __syncwarp();
            advance();
        }
        pos = seg_end;
        if (seg_end == B && h == a.Hkv - 1 && g == ngrp - 1) {
            before = B;
            ++req;
        }
    }
    if (!next_stage()) return;
    if (lane == 0) {
        reinterpret_cast<Desc *>(sm + C::OFF_DESC + stage * 64)->flags = END;
        mbar_arrive(&full[stage]);
    }
    __syncwarp();
    drain();
}

// ---------------------------------------------------------------- a warp's rows
// fp32: lane = (key lane % 16, half of the channels lane / 16) for the scores, four
// channels for the output; maxima and sums of row r in lane r.
struct RowsF32 {
    float o[RW][4], m, l;
    // RM: rows that the code is laid out for (R <= RM)
    template <int RM>
    __device__ __forceinline__ void tile(const float *q, float *ps, const uint8_t *k, const uint8_t *v, int lane, int R, float sc,
                                         const Desc &d, int row0, int G, int window, bool mask) {
        const int key = lane & 15, hf = lane >> 4;
        // All rows at once, so that a chain of sums or shuffles does not wait for itself, and
        // half of the lane's channels at a time, which the registers hold (rows past R hold an
        // earlier item's queries; nothing of theirs is read).
        float2 acc[RM];
        float s[RM], top[RM];
#pragma unroll
        for (int r = 0; r < RM; ++r) acc[r] = make_float2(0.f, 0.f);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            float4 kr[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
                kr[c] = *reinterpret_cast<const float4 *>(k + (2 * hf + part) * 2048 + key * 128 + ((c ^ (key & 7)) << 4));
            const float4 *qr = reinterpret_cast<const float4 *>(q) + 16 * hf + 8 * part;
#pragma unroll
            for (int r = 0; r < RM; ++r) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float4 x = qr[r * (D / 4) + c];
                    acc[r].x = fmaf(x.x, kr[c].x, acc[r].x);
                    acc[r].y = fmaf(x.y, kr[c].y, acc[r].y);
                    acc[r].x = fmaf(x.z, kr[c].z, acc[r].x);
                    acc[r].y = fmaf(x.w, kr[c].w, acc[r].y);
                }
            }
        }
        float corr = 1.f;  // of row `lane`
#pragma unroll
        for (int r = 0; r < RM; ++r) {
            s[r] = acc[r].x + acc[r].y;
            s[r] += __shfl_xor_sync(0xffffffffu, s[r], 16);
        }
        if (mask) {
#pragma unroll
            for (int r = 0; r < RM; ++r) {
                const int pos = d.pos0 + (row0 + r) / G, at = d.key0 + key;
                if (!(at <= pos && (window <= 0 || at > pos - window) && key < d.kvalid)) s[r] = -INFINITY;
            }
        }
#pragma unroll
        for (int r = 0; r < RM; ++r) top[r] = s[r];
#pragma unroll
        for (int x = 8; x; x >>= 1)
#pragma unroll
            for (int r = 0; r < RM; ++r) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], x));
#pragma unroll
        for (int r = 0; r < RM; ++r) {
            const float old = __shfl_sync(0xffffffffu, m, r), mn = fmaxf(old, top[r] * sc);
            const float ref = mn == -INFINITY ? 0.f : mn;
            if (lane == r) {
                corr = ex2(m - ref);
                m = mn;
            }
            s[r] = ex2(fmaf(s[r], sc, -ref));
        }
#pragma unroll
        for (int r = 0; r < RM; ++r)
            if (lane < 16) ps[r * 16 + lane] = s[r];
        __syncwarp();
        const bool moved = __any_sync(0xffffffffu, corr != 1.f);
        l *= corr;
#pragma unroll
        for (int r = 0; r < RM; ++r) {
            if (r < R && moved) {
                const float f = __shfl_sync(0xffffffffu, corr, r);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[r][e] *= f;
            }
        }
#pragma unroll
        for (int kk = 0; kk < 16; kk += 4) {
            float4 vv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                vv[e] = *reinterpret_cast<const float4 *>(v + (lane >> 3) * 2048 + (kk + e) * 128 + (((lane & 7) ^ ((kk + e) & 7)) << 4));
#pragma unroll
            for (int r = 0; r < RM; ++r) {
                if (RM == 1 || r < R) {
                    const float4 p = *reinterpret_cast<const float4 *>(ps + r * 16 + kk);
                    o[r][0] = fmaf(p.w, vv[3].x, fmaf(p.z, vv[2].x, fmaf(p.y, vv[1].x, fmaf(p.x, vv[0].x, o[r][0]))));
                    o[r][1] = fmaf(p.w, vv[3].y, fmaf(p.z, vv[2].y, fmaf(p.y, vv[1].y, fmaf(p.x, vv[0].y, o[r][1]))));
                    o[r][2] = fmaf(p.w, vv[3].z, fmaf(p.z, vv[2].z, fmaf(p.y, vv[1].z, fmaf(p.x, vv[0].z, o[r][2]))));
                    o[r][3] = fmaf(p.w, vv[3].w, fmaf(p.z, vv[2].w, fmaf(p.y, vv[1].w, fmaf(p.x, vv[0].w, o[r][3]))));
                    const float sum = (p.x + p.y) + (p.z + p.w);
                    if (lane == r) l += sum;
                }
            }
        }
        __syncwarp();  // (ps is written again at the next tile)
    }
};

// ---------------------------------------------------------------- consumers
// V rows outside the keys that are seen may hold anything (0 x NaN is NaN): zero them.
__device__ __forceinline__ void zero_outside(uint8_t *vt, int kfirst, int kvalid, int lane) {
    for (int x = lane; x < (kfirst + TK - kvalid) * NSUB * 8; x += 32) {
        const int i = x / (NSUB * 8), row = i < kfirst ? i : kvalid + i - kfirst, c = x % (NSUB * 8);
        *reinterpret_cast<uint4 *>(vt + (c >> 3) * TK * 128 + row * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
    }
    fence_async_smem();
    __syncwarp();
}

struct Work {
    RowsF32 w;
    __device__ __forceinline__ void begin(const PagedAttn &a, const Desc &d, int wrow, int lane, float *q) {
        w.m = -INFINITY;
        w.l = 0.f;
        const int R = min(d.rpw, d.R - d.rpw * wrow);
        // the queries stand where the output goes at the end (four loads in flight at once)
#pragma unroll 1
        for (int r0 = 0; r0 < R; r0 += 4) {
            float4 x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int rr = d.r0 + d.rpw * wrow + min(r0 + u, R - 1), j = rr / a.G;
                x[u] = ((const float4 *)a.q + ((int64_t)(d.tok0 + j) * a.Hq + d.h * a.G + (rr - j * a.G)) * (D / 4))[lane];
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) reinterpret_cast<float4 *>(q + (r0 + u) * D)[lane] = x[u];
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) w.o[r][e] = 0.f;
    }
    __device__ __forceinline__ void tile(const PagedAttn &a, const Desc &d, int wrow, int lane, const uint8_t *kt, const uint8_t *vt,
                                         const float *q, float *ps) {
        const int R = min(d.rpw, d.R - d.rpw * wrow), row0 = d.r0 + d.rpw * wrow;
        const bool mask = d.flags & MASK;
        if (R <= 0) return;  // (a last, short row group)
        if (R == 1)
            w.tile<1>(q, ps, kt, vt, lane, R, a.scale_log2, d, row0, a.G, a.window, mask);
        else if (R <= 4)
            w.tile<4>(q, ps, kt, vt, lane, R, a.scale_log2, d, row0, a.G, a.window, mask);
        else
            w.tile<RW>(q, ps, kt, vt, lane, R, a.scale_log2, d, row0, a.G, a.window, mask);
    }
    __device__ __forceinline__ void end(int lane, float *red, float2 *ml) {
        if (lane < RW) ml[lane] = make_float2(w.m, w.l);
        __syncwarp();
#pragma unroll
        for (int r = 0; r < RW; ++r)
            *reinterpret_cast<float4 *>(red + r * D + ((lane ^ (r & 7)) << 2)) = make_float4(w.o[r][0], w.o[r][1], w.o[r][2], w.o[r][3]);
    }
};

template <class C>
__device__ __forceinline__ void consume(const PagedAttn &a, uint8_t *sm) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR), *empty = full + STAGES;
    volatile int *abort = reinterpret_cast<volatile int *>(sm + C::OFF_ABORT);
    float *red = reinterpret_cast<float *>(sm + C::OFF_RED), *mine = red + warp * RW * D;
    float *ps = reinterpret_cast<float *>(sm + C::OFF_P) + warp * RW * 16;
    float2 *ml = reinterpret_cast<float2 *>(sm + C::OFF_ML);

    Work work;
    int stage = 0, phase = 0;
    uint64_t *meet = reinterpret_cast<uint64_t *>(sm + C::OFF_MEET);
    int meet_phase = 0;
    auto stop = [&]() {
        if (lane == 0) {
            *abort = 1;
            if (a.err) atomicOr(a.err, KDA_DEVERR_TIMEOUT);
        }
    };
    // (a bounded wait, unlike a named barrier: a warp that gave up never comes)
    auto meet_all = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(meet);
        const bool ok = wait_for<C>(a, meet, meet_phase, abort);
        meet_phase ^= 1;
        if (!ok) stop();
        return ok;
    };
    while (true) {
        if (!wait_for<C>(a, &full[stage], phase, abort)) {
            stop();
            break;
        }
        const Desc *ds = reinterpret_cast<const Desc *>(sm + C::OFF_DESC + stage * 64);
        const int4 head = *reinterpret_cast<const int4 *>(ds);  // flags, ord, wr, key0
        if (head.x & END) break;
        // wr = 1, 2, 4 or 8 warps side by side on the rows, wk = CONS / wr on the tiles in turn
        const int wl = __ffs(head.z) - 1, wrow = warp & (head.z - 1), wk = C::CONS >> wl, wpart = warp >> wl;
        if (!(head.x & (FIRST | LAST)) && (head.y & (wk - 1)) != wpart) {  // another warp's tile
            __syncwarp();  // (every lane has read the descriptor, which the producer may write next)
            if (lane == 0) mbar_arrive(&empty[stage]);
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1;
            }
            continue;
        }
        const Desc d = *ds;
        if (d.flags & FIRST) work.begin(a, d, wrow, lane, mine);
        if ((d.ord & (wk - 1)) == wpart && d.kvalid > 0) {
            uint8_t *kt = sm + stage * STAGE, *vt = kt + HALF;
            if (d.kfirst > 0 || d.kvalid < TK) zero_outside(vt, d.kfirst, d.kvalid, lane);
            work.tile(a, d, wrow, lane, kt, vt, mine, ps);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
        }
        if (d.flags & LAST) {
            // merge the warps that share rows, in warp order
            work.end(lane, mine, ml + warp * RW);
            if (!meet_all()) break;
            float *slot = paged_slot(a, d.slot);
            for (int r = warp; r < d.R; r += C::CONS) {
                const int rb = r / d.rpw, rl = r - rb * d.rpw;
                float M = -INFINITY, L = 0.f;
                for (int w = 0; w < wk; ++w) M = fmaxf(M, ml[(rb + w * d.wr) * RW + rl].x);
                const float refm = M == -INFINITY ? 0.f : M;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int w = 0; w < wk; ++w) {
                    const int src = (rb + w * d.wr) * RW + rl;
                    const float2 x = ml[src];
                    const float f = ex2(x.x - refm);
                    const float4 y = *reinterpret_cast<const float4 *>(red + src * D + ((lane ^ (rl & 7)) << 2));
                    L += f * x.y;
                    acc.x += f * y.x;
                    acc.y += f * y.y;
                    acc.z += f * y.z;
                    acc.w += f * y.w;
                }
                if (d.flags & WHOLE) {
                    const int rr = d.r0 + r, j = rr / a.G;
                    paged_store_row(a, true, d.tok0 + j, d.h * a.G + (rr - j * a.G), lane, acc, M, L, 1.f);
                } else {
                    if (lane == 0) reinterpret_cast<float2 *>(slot)[r] = make_float2(M, L);
                    reinterpret_cast<float4 *>(slot + 2 * a.slot_rows)[r * (D / 4) + lane] = acc;
                }
            }
            if (!(d.flags & WHOLE) && d.c0 == (int)blockIdx.x && threadIdx.x == 0) {  // the item's first piece
                a.lead[2 * blockIdx.x] = make_int4(d.tok0, d.h, d.r0, d.R);
                a.lead[2 * blockIdx.x + 1] = make_int4(d.slot, d.c0, d.c1, 1);
            }
            if (!meet_all()) break;
        }
    }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 2)
    paged_rows_kernel(const __grid_constant__ PagedMaps maps, const PagedAttn a, int min_per) {
    extern __shared__ __align__(1024) uint8_t sm[];
    // the join may be scheduled as soon as blocks end; it waits for this grid's writes by itself
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR), *empty = full + STAGES;
    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], C::CONS);
        }
        mbar_init(reinterpret_cast<uint64_t *>(sm + C::OFF_MEET), C::CONS);
        mbar_fence_init();
        *reinterpret_cast<int *>(sm + C::OFF_ABORT) = 0;
        a.lead[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);  // (no piece of this block leads, so far)
    }
    int64_t *scratch = reinterpret_cast<int64_t *>(sm + C::OFF_RED);
    auto tiles = [&](int i, int *err) { return line_tiles<C>(a, i, err); };
    const PagedLine line = paged_line<C::THREADS>(a, scratch, min_per, tiles, [](int64_t) { return 1; });
    if (line.P0 >= line.P1) return;
    __syncthreads();  // (the sums stood where the consumers' rows will)
    if (tid >= C::CONS * 32)
        produce<C>(a, maps, sm, line.P0, line.P1, line.per, line.req, line.before);
    else
        consume<C>(a, sm);
}

}  // namespace

int paged_rows_blocks() { return 2 * device_sm_count(); }

template <class C> static int launch(const PagedAttn &a, const PagedMaps &maps, cudaStream_t s) {
    const int rc = prepare_kernel((const void *)paged_rows_kernel<C>, C::SMEM, C::THREADS, nullptr);
    if (rc) return rc;
    // (a block of fewer tiles would only wait for its first)
    paged_rows_kernel<C><<<paged_rows_blocks(), C::THREADS, C::SMEM, s>>>(maps, a, HEAD + 1);
    note_launch("paged_rows", s);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int launch_paged_rows(PagedAttn a, const void *k, const void *v, int64_t page_stride, cudaStream_t s) {
    a.box = TK;  // (page sizes are multiples of 16)
    PagedMaps maps;
    const int rc = make_paged_row_maps(k, v, a.Hkv, a.page_size, a.n_pages, page_stride, TK, &maps);
    if (rc) return rc;
    const bool brief = a.wait_budget < SHORT_BUDGET, few = (int64_t)a.max_q * a.G <= RW;
    if (brief) return few ? launch<Cfg<4, true>>(a, maps, s) : launch<Cfg<8, true>>(a, maps, s);
    return few ? launch<Cfg<4, false>>(a, maps, s) : launch<Cfg<8, false>>(a, maps, s);
}

}  // namespace kda
