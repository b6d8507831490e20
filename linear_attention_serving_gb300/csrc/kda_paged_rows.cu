// kda_paged_rows.cu -- paged attention for few rows (single tokens, draft
// windows) and for the types without a tensor-core tile kernel of their own:
// every key and value is used for at most 64 rows, so the time is the pages'
// bytes over HBM, and the kernel is built to keep many of them in flight.
//
// A block has four consumer warps and one producer warp.  The producer walks
// the block's line of key tiles (8 KB of K and 8 KB of V each: 32 bf16, 64 e4m3
// or 16 fp32 keys), looks pages up in the block table, and has the tensor
// memory accelerator fill a ring of five tiles, two blocks on an SM: 160 KB in
// flight.  Consumers hold 16 rows each in mma.sync fragments.  Few rows
// (<= 16): the four warps take every fourth tile, each with its own running
// maximum and sum, merged in shared memory at the item's end.  More rows: the
// warps take 16 rows each (two by two up to 32) and share the tiles.
//
// Products, with fp32 accumulators (contraction and output indices are
// relabelled where that lets a thread load 4 or 16 bytes at once):
//   bf16  m16n8k16 on K and V as they are; the probabilities are rounded to
//         bf16 (2^-9 relative each, averaging out below the output's rounding)
//   e4m3  widened to fp16 in registers, which is exact; q is scaled by a power
//         of two per row so that fp16 holds it as precisely as bf16 did
//   fp32  plain fp32 multiply-adds: tf32 parts would lose digits that the fp32
//         path of this library keeps (three products of two parts each left 2.5e-6
//         where this leaves 4e-7), and with up to 16 rows a warp the memory's time
//         covers them.  A lane holds half a key's channels for the scores and four
//         channels of all keys for the output
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kda_paged.cuh"

namespace kda {
namespace {
using namespace tc;

constexpr int CONS = 4;                      // consumer warps
constexpr int THREADS = (CONS + 1) * 32;
constexpr int STAGES = 5;
constexpr int HALF = 8192;                   // bytes of K (and of V) of one tile
constexpr int STAGE = 2 * HALF;
constexpr int OFF_RED = STAGES * STAGE;      // [4][16][128] fp32
constexpr int OFF_P = (STAGES - 1) * STAGE;    // fp32: probabilities [4][16][16], in place of the last stage
constexpr int OFF_ML = OFF_RED + CONS * 16 * D * 4;
constexpr int OFF_DESC = OFF_ML + CONS * 16 * 8;
constexpr int OFF_BAR = OFF_DESC + STAGES * 64;
constexpr int OFF_MEET = OFF_BAR + 2 * STAGES * 8;  // the consumer warps' meeting at an item's end
constexpr int OFF_ABORT = OFF_MEET + 8;
constexpr int SMEM = OFF_ABORT + 16;
static_assert(OFF_RED % 1024 == 0 && OFF_ML % 16 == 0 && OFF_DESC % 16 == 0 && OFF_BAR % 8 == 0, "shared memory layout");

constexpr int BF16 = 0, E4M3 = 1, F32 = 2;   // kinds
template <int KIND> struct Kind;
template <> struct Kind<BF16> { static constexpr int TK = 32, ES = 2, NST = STAGES; };
template <> struct Kind<E4M3> { static constexpr int TK = 64, ES = 1, NST = STAGES; };
template <> struct Kind<F32> { static constexpr int TK = 16, ES = 4, NST = STAGES - 1; };

// what the producer says about a tile
struct __align__(16) Desc {
    int flags, ord, wr, key0, kvalid, tok0, h, r0, R, pos0, slot, c0, c1, pad0, pad1, pad2;
};
static_assert(sizeof(Desc) == 64, "descriptor size");
constexpr int FIRST = 1, LAST = 2, WHOLE = 4, END = 8, MASK = 16;

__device__ __forceinline__ int row_group(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

template <int KIND>
__device__ __forceinline__ int req_tiles(const PagedReq &r) {
    const int keys = r.kend - r.k0;
    return keys > 0 ? (keys + Kind<KIND>::TK - 1) / Kind<KIND>::TK : 1;
}
template <int KIND>
__device__ __forceinline__ int64_t line_tiles(const PagedAttn &a, int i, int *err) {
    const PagedReq r = paged_req(a, i, err);
    if (r.rows == 0) return 0;
    const int grp = row_group(r.rows);
    return (int64_t)a.Hkv * ((r.rows + grp - 1) / grp) * req_tiles<KIND>(r);
}

// ---------------------------------------------------------------- producer
template <int KIND>
__device__ __forceinline__ void produce(const PagedAttn &a, const PagedMaps &maps, uint8_t *sm, int64_t P0, int64_t P1,
                                        int64_t per, int req, int64_t before) {
    constexpr int TK = Kind<KIND>::TK, ES = Kind<KIND>::ES, NSUB = D * ES / 128, NST = Kind<KIND>::NST;
    const int lane = threadIdx.x & 31;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + OFF_BAR), *empty = full + STAGES;
    volatile int *abort = reinterpret_cast<volatile int *>(sm + OFF_ABORT);
    const int box = a.box, nbx = TK / box;
    int stage = 0, phase = 0, issued = 0;
    auto next_stage = [&]() -> bool {
        const bool ok = mbar_wait_ab(&empty[stage], phase ^ 1, abort);
        if (!__all_sync(0xffffffffu, ok)) {
            if (lane == 0) {
                *abort = 1;
                if (a.err) atomicOr(a.err, KDA_DEVERR_TIMEOUT);
                // let the copies in flight land before the block ends
                for (int i = 1; i <= NST && i <= issued; ++i) {
                    const int u = issued - i;
                    mbar_wait(&full[u % NST], (u / NST) & 1);
                }
            }
            __syncwarp();
            return false;
        }
        ++issued;
        return true;
    };
    auto advance = [&]() {
        if (++stage == NST) {
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
        const int nt = req_tiles<KIND>(r), grp = row_group(r.rows), ngrp = (r.rows + grp - 1) / grp;
        const int64_t in = pos - before, item = in / nt;
        const int h = (int)(item / ngrp), g = (int)(item - (int64_t)h * ngrp);
        const int64_t A = before + item * nt, B = A + nt;
        const int64_t seg_end = B < P1 ? B : P1;
        const int t_begin = (int)(pos - A), t_end = (int)(seg_end - A);
        const int r0 = g * grp, R = min(grp, r.rows - r0);
        const int posf = r.pos0 + r0 / a.G, posl = r.pos0 + (r0 + R - 1) / a.G;
        const int lo = a.window > 0 ? max(0, posf - a.window + 1) : 0, hi = posl + 1;  // keys that the group sees
        int tb = t_begin, te = t_end;
        if (hi <= lo) {
            te = tb;
        } else {
            tb = max(tb, (lo - r.k0) / TK);
            te = min(te, (hi - r.k0 + TK - 1) / TK);
        }
        Desc d;
        d.wr = grp / 16;
        d.tok0 = r.tok0;
        d.h = h;
        d.r0 = r0;
        d.R = R;
        d.pos0 = r.pos0;
        d.c0 = (int)(A / per);
        d.c1 = (int)((B - 1) / per);
        d.slot = 2 * (int)blockIdx.x + (pos == P0 ? 0 : 1);
        const int whole = pos == A && seg_end == B ? WHOLE : 0;
        if (te <= tb) {  // nothing to read: one empty tile so that the segment is finished all the same
            if (!next_stage()) return;
            if (lane == 0) {
                d.flags = FIRST | LAST | MASK | whole;
                d.ord = 0;
                d.key0 = 0;
                d.kvalid = 0;
                *reinterpret_cast<Desc *>(sm + OFF_DESC + stage * 64) = d;
                mbar_arrive(&full[stage]);
            }
            advance();
        }
        int cbase = -32, page = 0;
        for (int t = tb; t < te; ++t) {
            const int b0 = t * nbx;
            if (t == tb || b0 + nbx > cbase + 32) {  // pages of the next 32 boxes, one per lane
                cbase = b0;
                const int key = r.k0 + (cbase + lane) * box;
                page = 0;
                if (key < hi) {
                    page = a.table[(int64_t)req * a.max_blocks + key / a.page_size];
                    if (page < 0 || page >= a.n_pages) {
                        if (a.err) atomicOr(a.err, KDA_DEVERR_PAGE);
                        page = 0;
                    }
                }
            }
            const int key0 = r.k0 + t * TK, kvalid = min(TK, hi - key0);
            const int nb = (kvalid + box - 1) / box;
            const int pg = __shfl_sync(0xffffffffu, page, (b0 - cbase + lane) & 31);
            if (!next_stage()) return;
            if (lane == 0) {
                d.flags = (t == tb ? FIRST : 0) | (t == te - 1 ? LAST : 0) | whole;
                if (kvalid < TK || key0 + TK - 1 > posf || (a.window > 0 && key0 <= posl - a.window)) d.flags |= MASK;
                d.ord = t - tb;
                d.key0 = key0;
                d.kvalid = kvalid;
                *reinterpret_cast<Desc *>(sm + OFF_DESC + stage * 64) = d;
                mbar_expect_tx(&full[stage], (uint32_t)(nb * box * D * ES * 2));
            }
            __syncwarp();
            if (lane < nb) {
                const int key = key0 + lane * box, y = h * a.page_size + key % a.page_size;
                uint8_t *dst = sm + stage * STAGE + lane * box * 128;
#pragma unroll
                for (int sub = 0; sub < NSUB; ++sub) {
                    tma_load_3d(dst + sub * TK * 128, &maps.k, sub * (128 / ES), y, pg, &full[stage]);
                    tma_load_3d(dst + HALF + sub * TK * 128, &maps.v, sub * (128 / ES), y, pg, &full[stage]);
                }
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
        reinterpret_cast<Desc *>(sm + OFF_DESC + stage * 64)->flags = END;
        mbar_arrive(&full[stage]);
    }
}

// ---------------------------------------------------------------- fragments
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_b(float (&c)[4], const uint32_t (&x)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_h(float (&c)[4], const uint32_t (&x)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint32_t pack_f16(float x, float y) {
    const __half2 p = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return (uint32_t)r.x | ((uint32_t)r.y << 16);
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Key of column c of an 8-key group for the kinds that load whole 16-byte
// pieces of a row: threads that read together then hit different banks, for K
// (columns 2p and 2p + 1: rows differ in bit 2) and for V (columns 0, 2, 4, 6
// and 1, 3, 5, 7: bits 1 and 2 take all four values).
__device__ __forceinline__ int key_of_col(int c) { return (c & 1) ? ((c - 1) ^ 5) : c; }

template <int KIND> struct Rows;  // a warp's 16 rows: q fragments and products

template <> struct Rows<BF16> {
    uint32_t q[8][4];
    __device__ __forceinline__ void load(const void *p0, const void *p1, int t, float &f0, float &f1) {
        const uint32_t *a = (const uint32_t *)p0, *b = (const uint32_t *)p1;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            q[s][0] = a ? a[8 * s + t] : 0;
            q[s][1] = b ? b[8 * s + t] : 0;
            q[s][2] = a ? a[8 * s + 4 + t] : 0;
            q[s][3] = b ? b[8 * s + 4 + t] : 0;
        }
        f0 = f1 = 1.f;
    }
    static __device__ __forceinline__ int key(int c) { return c; }
    __device__ __forceinline__ void qk(const uint8_t *k, int lane, float (&s)[4][4]) {
        const uint32_t base = smem_u32(k);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = 8 * j + (lane & 7);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < 8; ks += 2) {
                const int ch = 2 * ks + (lane >> 3);  // 16-byte chunk of the row, 0..15
                uint32_t b[4];
                ldsm4(base + (ch >> 3) * 4096 + row * 128 + (((ch & 7) ^ (row & 7)) << 4), b);
                mma_b(s[j], q[ks], b[0], b[1]);
                mma_b(s[j], q[ks + 1], b[2], b[3]);
            }
        }
    }
    __device__ __forceinline__ void pv(const uint8_t *v, int lane, const float (&p)[4][4], float (&o)[16][4]) {
        const uint32_t base = smem_u32(v);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const uint32_t x[4] = {pack_bf16(p[2 * ks][0], p[2 * ks][1]), pack_bf16(p[2 * ks][2], p[2 * ks][3]),
                                   pack_bf16(p[2 * ks + 1][0], p[2 * ks + 1][1]), pack_bf16(p[2 * ks + 1][2], p[2 * ks + 1][3])};
            const int row = 16 * ks + (lane & 15);
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                const int ch = j + (lane >> 4);
                uint32_t b[4];
                ldsm4t(base + (ch >> 3) * 4096 + row * 128 + (((ch & 7) ^ (row & 7)) << 4), b);
                mma_b(o[j], x, b[0], b[1]);
                mma_b(o[j + 1], x, b[2], b[3]);
            }
        }
    }
    // the fragments' 16-byte pieces of a row in the merge buffer
    static __device__ __forceinline__ void put(float *red, int g, int t, const float (&o)[16][4]) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int row = g + 8 * hf, c = 2 * j + (t >> 1);
                *reinterpret_cast<float2 *>(red + row * D + ((c ^ (row & 7)) << 2) + 2 * (t & 1)) =
                    make_float2(o[j][2 * hf], o[j][2 * hf + 1]);
            }
    }
};

// relabelled output columns (e4m3, fp32): n-tile j, column c is channel
// 4 c + (j & 3) + 32 (j >> 2), so the thread's columns 2t, 2t + 1 of four
// n-tiles are eight channels in a row
__device__ __forceinline__ void put_relabelled(float *red, int g, int t, const float (&o)[16][4]) {
#pragma unroll
    for (int jq = 0; jq < 4; ++jq)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = g + 8 * hf, c = 8 * jq + 2 * t + e;
                *reinterpret_cast<float4 *>(red + row * D + ((c ^ (row & 7)) << 2)) =
                    make_float4(o[4 * jq][2 * hf + e], o[4 * jq + 1][2 * hf + e], o[4 * jq + 2][2 * hf + e],
                                o[4 * jq + 3][2 * hf + e]);
            }
}

template <> struct Rows<E4M3> {
    uint32_t q[8][4];
    // k-step 4 hf + j of thread t holds channels 16 (t + 4 hf) + 4 j + 0..3
    __device__ __forceinline__ void load(const void *p0, const void *p1, int t, float &f0, float &f1) {
        const void *p[2] = {p0, p1};
        float *f[2] = {&f0, &f1};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            uint2 w[8];
            float top = 0.f;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                w[s] = p[r] ? ((const uint2 *)p[r])[4 * (t + 4 * (s >> 2)) + (s & 3)] : make_uint2(0, 0);
                top = fmaxf(top, fmaxf(fmaxf(fabsf(bf_lo(w[s].x)), fabsf(bf_hi(w[s].x))),
                                       fmaxf(fabsf(bf_lo(w[s].y)), fabsf(bf_hi(w[s].y)))));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^-e with e the exponent of the row's largest value (none for 0, inf and the ends of the range)
            const int e = (int)(__float_as_uint(top) >> 23) - 127;
            const bool ok = e > -120 && e < 120;
            const float down = ok ? __uint_as_float((uint32_t)(127 - e) << 23) : 1.f;
            *f[r] = ok ? __uint_as_float((uint32_t)(127 + e) << 23) : 1.f;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                q[s][r] = pack_f16(bf_lo(w[s].x) * down, bf_hi(w[s].x) * down);
                q[s][2 + r] = pack_f16(bf_lo(w[s].y) * down, bf_hi(w[s].y) * down);
            }
        }
    }
    static __device__ __forceinline__ int key(int c) { return key_of_col(c); }
    __device__ __forceinline__ void qk(const uint8_t *k, int lane, float (&s)[8][4]) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int row = 8 * j + key_of_col(g);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint4 w = *reinterpret_cast<const uint4 *>(k + row * 128 + (((t + 4 * hf) ^ (row & 7)) << 4));
                const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) mma_h(s[j], q[4 * hf + i], e4m3x2_f16x2(x[i] & 0xffff), e4m3x2_f16x2(x[i] >> 16));
            }
        }
    }
    __device__ __forceinline__ void pv(const uint8_t *v, int lane, const float (&p)[8][4], float (&o)[16][4]) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            const uint32_t x[4] = {pack_f16(p[2 * ks][0], p[2 * ks][1]), pack_f16(p[2 * ks][2], p[2 * ks][3]),
                                   pack_f16(p[2 * ks + 1][0], p[2 * ks + 1][1]), pack_f16(p[2 * ks + 1][2], p[2 * ks + 1][3])};
#pragma unroll
            for (int jq = 0; jq < 4; ++jq) {
                const int ch = 2 * jq + (g >> 2);
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // keys of columns 2t, 2t + 1 of the two 8-key groups
                    const int row = 16 * ks + 8 * (e >> 1) + key_of_col(2 * t + (e & 1));
                    w[e] = *reinterpret_cast<const uint32_t *>(v + row * 128 + ((ch ^ (row & 7)) << 4) + 4 * (g & 3));
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // channel 4 g + e + 32 jq: byte e of each
                    const uint32_t sel = (uint32_t)e | ((uint32_t)(4 + e) << 4);
                    mma_h(o[4 * jq + e], x, e4m3x2_f16x2(__byte_perm(w[0], w[1], sel) & 0xffff),
                          e4m3x2_f16x2(__byte_perm(w[2], w[3], sel) & 0xffff));
                }
            }
        }
    }
    static __device__ __forceinline__ void put(float *red, int g, int t, const float (&o)[16][4]) { put_relabelled(red, g, t, o); }
};

// fp32: lane = (key lane % 16, half of the channels lane / 16) for the scores, four
// channels for the output; maxima and sums of row r in lane r.
struct RowsF32 {
    float o[16][4], m, l;
    __device__ __forceinline__ void tile(const float *q, float *ps, const uint8_t *k, const uint8_t *v, int lane, int R, float sc,
                                         const Desc &d, int row0, int G, int window, bool mask) {
        const int key = lane & 15, hf = lane >> 4;
        float4 kr[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            const int ch = 16 * hf + c;
            kr[c] = *reinterpret_cast<const float4 *>(k + (ch >> 3) * 2048 + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
        }
        float corr = 1.f;  // of row `lane`
#pragma unroll 1
        for (int r = 0; r < R; ++r) {
            const float4 *qr = reinterpret_cast<const float4 *>(q + r * D) + 16 * hf;
            float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const float4 x = qr[c];
                a0 = fmaf(x.x, kr[c].x, a0);
                a1 = fmaf(x.y, kr[c].y, a1);
                a2 = fmaf(x.z, kr[c].z, a2);
                a3 = fmaf(x.w, kr[c].w, a3);
            }
            float s = (a0 + a1) + (a2 + a3);
            s += __shfl_xor_sync(0xffffffffu, s, 16);
            if (mask) {
                const int pos = d.pos0 + (row0 + r) / G, at = d.key0 + key;
                if (!(at <= pos && (window <= 0 || at > pos - window) && key < d.kvalid)) s = -INFINITY;
            }
            float top = s;
#pragma unroll
            for (int x = 8; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float old = __shfl_sync(0xffffffffu, m, r), mn = fmaxf(old, top * sc);
            const float ref = mn == -INFINITY ? 0.f : mn;
            if (lane == r) {
                corr = ex2(m - ref);
                m = mn;
            }
            const float p = ex2(fmaf(s, sc, -ref));
            if (lane < 16) ps[r * 16 + lane] = p;
        }
        __syncwarp();
        const bool moved = __any_sync(0xffffffffu, corr != 1.f);
        l *= corr;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
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
            for (int r = 0; r < 16; ++r) {
                if (r < R) {
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
// V rows past the keys may hold anything (0 x NaN is NaN): zero them.
template <int KIND>
__device__ __forceinline__ void zero_past(uint8_t *vt, int kvalid, int lane) {
    constexpr int TK = Kind<KIND>::TK, NSUB = D * Kind<KIND>::ES / 128;
    for (int x = lane; x < (TK - kvalid) * NSUB * 8; x += 32) {
        const int row = kvalid + x / (NSUB * 8), c = x % (NSUB * 8);
        *reinterpret_cast<uint4 *>(vt + (c >> 3) * TK * 128 + row * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
    }
    fence_async_smem();
    __syncwarp();
}

// A warp's 16 rows in mma.sync fragments (bf16, e4m3).
template <int KIND> struct Work {
    static constexpr int TK = Kind<KIND>::TK, NT = TK / 8;
    Rows<KIND> rows;
    float o[16][4], m[2], l[2], sc[2];
    int last[2];  // position of the thread's two rows

    __device__ __forceinline__ void begin(const PagedAttn &a, const Desc &d, int wrow, int lane, float *) {
        const int g = lane >> 2, t = lane & 3;
        const char *p[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 16 * wrow + g + 8 * e, rr = d.r0 + r, j = rr / a.G;
            last[e] = d.pos0 + j;
            p[e] = r < d.R ? (const char *)a.q + ((int64_t)(d.tok0 + j) * a.Hq + d.h * a.G + (rr - j * a.G)) * D * 2 : nullptr;
            m[e] = -INFINITY;
            l[e] = 0.f;
        }
        rows.load(p[0], p[1], t, sc[0], sc[1]);
        const float f = a.scale_log2 * (KIND == E4M3 ? a.k_scale[d.h] : 1.f);
        sc[0] *= f;
        sc[1] *= f;
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    }
    __device__ __forceinline__ void tile(const PagedAttn &a, const Desc &d, int, int lane, const uint8_t *kt, const uint8_t *vt,
                                         const float *, float *) {
        const int t = lane & 3;
        float s[NT][4];
        rows.qk(kt, lane, s);
        if (d.flags & MASK) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = 8 * j + Rows<KIND>::key(2 * t + (e & 1)), key = d.key0 + at, pos = last[e >> 1];
                    const bool seen = key <= pos && (a.window <= 0 || key > pos - a.window) && at < d.kvalid;
                    if (!seen) s[j][e] = -INFINITY;
                }
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[j][e]);
        float ref[2], corr[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
            const float mn = fmaxf(m[e], top[e] * sc[e]);
            ref[e] = mn == -INFINITY ? 0.f : mn;
            corr[e] = ex2(m[e] - ref[e]);
            m[e] = mn;
            l[e] *= corr[e];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[j][e] = ex2(fmaf(s[j][e], sc[e >> 1], -ref[e >> 1]));
                l[e >> 1] += s[j][e];
            }
        if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][e] *= corr[e >> 1];
        }
        rows.pv(vt, lane, s, o);
    }
    __device__ __forceinline__ void end(int lane, float *red, float2 *ml) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            if (t == 0) ml[g + 8 * e] = make_float2(m[e], l[e]);
        }
        Rows<KIND>::put(red, g, t, o);
    }
};
template <> struct Work<F32> {
    RowsF32 w;
    __device__ __forceinline__ void begin(const PagedAttn &a, const Desc &d, int wrow, int lane, float *q) {
        w.m = -INFINITY;
        w.l = 0.f;
        const int R = min(16, d.R - 16 * wrow);
        for (int r = 0; r < R; ++r) {  // the queries stand where the output goes at the end
            const int rr = d.r0 + 16 * wrow + r, j = rr / a.G;
            const float4 *src = (const float4 *)a.q + ((int64_t)(d.tok0 + j) * a.Hq + d.h * a.G + (rr - j * a.G)) * (D / 4);
            reinterpret_cast<float4 *>(q + r * D)[lane] = src[lane];
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 16; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) w.o[r][e] = 0.f;
    }
    __device__ __forceinline__ void tile(const PagedAttn &a, const Desc &d, int wrow, int lane, const uint8_t *kt, const uint8_t *vt,
                                         const float *q, float *ps) {
        w.tile(q, ps, kt, vt, lane, min(16, d.R - 16 * wrow), a.scale_log2, d, d.r0 + 16 * wrow, a.G, a.window, d.flags & MASK);
    }
    __device__ __forceinline__ void end(int lane, float *red, float2 *ml) {
        if (lane < 16) ml[lane] = make_float2(w.m, w.l);
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 16; ++r)
            *reinterpret_cast<float4 *>(red + r * D + ((lane ^ (r & 7)) << 2)) = make_float4(w.o[r][0], w.o[r][1], w.o[r][2], w.o[r][3]);
    }
};

template <int KIND>
__device__ __forceinline__ void consume(const PagedAttn &a, uint8_t *sm) {
    constexpr int TK = Kind<KIND>::TK, NST = Kind<KIND>::NST;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + OFF_BAR), *empty = full + STAGES;
    volatile int *abort = reinterpret_cast<volatile int *>(sm + OFF_ABORT);
    float *red = reinterpret_cast<float *>(sm + OFF_RED), *mine = red + warp * 16 * D;
    float *ps = reinterpret_cast<float *>(sm + OFF_P) + warp * 256;
    float2 *ml = reinterpret_cast<float2 *>(sm + OFF_ML);

    Work<KIND> work;
    int stage = 0, phase = 0;
    uint64_t *meet = reinterpret_cast<uint64_t *>(sm + OFF_MEET);
    int meet_phase = 0;
    // (a bounded wait, unlike a named barrier: a warp that gave up never comes)
    auto meet_all = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(meet);
        const bool ok = __all_sync(0xffffffffu, mbar_wait_ab(meet, meet_phase, abort));
        meet_phase ^= 1;
        if (!ok && lane == 0) *abort = 1;
        return ok;
    };
    while (true) {
        const bool ok = mbar_wait_ab(&full[stage], phase, abort);
        if (!__all_sync(0xffffffffu, ok)) {
            if (lane == 0) {
                *abort = 1;
                if (a.err) atomicOr(a.err, KDA_DEVERR_TIMEOUT);
            }
            break;
        }
        const Desc d = *reinterpret_cast<const Desc *>(sm + OFF_DESC + stage * 64);
        if (d.flags & END) break;
        const int wrow = warp % d.wr, wk = CONS / d.wr, wpart = warp / d.wr;
        if (d.flags & FIRST) work.begin(a, d, wrow, lane, mine);
        if (d.ord % wk == wpart && d.kvalid > 0) {
            uint8_t *kt = sm + stage * STAGE, *vt = kt + HALF;
            if (d.kvalid < TK) zero_past<KIND>(vt, d.kvalid, lane);
            work.tile(a, d, wrow, lane, kt, vt, mine, ps);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == NST) {
            stage = 0;
            phase ^= 1;
        }
        if (d.flags & LAST) {
            // merge the warps that share rows, in warp order
            work.end(lane, mine, ml + warp * 16);
            if (!meet_all()) break;
            float *slot = paged_slot(a, d.slot);
            const float vs = KIND == E4M3 ? a.v_scale[d.h] : 1.f;
            for (int r = warp; r < d.R; r += CONS) {
                const int rb = r >> 4, rl = r & 15;
                float M = -INFINITY, L = 0.f;
                for (int w = 0; w < wk; ++w) M = fmaxf(M, ml[(rb + w * d.wr) * 16 + rl].x);
                const float refm = M == -INFINITY ? 0.f : M;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int w = 0; w < wk; ++w) {
                    const int src = (rb + w * d.wr) * 16 + rl;
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
                    paged_store_row(a, KIND == F32, d.tok0 + j, d.h * a.G + (rr - j * a.G), lane, acc, M, L, vs);
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

template <int KIND>
__global__ void __launch_bounds__(THREADS, 2)
    paged_rows_kernel(const __grid_constant__ PagedMaps maps, const PagedAttn a, int min_per) {
    extern __shared__ __align__(1024) uint8_t sm[];
    // the join may be scheduled as soon as blocks end; it waits for this grid's writes by itself
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + OFF_BAR), *empty = full + STAGES;
    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], CONS);
        }
        mbar_init(reinterpret_cast<uint64_t *>(sm + OFF_MEET), CONS);
        mbar_fence_init();
        *reinterpret_cast<int *>(sm + OFF_ABORT) = 0;
        a.lead[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);  // (no piece of this block leads, so far)
    }
    int64_t *scratch = reinterpret_cast<int64_t *>(sm + OFF_RED);
    auto tiles = [&](int i, int *err) { return line_tiles<KIND>(a, i, err); };
    const PagedLine line = paged_line<THREADS>(a, scratch, min_per, 1, tiles);
    if (line.P0 >= line.P1) return;
    if (tid >= CONS * 32)
        produce<KIND>(a, maps, sm, line.P0, line.P1, line.per, line.req, line.before);
    else
        consume<KIND>(a, sm);
}

template <int KIND>
int launch_kind(PagedAttn a, const void *k, const void *v, int cache_dtype, int64_t page_stride, cudaStream_t s) {
    constexpr int TK = Kind<KIND>::TK;
    int box = 16;
    while (box < TK && a.page_size % (2 * box) == 0) box *= 2;
    a.box = box;
    PagedMaps maps;
    int rc = make_paged_maps(k, v, cache_dtype, a.Hkv, a.page_size, a.n_pages, page_stride, box, &maps);
    if (rc) return rc;
    const void *f = (const void *)paged_rows_kernel<KIND>;
    if ((rc = prepare_kernel(f, SMEM, THREADS, nullptr))) return rc;
    const int blocks = paged_rows_blocks();
    // at least 8 tiles a block (two for each warp): below that the pieces cost more than they save
    paged_rows_kernel<KIND><<<blocks, THREADS, SMEM, s>>>(maps, a, 8);
    note_launch("paged_rows", s);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

int paged_rows_blocks() { return 2 * device_sm_count(); }

int launch_paged_rows(const PagedAttn &a, int cache_dtype, const void *k, const void *v, int64_t page_stride,
                      cudaStream_t s) {
    switch (cache_dtype) {
        case KDA_BF16: return launch_kind<BF16>(a, k, v, cache_dtype, page_stride, s);
        case KDA_E4M3: return launch_kind<E4M3>(a, k, v, cache_dtype, page_stride, s);
        default: return launch_kind<F32>(a, k, v, cache_dtype, page_stride, s);
    }
}

}  // namespace kda
