// kda_paged_tc.cuh -- what the two tensor-core kernels of paged attention share:
// key tiles of 128 keys and their count in closed form, bounded waits, TMEM loads
// and stores, paired fp32 arithmetic.
#pragma once

#include "kda_paged.cuh"

namespace kda {
namespace tc {

constexpr int KEY_TILE = 128;

// sum_{i < n} floor((a i + b) / m) for a, b >= 0: whole parts of a / m and b / m
// first; then, with K = floor((a (n - 1) + b) / m), counting the points below the
// line by rows instead of columns gives
//   K (n - 1) - sum_{j < K} floor((m j + m - b - 1) / a),
// the same kind of sum on smaller numbers (Euclid's steps on a and m).
// a (n - 1) + b < 2^32: key positions are below 2^31.
__device__ __forceinline__ int64_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
    if (n == 1) return b / m;
    int64_t s = 0, sign = 1;
    while (n > 0) {
        const uint32_t qa = a / m, qb = b / m;
        s += sign * ((int64_t)qa * ((int64_t)n * (n - 1) / 2) + (int64_t)qb * n);
        a -= qa * m;
        b -= qb * m;
        const uint32_t K = (a * (n - 1) + b) / m;
        if (K == 0) break;
        s += sign * ((int64_t)K * (n - 1));
        sign = -sign;
        b = m - b - 1;
        n = K;
        const uint32_t t = m;
        m = a;
        a = t;
    }
    return s;
}

// Key tiles [t0, t1) of the tokens j0 .. j1 of a request (none: t1 = t0).
__device__ __forceinline__ void key_tiles(const PagedAttn &a, const PagedReq &r, int j0, int j1, int &lo, int &hi, int &t0, int &t1) {
    hi = r.pos0 + j1 + 1;
    lo = first_seen(a, r.pos0 + j0);
    if (hi <= 0) {
        t0 = t1 = 0;
        return;
    }
    t0 = lo / KEY_TILE;
    t1 = (hi + KEY_TILE - 1) / KEY_TILE;
}
// Bounded waits of a whole converged warp that stop the block when one runs out.  The
// clock and the abort flag are looked at on every 64th try only: the waits are on the
// path of every tile.  SHORT: a budget of the launch's own, under SHORT_BUDGET, looked at
// on every try, none of which sleeps in hardware (one kernel for both made prompts 2% and
// e4m3 single tokens 1 to 5% slower, so the short budgets have one of their own).
template <bool SHORT>
struct Waits {
    volatile int *abort;
    int32_t *err;
    long long budget;
    __device__ bool operator()(uint64_t *bar, int parity) const {
        if constexpr (SHORT) {
            const long long t0 = clock64();
            while (!__all_sync(0xffffffffu, mbar_test_wait(bar, parity)))
                if (__any_sync(0xffffffffu, *abort || clock64() - t0 > budget)) return give_up();
            return true;
        } else {
            if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
            const long long t0 = clock64();
            for (uint32_t n = 1;; ++n) {
                if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
                if (n % 64 == 0 && __any_sync(0xffffffffu, *abort || clock64() - t0 > WAIT_BUDGET_CYCLES)) break;
            }
            return give_up();
        }
    }
    __device__ bool give_up() const {
        if ((threadIdx.x & 31) == 0) {
            if (!*abort && err) atomicOr(err, KDA_DEVERR_TIMEOUT);
            *abort = 1;
        }
        __syncwarp();
        return false;
    }
};

// How many of NTHR threads say so (a barrier of theirs).
template <int NTHR>
__device__ __forceinline__ int meet_count(int id, bool pred) {
    int n;
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %1, 0;\n barrier.red.popc.u32 %0, %2, %3, p;\n}\n"
                 : "=r"(n)
                 : "r"((uint32_t)pred), "r"(id), "n"(NTHR)
                 : "memory");
    return n;
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
// The loads above have arrived: nothing that uses the values moves before this.
__device__ __forceinline__ void tmem_arrived(float *o) {
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(o[i]));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *o) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]), "r"(o[8]), "r"(o[9]), "r"(o[10]),
        "r"(o[11]), "r"(o[12]), "r"(o[13]), "r"(o[14]), "r"(o[15])
        : "memory");
}
// two fp32 operations at once, and the largest of three
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float &x, float &y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r)); }
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
// 32 bytes of one thread at once (dst 32-byte aligned)
__device__ __forceinline__ void store32(void *dst, const uint32_t (&u)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]),
                 "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }


}  // namespace tc
}  // namespace kda
