// Building blocks of the warp-specialised tcgen05 kernels (chunked prefill,
// shared-prefix decode): shared-memory and instruction descriptors, products,
// tensor-memory loads and stores, bounded waits.
#pragma once

#include "kvc_device.cuh"

namespace kvc {

constexpr int kWsKeys = 64;                 // keys per tile
constexpr int kWsRows = 128;                // rows per Q tile (TMEM lanes)

__device__ __forceinline__ uint64_t ws_sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

__host__ __device__ constexpr uint32_t ws_idesc(int M, int N, int b_n_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_n_major << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void ws_mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// The same with A from tensor memory (a_tmem: lane = row, two 16-bit elements
// along K per 32-bit column).
__device__ __forceinline__ void ws_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void ws_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// S[128 x 64] = Q[128 x D] K[64 x D]^T, both in shared memory; qd, kd: descriptors
// of their first column blocks (QB and KB bytes between blocks).  A descriptor's
// address field counts 16 bytes and never carries out of its 14 bits here, so
// the k-steps add constants: a thread that builds descriptors anew for each
// product spends more time on them than the tensor cores on the product.
template <int D, int QB, int KB>
__device__ __forceinline__ void ws_issue_s(uint32_t d_tmem, uint64_t qd, uint64_t kd) {
    constexpr uint32_t idesc = ws_idesc(kWsRows, kWsKeys, 0);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
        ws_mma(d_tmem, qd + (uint64_t)(((ks >> 2) * QB + (ks & 3) * 32) >> 4),
               kd + (uint64_t)(((ks >> 2) * KB + (ks & 3) * 32) >> 4), idesc, ks > 0);
}

// O[128 x D] (+)= P[128 x 64] V[64 x D]: P in tensor memory (bf16 pairs), vd: the
// descriptor of V's rows 0 .. 15; `more`: accumulate onto O.
template <int D>
__device__ __forceinline__ void ws_issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint64_t vd, uint32_t more) {
    constexpr uint32_t idesc = ws_idesc(kWsRows, D, 1);
#pragma unroll
    for (int ks = 0; ks < kWsKeys / 16; ++ks)
        ws_mma_ts(d_tmem, p_tmem + (uint32_t)(ks * 8), vd + (uint64_t)((ks * 16 * 128) >> 4), idesc,
                  ks > 0 ? 1u : more);
}

__device__ __forceinline__ void ws_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void ws_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void ws_ld32(uint32_t taddr, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}

__device__ __forceinline__ void ws_st32(uint32_t taddr, const float* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
        "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
        "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
        "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
        "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
        "r"(__float_as_uint(v[15])), "r"(__float_as_uint(v[16])), "r"(__float_as_uint(v[17])),
        "r"(__float_as_uint(v[18])), "r"(__float_as_uint(v[19])), "r"(__float_as_uint(v[20])),
        "r"(__float_as_uint(v[21])), "r"(__float_as_uint(v[22])), "r"(__float_as_uint(v[23])),
        "r"(__float_as_uint(v[24])), "r"(__float_as_uint(v[25])), "r"(__float_as_uint(v[26])),
        "r"(__float_as_uint(v[27])), "r"(__float_as_uint(v[28])), "r"(__float_as_uint(v[29])),
        "r"(__float_as_uint(v[30])), "r"(__float_as_uint(v[31]))
        : "memory");
}

__device__ __forceinline__ void ws_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void ws_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 2^a and 2^b in one special-function op: the arguments rounded to fp16
// (ex2.approx.f16x2) and the results widened to fp32.  Softmax arguments here
// are <= 8 (the lazy reference max), so fp16 keeps them to 2^-8 or better --
// finer than the bf16 rounding P gets for P V; a masked key's -inf gives 0.
__device__ __forceinline__ float2 ws_ex2_pair(float a, float b) {
    float2 r;
    asm("{\n\t.reg .b32 h;\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.f16x2.f32 h, %3, %2;\n\t"
        "ex2.approx.f16x2 h, h;\n\t"
        "mov.b32 {lo, hi}, h;\n\t"
        "cvt.f32.f16 %0, lo;\n\t"
        "cvt.f32.f16 %1, hi;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float ws_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float ws_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float ws_max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

__device__ __forceinline__ float ws_max3_nan(float a, float b, float c) {    // NaN if one of them is
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Largest of 64 values, in four chains of three-input maxima.
__device__ __forceinline__ float ws_max64(const float (&v)[kWsKeys]) {
    float m[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        m[u] = ws_max3(v[16 * u], v[16 * u + 1], v[16 * u + 2]);
#pragma unroll
        for (int k = 3; k < 15; k += 2) m[u] = ws_max3(m[u], v[16 * u + k], v[16 * u + k + 1]);
        m[u] = fmaxf(m[u], v[16 * u + 15]);
    }
    return fmaxf(ws_max3(m[0], m[1], m[2]), m[3]);
}

// p_k = 2^(a v_k + c) in place (a masked key's v = -inf gives 0); returns their sum.
__device__ __forceinline__ float ws_exp64(float (&v)[kWsKeys], float a, float c) {
    float2 ls[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    const float2 a2 = make_float2(a, a), c2 = make_float2(c, c);
#pragma unroll
    for (int k = 0; k < kWsKeys; k += 2) {
        const float2 d = __ffma2_rn(make_float2(v[k], v[k + 1]), a2, c2);
        v[k] = ws_ex2(d.x);
        v[k + 1] = ws_ex2(d.y);
        ls[(k >> 1) & 3] = __fadd2_rn(ls[(k >> 1) & 3], make_float2(v[k], v[k + 1]));
    }
    const float2 s = __fadd2_rn(__fadd2_rn(ls[0], ls[1]), __fadd2_rn(ls[2], ls[3]));
    return s.x + s.y;
}

__device__ __forceinline__ float ws_hold30(float x) {    // min(x, 30), NaN if x is
    float y;
    asm("min.NaN.f32 %0, %1, 0f41F00000;" : "=f"(y) : "f"(x));
    return y;
}

// v = -1 / (2^(ci x) + 1) in place, the argument of a capped score (cap tanh =
// 2 cap v + cap).  Reciprocals run at half the exponentials' rate here: four
// denominators share one, 1 / a = b (c d) / (a b c d) and so on (measured: 64 keys of
// two warps 1590 -> 1001 cycles).  Exponents are held to 30 so that no product
// overflows: tanh is 1 - 2^-29 there, 1 in fp32.  A NaN goes to its three neighbours
// too: one among the keys that the row attends makes its result NaN anyhow, others are to
// be masked before the cap.  Returns NaN if a score was NaN.
template <int N>
__device__ __forceinline__ float ws_cap(float (&v)[N], float ci) {
    const float2 c2 = make_float2(ci, ci), one = make_float2(1.f, 1.f);
    float any = 0.f, last = 0.f;
#pragma unroll
    for (int k = 0; k < N; k += 4) {
        const float2 y0 = __fmul2_rn(make_float2(v[k], v[k + 1]), c2), y1 = __fmul2_rn(make_float2(v[k + 2], v[k + 3]), c2);
        const float2 e0 = __fadd2_rn(make_float2(ws_ex2(ws_hold30(y0.x)), ws_ex2(ws_hold30(y0.y))), one);
        const float2 e1 = __fadd2_rn(make_float2(ws_ex2(ws_hold30(y1.x)), ws_ex2(ws_hold30(y1.y))), one);
        const float2 pq = __fmul2_rn(make_float2(e0.x, e1.x), make_float2(e0.y, e1.y));    // a b, c d
        const float r = -ws_rcp(pq.x * pq.y);
        const float2 rp = __fmul2_rn(make_float2(r, r), make_float2(pq.y, pq.x));          // -1 / (a b), -1 / (c d)
        const float2 x0 = __fmul2_rn(make_float2(e0.y, e0.x), make_float2(rp.x, rp.x));
        const float2 x1 = __fmul2_rn(make_float2(e1.y, e1.x), make_float2(rp.y, rp.y));
        v[k] = x0.x;
        v[k + 1] = x0.y;
        v[k + 2] = x1.x;
        v[k + 3] = x1.y;
        if (k & 4)
            any = ws_max3_nan(any, last, r);
        else
            last = r;
    }
    return any;
}

// Keys lo .. hi of a tile of N stay, the others become -inf (as bits of one word:
// two compares a key took three times as long).
template <int N>
__device__ __forceinline__ void ws_mask_range(float (&v)[N], int lo, int hi) {
#pragma unroll
    for (int w = 0; w < N / 32; ++w) {
        const int l = lo - 32 * w, h = hi - 32 * w;
        uint32_t m = h >= 31 ? 0xffffffffu : (h < 0 ? 0u : (2u << h) - 1u);
        m &= l <= 0 ? 0xffffffffu : (l > 31 ? 0u : 0xffffffffu << l);
#pragma unroll
        for (int k = 0; k < 32; ++k) v[32 * w + k] = ((m >> k) & 1u) ? v[32 * w + k] : -INFINITY;
    }
}

// try_wait with a suspend-time hint: a thread whose phase is not complete
// sleeps until it completes (or the hint, 0.1 ms, runs out) instead of coming
// back to re-issue the test, which would take issue slots from the softmax warps
__device__ __forceinline__ bool ws_try_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, 100000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Whether the phase of this parity has completed (asked once, without sleeping).
__device__ __forceinline__ bool ws_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// A bounded wait that also gives up once another role has given up.
__device__ __forceinline__ bool ws_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (ws_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!ws_try_wait(bar, parity)) {
        if (*abort || clock64() - t0 > kWaitCycles) return false;
    }
    return true;
}

}  // namespace kvc
