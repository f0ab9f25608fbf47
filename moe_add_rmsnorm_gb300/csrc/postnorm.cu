// The norms around a block: norm after it, its gate and residual scale, the residual add, and the norm before the next
// block with its int8 epilogue, in one pass (q8moe.h, postnorm_add_rmsnorm_q8).
//
// A row is one CTA's registers: its two inputs are read once, the two sums of squares are the only exchanges, and every
// output is written from the registers that hold it.  Both norms, the products and the residual sum are pairs of f32 up to
// the one rounding of s and the one of y, so that the words, which turn on values next to a border, are the formula's.
// Measured, replayed: 4096 rows of 4096, a gate a channel, y and the sum written, 54 us (268 MB, 5.0 TB/s, 73% of the measured
// copy rate): arithmetic in pairs, some 93 instructions a value, fills 80% of the issue slots.
// One row of 2048 3.3, 37 of 5120 7.5: two reductions across the CTA, one after the other.
#include <math.h>

#include "common.cuh"
#include "ffn4.h"

namespace q8 {
namespace {

struct PostnormParams {
    const float *a, *b, *w_post, *w_pre, *gate;
    int64_t gate_row, gate_col;
    float scale, eps;
    int d;
    float *sum, *y;
    int8_t *yq, *yl;
    float* ys;
};

// Values i .. i + 3 of a row of d (zeros past its end).
template <bool VEC>
__device__ __forceinline__ void load4(const float* p, int i, int d, float (&v)[4]) {
    if (VEC) {
        const float4 f = i < d ? *reinterpret_cast<const float4*>(p + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = i + e < d ? p[i + e] : 0.f;
    }
}

template <bool VEC>
__device__ __forceinline__ void store4(float* p, int i, int d, const float (&v)[4]) {
    if (VEC) {
        if (i < d) *reinterpret_cast<float4*>(p + i) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < d) p[i + e] = v[e];
    }
}

// A running sum of squares in a pair: the product's and the sum's errors go to the low part.
__device__ __forceinline__ void add_square(F2& s, float x) {
    const F2 p = f2_two_prod(x, x);
    const F2 t = f2_two_sum(s.hi, p.hi);
    s.hi = t.hi;
    s.lo += t.lo + p.lo;
}

// The CTA's sum of s, in every thread and in one order (`red` is used once a kernel).
template <int T>
__device__ __forceinline__ F2 block_sum(F2 s, F2* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s = f2_add(s, F2{__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    s = lane < T / 32 ? red[lane] : F2{0.f, 0.f};
#pragma unroll
    for (int o = T / 64; o > 0; o >>= 1)
        s = f2_add(s, F2{__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
    return F2{__shfl_sync(0xffffffffu, s.hi, 0), __shfl_sync(0xffffffffu, s.lo, 0)};
}

// 1 / sqrt(sum / d + eps) as a pair (the quotient's remainder by FMA).
__device__ __forceinline__ F2 norm_factor(F2 sum, int d, float eps) {
    const float df = (float)d;
    const float qh = sum.hi / df;
    const float ql = (fmaf(-qh, df, sum.hi) + sum.lo) / df;
    return f2_rsqrt(f2_add(f2_quick(qh, ql), F2{eps, 0.f}));
}

__device__ __forceinline__ F2 f2_scale(F2 a, float b) {
    const F2 p = f2_two_prod(a.hi, b);
    return F2{p.hi, fmaf(a.lo, b, p.lo)};
}

// T threads a row, PER vectors of four values each; a thread's 32-value block is eight lanes.
template <int T, int PER, bool VEC>
__global__ void __launch_bounds__(T) postnorm_kernel(const PostnormParams p) {
    __shared__ F2 red[2][32];
    const int d = p.d, t = threadIdx.x;
    const int64_t row = blockIdx.x, at = row * d;
    griddep_wait();  // (launches overlap up to here: nothing is read before the launch before has ended)
    griddep_launch();
    float a[PER][4], b[PER][4];
#pragma unroll
    for (int j = 0; j < PER; ++j) load4<VEC>(p.b + at, 4 * (j * T + t), d, b[j]);
#pragma unroll
    for (int j = 0; j < PER; ++j) load4<VEC>(p.a + at, 4 * (j * T + t), d, a[j]);
    F2 factor = {p.scale, 0.f};  // what a row's values share: scale, 1 / rms and a row's gate
    if (p.w_post) {
        F2 ss = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < PER; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) add_square(ss, b[j][e]);
        factor = f2_scale(norm_factor(block_sum<T>(ss, red[0]), d, p.eps), p.scale);
    }
    const bool gates = p.gate && p.gate_col != 0;
    const float* gate = p.gate + row * p.gate_row;
    if (p.gate && !gates) factor = f2_scale(factor, *gate);
    F2 ss = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = 4 * (j * T + t);
        float w[4] = {1.f, 1.f, 1.f, 1.f}, g[4] = {1.f, 1.f, 1.f, 1.f};
        if (p.w_post) load4<VEC>(p.w_post, i, d, w);
        if (gates) {
            if (p.gate_col == 1) {
                load4<VEC>(gate, i, d, g);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) g[e] = i + e < d ? gate[(i + e) * p.gate_col] : 0.f;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const F2 q = f2_two_prod(b[j][e], w[e]);
            F2 z = f2_two_prod(q.hi, factor.hi);
            z.lo += fmaf(q.hi, factor.lo, q.lo * factor.hi);
            if (gates) z = f2_scale(z, g[e]);
            const F2 s = f2_two_sum(a[j][e], z.hi);
            a[j][e] = isfinite(s.hi) ? s.hi + (s.lo + z.lo) : s.hi;  // (an infinity's error terms are no numbers)
            if (i + e < d) add_square(ss, a[j][e]);
        }
        if (p.sum) store4<VEC>(p.sum + at, i, d, a[j]);
    }
    if (!p.y && !p.yq) return;
    const F2 inv = norm_factor(block_sum<T>(ss, red[1]), d, p.eps);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = 4 * (j * T + t);
        float w[4], y[4];
        load4<VEC>(p.w_pre, i, d, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = i + e < d ? f2_mul3_round(a[j][e], w[e], inv) : 0.f;
        if (p.y) store4<VEC>(p.y + at, i, d, y);
        if (!p.yq) continue;
        float m = fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3])));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float dq = div127(m);
        float q[4];
        uint32_t hi = 0, lo = 0;
        bool near = p.yl != nullptr;  // (the low word turns on the quotient's last bits: always the IEEE one)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            q[e] = __fdividef(y[e], dq);
            near |= quotient_near_tie(q[e], dq);
        }
        if (__any_sync(0xffffffffu, near)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) q[e] = __fdiv_rn(y[e], dq);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float r = fminf(fmaxf(roundf(q[e]), -127.f), 127.f);
            const float f = fminf(fmaxf(roundf(__fmul_rn(__fsub_rn(q[e], r), 128.f)), -127.f), 127.f);
            hi |= (uint32_t)(uint8_t)(int8_t)(int)r << (8 * e);
            lo |= (uint32_t)(uint8_t)(int8_t)(int)f << (8 * e);
        }
        if (i >= d) continue;
        *reinterpret_cast<uint32_t*>(p.yq + at + i) = dq == 0.f ? 0u : hi;
        if (p.yl) *reinterpret_cast<uint32_t*>(p.yl + at + i) = dq == 0.f ? 0u : lo;
        if ((t & 7) == 0) p.ys[(at + i) >> 5] = dq;
    }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace

cudaError_t launch_postnorm(const PostnormCall& c, cudaStream_t st) {
    const PostnormParams p = {c.a, c.b, c.w_post, c.w_pre, c.gate, c.gate_row, c.gate_col, c.scale, c.eps, (int)c.d,
                              c.sum, c.y, c.yq, c.yl, c.ys};
    bool vec = c.d % 4 == 0 && (c.gate_col != 1 || c.gate_row % 4 == 0);
    for (const void* q : {(const void*)c.a, (const void*)c.b, (const void*)c.w_post, (const void*)c.w_pre, (const void*)c.sum,
                          (const void*)c.y, c.gate_col == 1 ? (const void*)c.gate : nullptr})
        vec = vec && aligned16(q);
    const dim3 grid((unsigned)c.rows);
    if (!vec) return launch(postnorm_kernel<512, 8, false>, grid, dim3(512), 0, st, 1, p);
    // A row's time is its chain of reductions: up to a row an SM as many threads as it has vectors; with more, the CTAs of an SM
    // hide one another's chains and 256 threads of several vectors spend less on the reductions.  Measured, us, rows of 2048: 152
    // rows 3.5 and 3.9, 304 rows 5.0 and 4.7, 4096 rows 51 and 38; of 4096: 64 rows 5.2 and 6.0, 304 rows 8.7 and 7.3.
    const int n4 = (int)((c.d + 3) / 4);
    const bool many = c.rows > device_info().sms;
#define Q8_POSTNORM(T, PER) \
    if (n4 <= (T) * (PER)) return launch(postnorm_kernel<T, PER, true>, grid, dim3(T), 0, st, 1, p);
    if (many) {
        Q8_POSTNORM(128, 1)
        Q8_POSTNORM(256, 1)
        Q8_POSTNORM(256, 2)
        Q8_POSTNORM(256, 4)
        Q8_POSTNORM(256, 8)
        Q8_POSTNORM(512, 8)
    }
    Q8_POSTNORM(128, 1)
    Q8_POSTNORM(256, 1)
    Q8_POSTNORM(512, 1)
    Q8_POSTNORM(1024, 1)
    Q8_POSTNORM(1024, 2)
    Q8_POSTNORM(1024, 4)
#undef Q8_POSTNORM
    return cudaErrorInvalidValue;
}

}  // namespace q8
