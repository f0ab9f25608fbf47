// The paged, quantized key/value cache: writing a batch's new rows (per-head RMSNorm and rotation of queries and keys, and
// the keys and values quantized into their page slots, in one pass), and reading rows back.
//
// What it computes: qwen_emit docs, emit_qwen30b_generate (per-head QK-norm, then RoPE on pairs (i, i + head_dim/2), then
// the key/value append), for ragged batches over pages of 8-bit words (q8moe.h, q8_kv_pages).
//
// How: both are streams, with floors set by the bytes of the f32 rows (a row of 32 + 4 + 4 heads of 128 is 20 KiB in and 16 KiB of
// queries and 1 KiB of words out).  A warp takes one row's group of head vectors; LPV lanes hold a vector, each lane two
// float4 (dims 4l.. of either half), so both elements of every rotation pair sit in one lane and the row's sums are
// shuffles among LPV lanes.  All of a warp's loads are issued before the row's sequence and page are looked up (a chain
// of three dependent loads), which hides that chain behind them.  Measured: 2318 rows of 24 + 8 + 8 heads of 128 in 24.3 us
// (3.4 TB/s at 60% of the issue slots: all keys are turned in pairs of f32, though the words next to a border alone need it), 34182 rows of 8 heads of 64 read back
// in 32.7 us (5.4 TB/s, the memory's: a copy runs at 6.8).
#include <cuda_fp16.h>

#include "common.cuh"
#include "kv_pages.cuh"

namespace q8 {

namespace {

constexpr int KV_ITERS = 4;  // vectors a lane group of the writing kernel holds: 8 float4 loads in flight a lane
constexpr int KV_READ = 2;   // and of the reading one

struct AppendParams {
    KvView view;
    int heads, groups;  // query heads; warps a row
    const float *q, *k, *v;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    const float *q_norm, *k_norm;
    float eps;
    const float *cos_t, *sin_t;
    int64_t rope_positions;
    float* q_out;
};

// The int8 words of 4 values with the scale d > 0, packed: the IEEE quotients rounded halves away from zero and clamped.
__device__ __forceinline__ uint32_t kv_words4_exact(const float* x, float d) {
    uint32_t u = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u |= ((uint32_t)(int)fminf(fmaxf(roundf(__fdiv_rn(x[i], d)), -127.f), 127.f) & 0xffu) << (8 * i);
    return u;
}

// The words of 8 values with the scale d > 0: rounded halves away from zero (int8) or to nearest even (e4m3).  An int8 word
// needs only the integer that the quotient rounds to: x times the approximate inverse is within 5e-5 of the quotient (of at
// most 127), so it rounds to the same one unless it lies within 1e-4 of a half; there, and where d is so small that its
// inverse is not normal, the IEEE quotients decide (half of the instructions of dividing always).
template <int WORDS>
__device__ __forceinline__ uint2 kv_words8(const float (&x)[8], float d) {
    uint32_t w[2];
    if (WORDS == Q8_KV_INT8) {
        const float inv = __fdividef(1.f, d);
        bool near = !(d >= 1e-30f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t u = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = x[4 * h + i], a = fmaf(fabsf(v), inv, 0.5f), k = floorf(a);
                near |= fabsf((a - k) - 0.5f) > 0.4999f;
                u |= ((uint32_t)(int)copysignf(k, v) & 0xffu) << (8 * i);
            }
            w[h] = u;
        }
        if (near) w[0] = kv_words4_exact(x, d), w[1] = kv_words4_exact(x + 4, d);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float t[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] = __fdiv_rn(x[4 * h + i], d);
            uint16_t a, b;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(t[1]), "f"(t[0]));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(t[3]), "f"(t[2]));
            w[h] = (uint32_t)a | ((uint32_t)b << 16);
        }
    }
    return make_uint2(w[0], w[1]);
}

template <int LPV>
__device__ __forceinline__ F2 f2_group_sum(F2 v) {
#pragma unroll
    for (int o = LPV / 2; o > 0; o >>= 1)
        v = f2_add(v, F2{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
    return v;
}

// f32((a * wa * ca + b * wb * cb) * inv), every step but the rounding at the end to about 2^-44.
__device__ __forceinline__ float f2_turn(float a, float wa, float ca, float b, float wb, float cb, F2 inv) {
    const F2 pa = f2_two_prod(a, wa), pb = f2_two_prod(b, wb);
    F2 ta = f2_two_prod(pa.hi, ca), tb = f2_two_prod(pb.hi, cb);
    ta.lo = fmaf(pa.lo, ca, ta.lo);
    tb.lo = fmaf(pb.lo, cb, tb.lo);
    const F2 s = f2_add(ta, tb);
    const F2 y = f2_two_prod(s.hi, inv.hi);
    return y.hi + (y.lo + fmaf(s.hi, inv.lo, s.lo * inv.hi));
}

template <int HD, int WORDS>
__global__ void __launch_bounds__(256, 4) kv_append_kernel(const AppendParams pk) {
    constexpr int LPV = HD / 8, VPW = 32 / LPV, HALF = HD / 2;
    const KvView& kv = pk.view;
    const int lane = threadIdx.x & 31, sub = lane / LPV, l = lane % LPV;
    const int64_t warp = (int64_t)blockIdx.x * Q8_WARPS + (threadIdx.x >> 5);
    const int64_t r = warp / pk.groups;
    if (kv.error && blockIdx.x == gridDim.x - 1) return kv_check(kv);
    if (r >= kv.rows) return;
    // A row's warps take its vectors in turn, so that each has its share of the keys and values, whose words cost several
    // times a query's work (a warp of keys alone held its CTA: with the rounding above, 2318 rows of 24 + 8 + 8 heads went from
    // 35.8 to 25.0 us; four CTAs an SM, by 64 registers for 76, to 23.9, now 24.3).
    const int v0 = (int)(warp % pk.groups) * VPW + sub, step = pk.groups * VPW, nvec = pk.heads + 2 * kv.kv;
    float x[KV_ITERS][8];
#pragma unroll
    for (int it = 0; it < KV_ITERS; ++it) {
        const int vec = v0 + it * step;
        const float* src = nullptr;
        if (vec < pk.heads) src = pk.q + r * pk.q_stride + (int64_t)vec * HD;
        else if (vec < pk.heads + kv.kv) src = pk.k + r * pk.k_stride + (int64_t)(vec - pk.heads) * HD;
        else if (vec < nvec) src = pk.v + r * pk.v_stride + (int64_t)(vec - pk.heads - kv.kv) * HD;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (src) {
            a = *reinterpret_cast<const float4*>(src + 4 * l);
            b = *reinterpret_cast<const float4*>(src + HALF + 4 * l);
        }
        x[it][0] = a.x, x[it][1] = a.y, x[it][2] = a.z, x[it][3] = a.w;
        x[it][4] = b.x, x[it][5] = b.y, x[it][6] = b.z, x[it][7] = b.w;
    }
    const int b = kv_find_seq(kv, r);
    if (b < 0) return;
    const KvSeq s = kv_seq(kv, b);
    if (!s.holds(r)) return;
    const int pos = (int)(s.len - s.n + (r - s.first));
    float c[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (pk.cos_t) {
        if (pos >= pk.rope_positions) {
            if (lane == 0) kv_flag(kv, Q8_KV_ERR_ROPE);
            return;
        }
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(pk.cos_t + (int64_t)pos * HALF) + l);
        const float4 s4 = __ldg(reinterpret_cast<const float4*>(pk.sin_t + (int64_t)pos * HALF) + l);
        c[0] = c4.x, c[1] = c4.y, c[2] = c4.z, c[3] = c4.w;
        sn[0] = s4.x, sn[1] = s4.y, sn[2] = s4.z, sn[3] = s4.w;
    }
    const int page = kv_page(kv, b, pos);
    if (page < 0 && lane == 0) kv_flag(kv, Q8_KV_ERR_PAGE);
#pragma unroll
    for (int it = 0; it < KV_ITERS; ++it) {
        const int vec = v0 + it * step;
        const int first = vec - sub;  // the iteration's first vector: the warp's branches go by it
        if (first >= nvec) break;
        if (first < pk.heads) {  // queries, in f32 (their last bits decide no word)
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[it][i], x[it][i], ss);
            ss = group_sum<LPV>(ss);
            const float inv = pk.q_norm ? rsqrtf(ss / (float)HD + pk.eps) : 1.0f;
            if (vec < pk.heads) {
                float z[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a = x[it][i], d = x[it][4 + i];
                    if (pk.q_norm) {
                        a *= inv * __ldg(pk.q_norm + 4 * l + i);
                        d *= inv * __ldg(pk.q_norm + HALF + 4 * l + i);
                    }
                    z[i] = a * c[i] - d * sn[i];
                    z[4 + i] = a * sn[i] + d * c[i];
                }
                float* dst = pk.q_out + r * pk.q_out_stride + (int64_t)vec * HD;
                *reinterpret_cast<float4*>(dst + 4 * l) = make_float4(z[0], z[1], z[2], z[3]);
                *reinterpret_cast<float4*>(dst + HALF + 4 * l) = make_float4(z[4], z[5], z[6], z[7]);
            }
        }
        if (first + VPW <= pk.heads) continue;
        const bool key = vec >= pk.heads && vec < pk.heads + kv.kv;
        if (first < pk.heads + kv.kv) {  // keys: the norm and the rotation as pairs of f32, rounded once
            F2 ss = F2{0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = f2_add(ss, f2_two_prod(x[it][i], x[it][i]));
            ss = f2_group_sum<LPV>(ss);
            if (key) {
                F2 inv = F2{1.f, 0.f};
                if (pk.k_norm) inv = f2_rsqrt(f2_add(F2{ss.hi / HD, ss.lo / HD}, F2{pk.eps, 0.f}));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = x[it][i], d = x[it][4 + i];
                    float wa = 1.f, wd = 1.f;
                    if (pk.k_norm) wa = __ldg(pk.k_norm + 4 * l + i), wd = __ldg(pk.k_norm + HALF + 4 * l + i);
                    x[it][i] = f2_turn(a, wa, c[i], d, wd, -sn[i], inv);
                    x[it][4 + i] = f2_turn(a, wa, sn[i], d, wd, c[i], inv);
                }
            }
        }
        // the row's largest magnitude, as bits (an infinity's or a NaN's lie above every finite value's)
        unsigned m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[it][i]) & 0x7fffffffu);
#pragma unroll
        for (int o = LPV / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (vec < pk.heads || vec >= nvec || page < 0) continue;
        const bool finite = m < 0x7f800000u;
        float d = __uint_as_float(0x7fc00000u);
        if (finite) d = WORDS == Q8_KV_INT8 ? div127(__uint_as_float(m)) : __fdiv_rn(__uint_as_float(m), 448.f);
        const uint2 w = finite && d > 0.f ? kv_words8<WORDS>(x[it], d) : make_uint2(0u, 0u);
        const int64_t row = kv_row(kv, page, key ? vec - pk.heads : vec - pk.heads - kv.kv, pos);
        int8_t* dst = (key ? kv.k : kv.v) + row * HD;
        *reinterpret_cast<uint32_t*>(dst + 4 * l) = w.x;
        *reinterpret_cast<uint32_t*>(dst + HALF + 4 * l) = w.y;
        if (l == 0) (key ? kv.ks : kv.vs)[row] = d;
    }
}

struct ReadParams {
    KvView view;
    int groups;  // warps a row
    float *k_out, *v_out;
    int64_t row_stride, head_stride;
};

__device__ __forceinline__ void store8(float* p, const float (&y)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]),
                 "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7])
                 : "memory");
}

// LPV lanes a vector, a lane 8 words (8 bytes in, 32 bytes out), a warp a group of one row's vectors, all of its loads in
// flight together.  Many warps hide the chain sequence, page, words best: 38912 rows of 4 heads of 128 take 36.4 us in int8
// words and 33.4 in e4m3 (4096 rows 5.5 and 5.4) with two vectors a lane group, 39.7 and 33.0 (5.7 and 5.5) with four, and
// 54 and 35 (10.2 and 6.5) with four rows a warp.
template <int HD, int WORDS>
__global__ void __launch_bounds__(256) kv_read_kernel(const ReadParams pk) {
    constexpr int LPV = HD / 8, VPW = 32 / LPV;
    const KvView& kv = pk.view;
    const int lane = threadIdx.x & 31, sub = lane / LPV, l = lane % LPV;
    const int64_t warp = (int64_t)blockIdx.x * Q8_WARPS + (threadIdx.x >> 5);
    const int64_t r = warp / pk.groups;
    if (kv.error && blockIdx.x == gridDim.x - 1) return kv_check(kv);
    if (r >= kv.rows) return;
    const int v0 = (int)(warp % pk.groups) * (KV_READ * VPW) + sub;
    const int b = kv_find_seq(kv, r);
    if (b < 0) return;
    const KvSeq s = kv_seq(kv, b);
    if (!s.holds(r)) return;
    const int pos = (int)(s.len - s.n + (r - s.first));
    const int page = kv_page(kv, b, pos);
    if (page < 0) {
        if (lane == 0) kv_flag(kv, Q8_KV_ERR_PAGE);
        return;
    }
    uint2 w[KV_READ];
    float d[KV_READ];
#pragma unroll
    for (int it = 0; it < KV_READ; ++it) {
        const int vec = v0 + it * VPW;
        if (vec < 2 * kv.kv) {
            const bool key = vec < kv.kv;
            const int64_t row = kv_row(kv, page, key ? vec : vec - kv.kv, pos);
            w[it] = *reinterpret_cast<const uint2*>((key ? kv.k : kv.v) + row * HD + 8 * l);
            d[it] = (key ? kv.ks : kv.vs)[row];
        }
    }
#pragma unroll
    for (int it = 0; it < KV_READ; ++it) {
        const int vec = v0 + it * VPW;
        float* out = vec < kv.kv ? pk.k_out : pk.v_out;
        if (vec >= 2 * kv.kv || !out) continue;
        float y[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t u = h ? w[it].y : w[it].x;
            if (WORDS == Q8_KV_INT8) {
                const uint32_t f = u ^ 0x80808080u;
                y[4 * h] = i8_to_f32<0>(f), y[4 * h + 1] = i8_to_f32<1>(f);
                y[4 * h + 2] = i8_to_f32<2>(f), y[4 * h + 3] = i8_to_f32<3>(f);
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t h2 = e4m3x2_to_f16x2((uint16_t)(u >> (16 * j)));
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                    y[4 * h + 2 * j] = f.x, y[4 * h + 2 * j + 1] = f.y;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= d[it];
        store8(out + r * pk.row_stride + (vec < kv.kv ? vec : vec - kv.kv) * pk.head_stride + 8 * l, y);
    }
}

// Warps a row for `vectors` head vectors of hd values, `held` a lane group, and the CTAs of the view's rows (and the one that
// checks the batch).
int warps_a_row(int vectors, int hd, int held) {
    const int each = held * (32 / (hd / 8));
    return (vectors + each - 1) / each;
}

unsigned ctas(const KvView& v, int groups) {
    return (unsigned)(((int64_t)v.rows * groups + Q8_WARPS - 1) / Q8_WARPS) + (v.error ? 1 : 0);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendCall& c, cudaStream_t st) {
    AppendParams p;
    p.view = c.view;
    p.heads = c.heads;
    p.groups = warps_a_row(c.heads + 2 * c.view.kv, c.hd, KV_ITERS);
    p.q = c.q, p.k = c.k, p.v = c.v;
    p.q_stride = c.q_stride, p.k_stride = c.k_stride, p.v_stride = c.v_stride, p.q_out_stride = c.q_out_stride;
    p.q_norm = c.q_norm, p.k_norm = c.k_norm;
    p.eps = c.eps;
    p.cos_t = c.cos_t, p.sin_t = c.sin_t;
    p.rope_positions = c.rope_positions;
    p.q_out = c.q_out;
    const unsigned grid = ctas(c.view, p.groups);
    if (c.hd == 128 && c.words == Q8_KV_INT8) kv_append_kernel<128, Q8_KV_INT8><<<grid, Q8_THREADS, 0, st>>>(p);
    else if (c.hd == 128) kv_append_kernel<128, Q8_KV_E4M3><<<grid, Q8_THREADS, 0, st>>>(p);
    else if (c.words == Q8_KV_INT8) kv_append_kernel<64, Q8_KV_INT8><<<grid, Q8_THREADS, 0, st>>>(p);
    else kv_append_kernel<64, Q8_KV_E4M3><<<grid, Q8_THREADS, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvReadCall& c, cudaStream_t st) {
    ReadParams p;
    p.view = c.view;
    p.groups = warps_a_row(2 * c.view.kv, c.hd, KV_READ);
    p.k_out = c.k_out, p.v_out = c.v_out;
    p.row_stride = c.row_stride, p.head_stride = c.head_stride;
    const unsigned grid = ctas(c.view, p.groups);
    if (c.hd == 128 && c.words == Q8_KV_INT8) kv_read_kernel<128, Q8_KV_INT8><<<grid, Q8_THREADS, 0, st>>>(p);
    else if (c.hd == 128) kv_read_kernel<128, Q8_KV_E4M3><<<grid, Q8_THREADS, 0, st>>>(p);
    else if (c.words == Q8_KV_INT8) kv_read_kernel<64, Q8_KV_INT8><<<grid, Q8_THREADS, 0, st>>>(p);
    else kv_read_kernel<64, Q8_KV_E4M3><<<grid, Q8_THREADS, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace q8
