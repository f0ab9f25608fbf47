// Causal attention of a ragged batch's rows over pages of 8-bit key and value words (q8moe.h, q8_paged_attention).
//
// A CTA a (row, head): its warps take the row's positions in turn, a lane HD/32 dimensions, with a running maximum and
// sum of the softmax each; the warps' results meet in shared memory.
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include "common.cuh"
#include "kv_pages.cuh"

namespace q8 {

namespace {

struct PagedParams {
    KvView view;
    int heads;
    const float* q;
    int64_t q_stride, out_stride;
    float scale;
    float* out;
    float* lse;
};

template <int WORDS>
__device__ __forceinline__ float word_value(const int8_t* p) {
    if (WORDS == Q8_KV_INT8) return (float)*p;
    const uint32_t h = e4m3x2_to_f16x2((uint16_t) * reinterpret_cast<const uint8_t*>(p));
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

template <int HD, int WORDS>
__global__ void __launch_bounds__(Q8_THREADS) paged_attention_kernel(const PagedParams pk) {
    constexpr int DPL = HD / 32;
    __shared__ float sm[Q8_WARPS], sl[Q8_WARPS], so[Q8_WARPS][HD];
    const KvView& kv = pk.view;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, h = blockIdx.y;
    const int64_t r = blockIdx.x;
    const int g = h / (pk.heads / kv.kv);
    const int b = kv_find_seq(kv, r);
    if (b < 0) return;
    const KvSeq s = kv_seq(kv, b);
    if ((!s.rows_ok || !s.len_ok) && threadIdx.x == 0) kv_flag(kv, Q8_KV_ERR_LENGTH);
    if (!s.rows_ok) return;
    const int end = s.len_ok ? (int)(s.len - s.n + (r - s.first)) + 1 : 0;  // positions the row attends
    float q[DPL], o[DPL], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < DPL; ++i) {
        q[i] = pk.q[r * pk.q_stride + (int64_t)h * HD + lane + 32 * i] * pk.scale;
        o[i] = 0.f;
    }
    for (int p = w; p < end; p += Q8_WARPS) {
        const int page = kv_page(kv, b, p);
        if (page < 0) {
            if (lane == 0) kv_flag(kv, Q8_KV_ERR_PAGE);
            continue;
        }
        const int64_t row = kv_row(kv, page, g, p);
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < DPL; ++i) d = fmaf(q[i], word_value<WORDS>(kv.k + row * HD + lane + 32 * i), d);
        const float sc = group_sum<32>(d) * kv.ks[row];
        const float mn = fmaxf(m, sc), a = m == -INFINITY ? 0.f : expf(m - mn), e = expf(sc - mn);
        l = l * a + e;
#pragma unroll
        for (int i = 0; i < DPL; ++i) o[i] = o[i] * a + e * kv.vs[row] * word_value<WORDS>(kv.v + row * HD + lane + 32 * i);
        m = mn;
    }
    if (lane == 0) sm[w] = m, sl[w] = l;
#pragma unroll
    for (int i = 0; i < DPL; ++i) so[w][lane + 32 * i] = o[i];
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int i = 0; i < Q8_WARPS; ++i) M = fmaxf(M, sm[i]);
    for (int i = 0; i < Q8_WARPS; ++i) L += sm[i] == -INFINITY ? 0.f : sl[i] * expf(sm[i] - M);
    for (int d = threadIdx.x; d < HD; d += Q8_THREADS) {
        float acc = 0.f;
        for (int i = 0; i < Q8_WARPS; ++i) acc += sm[i] == -INFINITY ? 0.f : so[i][d] * expf(sm[i] - M);
        pk.out[r * pk.out_stride + (int64_t)h * HD + d] = L == 0.f ? 0.f : acc / L;
    }
    if (threadIdx.x == 0 && pk.lse) pk.lse[r * pk.heads + h] = L == 0.f ? -INFINITY : M + logf(L);
}

}  // namespace

cudaError_t launch_paged_attention(const PagedAttnCall& c, Carve&, cudaStream_t st) {
    PagedParams p;
    p.view = c.view;
    p.heads = c.heads;
    p.q = c.q;
    p.q_stride = c.q_stride, p.out_stride = c.out_stride;
    p.scale = c.scale;
    p.out = c.out;
    p.lse = c.lse;
    const dim3 grid((unsigned)c.view.rows, (unsigned)c.heads);
    if (c.hd == 128 && c.words == Q8_KV_INT8) paged_attention_kernel<128, Q8_KV_INT8><<<grid, Q8_THREADS, 0, st>>>(p);
    else if (c.hd == 128) paged_attention_kernel<128, Q8_KV_E4M3><<<grid, Q8_THREADS, 0, st>>>(p);
    else if (c.words == Q8_KV_INT8) paged_attention_kernel<64, Q8_KV_INT8><<<grid, Q8_THREADS, 0, st>>>(p);
    else paged_attention_kernel<64, Q8_KV_E4M3><<<grid, Q8_THREADS, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace q8
