// What the two kernels of the paged attention share: the call as they read it, and the division of a batch's work over
// the CTAs of one launch.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "kv_pages.cuh"
#include "stream.cuh"

namespace q8 {

// A key/value head's query vectors of one sequence are its rows' heads of the group, vector m = row * group + head.  A
// kernel takes them in tiles, and a tile's positions in units; one (sequence, key/value head, tile) is an item.
struct PagedParams {
    KvView view;
    int heads = 0, group = 0;       // query heads, and query heads a key/value head
    const float* q = nullptr;
    int64_t q_stride = 0, out_stride = 0;
    float scale = 0.f;              // times log2(e): scores are kept in the base-2 logarithm
    float* out = nullptr;
    float* lse = nullptr;
    int64_t above = 0, upto = 0;    // the sequences taken: above < vectors a key/value head <= upto
    float* part = nullptr;          // partial results: two slots a CTA
    int* counters = nullptr;        // one a CTA, zero between launches
    int* failed = nullptr;          // the workspace's failure word: a launch that finds it set does nothing
    unsigned polls = 0;             // of a wait, before it gives up
    unsigned missing = 0;           // bytes that the copies are waited for beyond what they bring (the self-test's)
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a / b for a, b >= 0, in 32 bits where both fit (a 64-bit division is about a hundred instructions, kept out of line).
static __device__ __noinline__ int64_t div_large(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t div_small(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : div_large(a, b);
}

// The launch's units in one line, sequence by sequence, cut into equal runs: CTA c takes units c*T/C .. (c+1)*T/C - 1 of
// T, so ragged batches load every SM alike, whatever the device arrays hold when the launch runs.  An item's first units
// stand for what its start and end cost and are nobody's work; the others are its tiles of positions.  C is the launch's
// CTAs, or T when there are fewer units (the other CTAs leave), so every CTA below C has a unit.
struct PagedRun {
    int64_t total = 0, lo = 0, hi = 0;
    int ctas = 0;
    int seq = 0;          // the sequence of unit lo
    int64_t seq_at = 0;   // its first unit
    __device__ int64_t start(int64_t c) const { return div_small(c * total, ctas); }
    __device__ int owner(int64_t unit) const { return (int)div_small((unit + 1) * ctas - 1, total); }
};

// Forms the run; `units(s)` is a sequence's unit count (0: not this kernel's).  Every thread of the CTA calls it.  Each
// thread sums a run of sequences, the CTA scans the sums, and the thread whose sequences hold unit lo finds it.
template <int THREADS, typename Units>
__device__ __forceinline__ PagedRun paged_run(const PagedParams& pk, Units units) {
    __shared__ int64_t warp_sum[THREADS / 32];
    __shared__ int64_t found_at;
    __shared__ int found, failed;
    const KvView& kv = pk.view;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int was_failed = t == 0 ? *(volatile int*)pk.failed : 0;
    const int each = (kv.seqs + THREADS - 1) / THREADS;
    const int b0 = min(kv.seqs, t * each), b1 = min(kv.seqs, b0 + each);
    int64_t sum = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        const KvSeq s = kv_seq(kv, b);
        if (blockIdx.x == 0 && (!s.rows_ok || (s.n > 0 && !s.len_ok))) kv_flag(kv, Q8_KV_ERR_LENGTH);
        sum += units(s);
    }
    int64_t pre = sum;  // inclusive scan
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += up;
    }
    if (lane == 31) warp_sum[w] = pre;
    if (t == 0) {
        found = 0, found_at = 0, failed = was_failed;
        if (was_failed && blockIdx.x == 0) kv_flag(kv, Q8_KV_ERR_WAIT);
    }
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll 1
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < w) before += warp_sum[i];
        total += warp_sum[i];
    }
    PagedRun r;
    if (failed) total = 0;  // (a workspace whose counters may not be zero)
    r.total = total;
    r.ctas = (int)(total < gridDim.x ? total : gridDim.x);
    if (r.ctas > 0 && (int)blockIdx.x < r.ctas) {
        r.lo = r.start(blockIdx.x);
        r.hi = r.start(blockIdx.x + 1);
        int64_t at = before + pre - sum;
        if (at <= r.lo && r.lo < at + sum) {
#pragma unroll 1
            for (int b = b0; b < b1; ++b) {
                const int64_t n = units(kv_seq(kv, b));
                if (r.lo < at + n) {
                    found = b;
                    found_at = at;
                    break;
                }
                at += n;
            }
        }
    }
    __syncthreads();
    r.seq = found;
    r.seq_at = found_at;
    return r;
}

// The slot of the partial results where CTA c leaves its piece of an item: its first when its run begins in the item.
// (Only the item's first CTA, c0, may have a run that begins before it.)
__device__ __forceinline__ int paged_slot(int c, int c0, bool c0_opens) { return 2 * c + (c == c0 && !c0_opens ? 1 : 0); }

// Whether a sequence is one of this launch's.
__device__ __forceinline__ bool paged_takes(const PagedParams& pk, const KvSeq& s) {
    const int64_t vectors = s.n * pk.group;
    return s.rows_ok && s.n > 0 && vectors > pk.above && vectors <= pk.upto;
}

// ---- the pages' words by tensor copies -----------------------------------------------------------------------------
// A map of words [pages][kv * page_size][hd], read 16 rows of a page at a time with the 128- or 64-byte swizzle
// (paged_attn_tc.cu); false where the driver has no encoder.
bool paged_words_map(CUtensorMap* m, const void* words, const KvView& v, int hd);

// A tensor copy of one page's 16 rows from `row` of its [heads * page_size] rows into shared memory (zeros for a page out
// of range), counted on bar's transaction bytes.
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int row, int page, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(smem_addr(dst)), "l"(map), "r"(0), "r"(row), "r"(page), "r"(smem_addr(bar))
                 : "memory");
}

constexpr unsigned PA_POLL_NS = 20000;   // the longest the hardware may hold a warp at a poll
constexpr unsigned PA_POLLS = 1u << 20;  // polls before a wait gives up (seconds)
constexpr unsigned PA_DRAIN = 1u << 10;  // polls of a wait for what is in flight when a CTA leaves (many times its latency)

// One poll of a barrier's phase; the hardware may hold the warp for up to PA_POLL_NS, issuing nothing meanwhile (polls
// that return at once took about half of the SM's issue slots).
__device__ __forceinline__ bool try_wait(uint64_t* bar, unsigned parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(smem_addr(bar)), "r"(parity), "r"(PA_POLL_NS)
                 : "memory");
    return ok != 0;
}

// Waits for a phase, whatever else has given up.
__device__ __forceinline__ void drain(uint64_t* bar, unsigned parity) {
#pragma unroll 1
    for (unsigned i = 0; i < PA_DRAIN && !try_wait(bar, parity); ++i) {}
}

// What a wait that gave up leaves behind, whether the caller has an error word or not: later launches on this workspace do
// nothing (an item that several CTAs share may have been left part-way) until q8_workspace_check has cleared it.
// (One thread calls it as the CTA leaves: in every wait it would be code beside the loops that have to stay in the
// instruction cache, 2309 us for 2057 over 32768 positions.)
__device__ __forceinline__ void wait_gave_up(const PagedParams& pk) {
    kv_flag(pk.view, Q8_KV_ERR_WAIT);
    atomicOr(pk.failed, 1);
}

// ---- words and parts -------------------------------------------------------------------------------------------------
// Bytes 0 and 1 (HALF 1: 2 and 3) of w, flipped by words_flip, as two f16 values (exact).
template <int WORDS, int HALF>
__device__ __forceinline__ uint32_t words2_f16(uint32_t w) {
    if (WORDS == Q8_KV_INT8) {
        // byte + 128 in the low mantissa byte of 1024.0, less 1152: exact
        const uint32_t u = __byte_perm(w, 0x64646464u, HALF ? 0x4342 : 0x4140);
        const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6480)));
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    return e4m3x2_to_f16x2((uint16_t)(HALF ? w >> 16 : w & 0xffffu));
}

template <int WORDS>
__device__ __forceinline__ uint32_t words_flip(uint32_t w) {
    return WORDS == Q8_KV_INT8 ? w ^ 0x80808080u : w;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }  // e in [-126, 127]

// The unbiased exponent of a non-negative float's bits, at least -100 (so that scalings by its inverse and by 2^14 stay
// finite); infinities and NaN: 0 (whatever they scale stays not finite).
__device__ __forceinline__ int exponent_of(unsigned bits) {
    return bits >= 0x7f800000u ? 0 : max((int)(bits >> 23) - 127, -100);
}

// The magnitude's bits of a value scale, or 0 where it is not finite: such a row makes a number of no sum that it enters, and
// must not decide how the others are scaled, which are read by rows that do not see it.
__device__ __forceinline__ unsigned finite_bits(float x) {
    const unsigned b = __float_as_uint(x) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0u;
}

// Weights are scaled by the largest value scale of the positions taken together, and split into two f16 parts.  A row of which
// the mask hides that one, and which sees none within 2^PA_SPREAD of it, scales its own weights up further, so that what it
// does not see, up to 2^100 times what it does, costs it no bits.  (Within that spread its weights of 1 lie at 2^6 or above,
// and an f16 part resolves 2^-24.)
constexpr int PA_SPREAD = 8;

cudaError_t launch_paged_rows(const PagedParams& p, int hd, int words, int tiles, cudaStream_t st);
int paged_rows_ctas(int tiles);   // the launch's CTAs
size_t paged_rows_slot(int hd);   // bytes of one partial result
cudaError_t launch_paged_tiles(const PagedParams& p, int hd, int words, cudaStream_t st);
size_t paged_tiles_slot(int hd);

}  // namespace q8
