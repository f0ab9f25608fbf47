// Router scores to experts (q8moe.h, moe_route_scored): scores, groups, the k best, gates, and the grouping by expert.
//
// A warp takes a row: lane L holds experts L, L + 32, ... as order-preserving integer keys.  The K-th largest of the lanes' maxima
// bounds the K-th largest key from below; the keys from there on, a few more than K, are gathered one a lane, and each counts
// those before it.  Scores are formed in f32 by the fast exponential and quotient, whose errors can exchange two experts that
// 64 bits would order: where two of the gathered ones are closer than those errors reach, all of them are formed again in 64
// bits and counted by those; where kept and left groups are, or a softmax with a bias (whose sum all scores share) or more
// candidates than lanes, the whole row is chosen again in 64 bits.  What bounds it is instructions, about 1200 a row of 256
// with eight groups, and where few rows share a warp's SM the rows with near ties, which take microseconds each.  Measured,
// replayed: 15001 rows of 256 experts, 8 of 4 groups' chosen and grouped by expert, 41.6 us (17 MB, 2.5 at the measured copy rate), of
// which the grouping's own launch is a third: its CTAs each read all CTAs' counts.  61 rows 8.5, one row of 128 without a plan
// 2.7.  Taking the largest K times over the lanes took 73 and 30.
#include <math.h>

#include "common.cuh"
#include "ffn4.h"

namespace q8 {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kPlaceThreads = 1024;

struct RouteParams {
    const float* logits;
    int64_t stride;
    int rows, E, K;
    const float* bias;
    int sigmoid, groups, keep, top, renorm;
    float scale;
    int32_t* ids;
    float* gates;
    PlanPtrs plan;
    int32_t* hist;  // [CTAs][E] when a second launch groups the choices
    int* arrived;   // else: the CTAs that are done, zero between calls; the last one groups the choices
    int per;        // rows a CTA (0: rows are dealt out warp by warp)
    const int* failed;  // with a plan: the workspace's word; when it is set `arrived` may not be zero, and nothing is written
};

// f32 -> an unsigned integer of the same order (both zeros alike).
__device__ __forceinline__ unsigned order_key(float x) {
    const unsigned u = __float_as_uint(x + 0.f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(unsigned k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
constexpr unsigned kHidden = 0u, kOff = 1u;  // below every number's key: of another group or taken; out of service

template <typename T>
__device__ __forceinline__ T minus_inf();
template <>
__device__ __forceinline__ float minus_inf<float>() { return -INFINITY; }
template <>
__device__ __forceinline__ double minus_inf<double>() { return -INFINITY; }

// The kept groups as a bit mask, from the marks c [E] of the warp's row in shared memory (-infinity: out of service).
// `close`: whether a kept and a left group are within `tol` of one another.
template <typename T>
__device__ __forceinline__ unsigned kept_groups(const T* c, int S, int groups, int keep, int top, T tol, bool& close) {
    const int lane = threadIdx.x & 31;
    const int lpg_log2 = 31 - __clz(32 / groups), lpg = 1 << lpg_log2;  // lanes a group
    const int g = lane >> lpg_log2;
    const T none = minus_inf<T>();
    T t1 = none, t2 = none;
    if (g < groups)
#pragma unroll 4
        for (int i = lane & (lpg - 1); i < S; i += lpg) {
            const T v = c[g * S + i];
            t2 = max(t2, min(t1, v));
            t1 = max(t1, v);
        }
    for (int o = lpg >> 1; o > 0; o >>= 1) {
        const T o1 = __shfl_xor_sync(FULL, t1, o), o2 = __shfl_xor_sync(FULL, t2, o);
        t2 = max(min(t1, o1), max(t2, o2));
        t1 = max(t1, o1);
    }
    const T sum = top == 2 && t2 > none ? t1 + t2 : t1;
    const T mark = __shfl_sync(FULL, sum, (lane < groups ? lane : 0) << lpg_log2);  // lane j: group j's
    int rank = 0;
    for (int j = 0; j < groups; ++j) {
        const T m = __shfl_sync(FULL, mark, j);
        rank += m > mark || (m == mark && j < lane);
    }
    const bool kept = lane < groups && rank < keep;
    T least = kept ? mark : -none, most = lane < groups && !kept ? mark : none;
    for (int o = 16; o > 0; o >>= 1) {
        least = min(least, __shfl_xor_sync(FULL, least, o));
        most = max(most, __shfl_xor_sync(FULL, most, o));
    }
    close = most > none && !(least - most > tol);
    return __ballot_sync(FULL, kept);
}

// A logit as the rule takes it: what is no number is out of service, +infinity the largest value.
__device__ __forceinline__ float logit_of(float v) { return isnan(v) ? -INFINITY : fminf(v, 3.402823466e38f); }

// The choice of the warp's row in 64 bits: lane j gets the j-th expert, and whether it is in service.  c is scratch, [E] of the
// warp in shared memory.
__device__ __noinline__ void choose_exactly(const RouteParams& p, const float* row, double* c, int& id, bool& on) {
    const int lane = threadIdx.x & 31;
    double m = -INFINITY, z = 0;
    if (!p.sigmoid) {
        for (int e = lane; e < p.E; e += 32) m = max(m, (double)logit_of(row[e]));
        for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(FULL, m, o));
        for (int e = lane; e < p.E; e += 32)
            if (logit_of(row[e]) != -INFINITY) z += exp((double)logit_of(row[e]) - m);
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(FULL, z, o);
    }
    for (int e = lane; e < p.E; e += 32) {
        double v = -INFINITY;
        const float l = logit_of(row[e]);
        if (l != -INFINITY) {
            v = p.sigmoid ? 1 / (1 + exp(-(double)l)) : exp((double)l - m) / z;
            if (p.bias) v += p.bias[e];
            if (isnan(v)) v = -INFINITY;
        }
        c[e] = v;
    }
    __syncwarp();
    unsigned kept = FULL;
    bool close;
    const int S = p.E / p.groups;
    if (p.groups > 1) kept = kept_groups<double>(c, S, p.groups, p.keep, p.top, 0, close);
    __syncwarp();
    // what is out of service goes below every number, what is hidden or taken below that
    for (int e = lane; e < p.E; e += 32) {
        if (p.groups > 1 && !((kept >> (e / S)) & 1u)) c[e] = -INFINITY;
        else if (c[e] == -INFINITY) c[e] = -1.7e308;
        else if (!p.bias) c[e] = logit_of(row[e]);
    }
    __syncwarp();
    for (int j = 0; j < p.K; ++j) {
        double best = -INFINITY;
        int at = p.E;
        for (int e = lane; e < p.E; e += 32)
            if (c[e] > best) best = c[e], at = e;
        for (int o = 16; o > 0; o >>= 1) {
            const double ob = __shfl_xor_sync(FULL, best, o);
            const int oa = __shfl_xor_sync(FULL, at, o);
            if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
        }
        at = min(at, p.E - 1);
        if (lane == j) id = at, on = best > -1.6e308;
        if ((at & 31) == lane) c[at] = -INFINITY;
        __syncwarp();
    }
}

// Adds the CTA's choices [first, first + n) (their experts in ids) to the lists, in ascending order: next[e] is expert e's
// first free place.  wh is [warps][E] of shared memory.  HOLD: ids are held within [0, E) (the last CTA of a launch reads the
// others' ids, which are not there yet should the workspace's counter be in use by another call at the same time).
template <bool HOLD>
__device__ __forceinline__ void place_choices(const int32_t* ids, int first, int n, int E, int* wh, int* next, int32_t* lists) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, W = blockDim.x >> 5;
    const int seg = ((n + W - 1) / W + 31) & ~31;
    const int lo = min(w * seg, n), hi = min(lo + seg, n);
    for (int i = threadIdx.x; i < W * E; i += blockDim.x) wh[i] = 0;
    __syncthreads();
    for (int i = lo + lane; i < hi; i += 32) {
        const unsigned e = __ldcg(ids + first + i);
        atomicAdd(&wh[w * E + (HOLD ? min(e, (unsigned)E - 1) : e)], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int run = next[e];
        for (int v = 0; v < W; ++v) {
            const int n_v = wh[v * E + e];
            wh[v * E + e] = run;
            run += n_v;
        }
    }
    __syncthreads();
    for (int i = lo; i < hi; i += 32) {
        const bool in = i + lane < hi;
        unsigned e = in ? __ldcg(ids + first + i + lane) : E;  // (lanes past the end stand together)
        if (HOLD) e = min(e, in ? (unsigned)E - 1 : (unsigned)E);
        const unsigned same = __match_any_sync(FULL, e);
        const int before = __popc(same & ((1u << lane) - 1));
        if (in) lists[wh[w * E + e] + before] = first + i + lane;
        __syncwarp();
        if (in && before == 0) wh[w * E + e] += __popc(same);
        __syncwarp();
    }
}

// From total[e] (shared memory): offsets into `off` (shared) and, when `write`, counts, offsets and the experts with
// choices to the plan.  E <= 1024; tmp is 64 ints.
__device__ __forceinline__ void scan_totals(const int* total, int E, int* off, int* tmp, const PlanPtrs& plan, bool write) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int base = 0, hits = 0;  // of the experts before this round's (a CTA of fewer threads than experts takes rounds)
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        const int n = e < E ? total[e] : 0;
        int run = n;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(FULL, run, o);
            if (lane >= o) run += v;
        }
        const unsigned some = __ballot_sync(FULL, n > 0);
        if (lane == 31) tmp[w] = run, tmp[32 + w] = __popc(some);
        __syncthreads();
        int before = base, hit = hits, all = 0, all_hits = 0;
        for (int v = 0; v < (int)(blockDim.x >> 5); ++v) {
            if (v < w) before += tmp[v], hit += tmp[32 + v];
            all += tmp[v], all_hits += tmp[32 + v];
        }
        base += all, hits += all_hits;
        if (e < E) {
            off[e] = before + run - n;
            if (write) {
                plan.counts[e] = n;
                plan.offsets[e] = before + run - n;
                if (n > 0) plan.active[1 + hit + __popc(some & ((1u << lane) - 1))] = e;
            }
        }
        __syncthreads();
    }
    if (write && threadIdx.x == 0) plan.offsets[E] = base, plan.active[0] = hits;
}

// p of logit l by the fast exponential and quotient: within 8e-7 of a sigmoid, and of a softmax's largest score times that.
__device__ __forceinline__ float fast_sigmoid(float l) { return __fdividef(1.f, 1.f + __expf(-l)); }

template <int NL>
__global__ void __launch_bounds__(NL <= 8 ? 1024 : NL == 16 ? 512 : 256) route_kernel(const RouteParams p) {
    extern __shared__ char smem[];
    __shared__ int tmp[64];
    __shared__ int last_cta;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, W = blockDim.x >> 5;
    double* c64 = reinterpret_cast<double*>(smem) + w * max(p.E, 32);  // a warp's marks (f32 in the same place)
    float* cs = reinterpret_cast<float*>(c64);
    uint2* found = reinterpret_cast<uint2*>(smem) + w * max(p.E, 32);  // candidates' keys and experts, in the marks' place
    griddep_wait();  // (launches overlap up to here: nothing is read before the launch before has ended)
    const int failed = p.failed ? __ldcg(p.failed) : 0;  // (looked at only with the first results)
    const int S = p.E / p.groups;
    uint32_t group[(NL + 3) / 4] = {};  // the group of expert lane + 32 i in byte i
    if (p.groups > 1) {
#pragma unroll
        for (int i = 0; i < NL; ++i) group[i >> 2] |= (uint32_t)min((lane + 32 * i) / S, 31) << (8 * (i & 3));
    }
    float b[NL], bmax = 0.f;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = lane + 32 * i;
        b[i] = p.bias && e < p.E ? p.bias[e] : 0.f;
        if (isfinite(b[i])) bmax = fmaxf(bmax, fabsf(b[i]));
    }
    bmax = warp_max(bmax);
    const int first = p.per ? blockIdx.x * p.per : 0;
    const int end = p.per ? min(first + p.per, p.rows) : p.rows;
    const int step = p.per ? W : W * gridDim.x;
    for (int r = first + (p.per ? w : blockIdx.x * W + w); r < end; r += step) {
        const float* row = p.logits + r * p.stride;
        float l[NL];
        unsigned key[NL];
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int e = lane + 32 * i;
            l[i] = logit_of(e < p.E ? row[e] : -INFINITY);
            m = fmaxf(m, l[i]);
        }
        float m0 = 0.f, z = 0.f, zi = 0.f;
        const bool marks = p.bias || p.groups > 1;
        if (!p.sigmoid) {
            m = warp_max(m);
            m0 = m == -INFINITY ? 0.f : m;
            if (marks || !p.renorm) {
#pragma unroll
                for (int i = 0; i < NL; ++i) z += __expf(l[i] - m0);
                z = group_sum<32>(z);
                zi = z > 0.f ? 1.f / z : 0.f;
            }
        }
        // How far two f32 scores can be out against one another: fast_sigmoid's errors, or a softmax's, the exponential's
        // argument (up to 3e-7 of the largest score) and its sum's NL + 5 roundings; and the sum p + b.
        const float pmax = p.sigmoid ? 1.f : zi;
        const float tol = 2e-6f * pmax + 2e-7f * bmax + (p.sigmoid ? 0.f : 1.2e-7f * (NL + 5) * pmax);
        bool slow = false;
        // (a loop for each of the rule's choices: tests of the rule for every expert took a third of the kernel's instructions)
        if (marks) {
            float c[NL];
            if (p.sigmoid) {
#pragma unroll
                for (int i = 0; i < NL; ++i) c[i] = fast_sigmoid(l[i]) + b[i];
            } else {
#pragma unroll
                for (int i = 0; i < NL; ++i) c[i] = fmaf(__expf(l[i] - m0), zi, b[i]);
            }
#pragma unroll
            for (int i = 0; i < NL; ++i)  // (a c that is no number is out of service too)
                c[i] = l[i] > -INFINITY && c[i] > -INFINITY ? c[i] : -INFINITY;
            if (p.groups > 1) {
#pragma unroll
                for (int i = 0; i < NL; ++i)
                    if (lane + 32 * i < p.E) cs[lane + 32 * i] = c[i];
            }
            if (p.bias) {
#pragma unroll
                for (int i = 0; i < NL; ++i) l[i] = c[i];  // what orders the experts
            }
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) key[i] = l[i] > -INFINITY ? order_key(l[i]) : kOff;
        if (p.E < 32 * NL) {
#pragma unroll
            for (int i = 0; i < NL; ++i)
                if (lane + 32 * i >= p.E) key[i] = kHidden;
        }
        if (p.groups > 1) {
            __syncwarp();
            const unsigned kept = kept_groups<float>(cs, S, p.groups, p.keep, p.top, 2.5f * tol, slow);
#pragma unroll
            for (int i = 0; i < NL; ++i)
                if (!((kept >> (group[i >> 2] >> (8 * (i & 3)) & 31u)) & 1u)) key[i] = kHidden;
        }
        // the keys that may be among the K largest: all from the K-th largest of the lanes' maxima on, and a biased order's
        // error below it
        unsigned mine = key[0], from = kHidden;
#pragma unroll
        for (int i = 1; i < NL; ++i) mine = max(mine, key[i]);
        for (int j = 0; j < p.K; ++j) {
            from = __reduce_max_sync(FULL, mine);
            if (lane == __ffs(__ballot_sync(FULL, mine == from)) - 1) mine = kHidden;
        }
        if (from > kOff && p.bias) from = max(order_key(key_value(from) - tol), kOff + 1);
        __syncwarp();  // (the marks have been read)
        const unsigned least = max(from, kOff + 1);
        int n = 0;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const unsigned here = __ballot_sync(FULL, key[i] >= least);
            if (here == 0) continue;
            if (key[i] >= least) found[n + __popc(here & ((1u << lane) - 1))] = make_uint2(key[i], lane + 32 * i);
            n += __popc(here);
        }
        if (from <= kOff && n <= 32) {  // too few in service: the first of the others behind them
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const unsigned here = __ballot_sync(FULL, key[i] == kOff);
                const int at = n + __popc(here & ((1u << lane) - 1));
                if (key[i] == kOff && at < 32) found[at] = make_uint2(kOff, lane + 32 * i);
                n = min(n + __popc(here), 32);
            }
        }
        __syncwarp();
        // lane j: candidate j (they stand in the order of their experts), and how many come before it
        unsigned k = kHidden;
        int id = 0, rank = 32;
        bool close = false;
        if (n <= 32) {
            if (lane < n) k = found[lane].x, id = found[lane].y;
            rank = lane < n ? 0 : 32;
            for (int j = 0; j < n; j += 4) {  // (lanes past the last hold what is before nothing)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const unsigned o = __shfl_sync(FULL, k, j + i);
                    rank += o > k || (o == k && j + i < lane);
                }
            }
            if (p.bias) {  // neighbours of the order that the errors reach across
                __syncwarp();
                if (lane < n) found[rank].x = k;
                __syncwarp();
                const unsigned here = found[lane].x, next = found[(lane + 1) & 31].x;
                close = lane < p.K && lane + 1 < n && next > kOff && !(key_value(here) - key_value(next) > tol);
            }
        }
        close = __any_sync(FULL, close);
        bool on = k > kOff;
        if (slow || n > 32 || (close && !p.sigmoid)) {
            __syncwarp();
            choose_exactly(p, row, c64, id, on);
            rank = lane;
        } else if (close) {  // the candidates' marks in 64 bits
            const double c = on ? 1 / (1 + exp(-(double)logit_of(row[id]))) + (double)p.bias[id] : k == kOff ? -1.7e308 : -INFINITY;
            rank = lane < n ? 0 : 32;
            for (int j = 0; j < n; ++j) {
                const double o = __shfl_sync(FULL, c, j);
                rank += o > c || (o == c && j < lane);
            }
        }
        // gates, of the lanes whose expert is chosen
        const bool kth = rank < p.K;
        id = min(max(id, 0), p.E - 1);
        float gate = 0.f;
        const float v = kth && on ? logit_of(row[id]) : -INFINITY;
        if (p.renorm) {  // relative to the largest: below -20 a sigmoid is e^l to less than f32's rounding
            const float most = warp_max(v);
            if (v > -INFINITY) gate = p.sigmoid && most >= -20.f ? 1.f / (1.f + expf(-v)) : expf(v - most);
            const float sum = group_sum<32>(gate);
            gate = sum > 0.f ? gate / sum : 0.f;
        } else if (p.sigmoid) {
            if (v > -INFINITY) gate = v < -80.f ? expf(v) : 1.f / (1.f + expf(-v));
        } else {  // (the sum again, by the exact exponential)
            float zs = 0.f;
#pragma unroll
            for (int i = 0; i < NL; ++i) zs += expf(logit_of(lane + 32 * i < p.E ? row[lane + 32 * i] : -INFINITY) - m0);
            zs = group_sum<32>(zs);
            if (v > -INFINITY) gate = expf(v - m0) / zs;
        }
        if (kth && failed == 0) {
            p.ids[(int64_t)r * p.K + rank] = id;
            p.gates[(int64_t)r * p.K + rank] = gate * p.scale;
        }
        __syncwarp();
    }
    if (!p.per || !p.plan.counts) return;
    // The grouping: by the last CTA of few choices, else this CTA's counts for the CTAs that place the choices.
    int from = first, n = (end - first) * p.K;
    if (__syncthreads_or(failed)) return;
    if (!p.hist) {
        if (gridDim.x > 1) {
            if (threadIdx.x == 0) last_cta = atomic_add_acq_rel_gpu(p.arrived, 1) == (int)gridDim.x - 1;
            __syncthreads();
            if (!last_cta) return;
            if (threadIdx.x == 0) *p.arrived = 0;
        }
        from = 0, n = p.rows * p.K;
    }
    int* wh = reinterpret_cast<int*>(smem);
    int* total = reinterpret_cast<int*>(smem + (size_t)W * p.E * 4);
    int* off = total + p.E;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) total[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const unsigned e = __ldcg(p.ids + (int64_t)from * p.K + i);
        atomicAdd(&total[min(e, (unsigned)p.E - 1)], 1);
    }
    __syncthreads();
    if (p.hist) {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.hist[(int64_t)blockIdx.x * p.E + e] = total[e];
        return;
    }
    scan_totals(total, p.E, off, tmp, p.plan, true);
    __syncthreads();
    place_choices<true>(p.ids, 0, n, p.E, wh, off, p.plan.lists);
}

// CTA b places the choices of route_kernel's CTA b: the counts of all CTAs give every expert's total and where CTA b's
// choices start.
__global__ void __launch_bounds__(kPlaceThreads) place_kernel(const RouteParams p) {
    extern __shared__ char smem[];
    __shared__ int tmp[64];
    int* total = reinterpret_cast<int*>(smem);
    int* off = total + p.E;
    int* before = off + p.E;
    int* wh = before + p.E;
    griddep_wait();
    const int failed = p.failed ? __ldcg(p.failed) : 0;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) total[e] = before[e] = 0;
    __syncthreads();
    const int mine = blockIdx.x;
    if (p.E % 4 == 0) {  // four experts a thread
        const int quads = p.E / 4, parts = max(1, (int)blockDim.x / quads);
        for (int i = threadIdx.x; i < parts * quads; i += blockDim.x) {
            const int q = i % quads;
            int4 all = make_int4(0, 0, 0, 0), pre = all;
#pragma unroll 10
            for (int b = i / quads; b < (int)gridDim.x; b += parts) {
                const int4 n = *reinterpret_cast<const int4*>(p.hist + (int64_t)b * p.E + 4 * q);
                all.x += n.x, all.y += n.y, all.z += n.z, all.w += n.w;
                if (b < mine) pre.x += n.x, pre.y += n.y, pre.z += n.z, pre.w += n.w;
            }
            atomicAdd(&total[4 * q], all.x), atomicAdd(&total[4 * q + 1], all.y), atomicAdd(&total[4 * q + 2], all.z);
            atomicAdd(&total[4 * q + 3], all.w), atomicAdd(&before[4 * q], pre.x), atomicAdd(&before[4 * q + 1], pre.y);
            atomicAdd(&before[4 * q + 2], pre.z), atomicAdd(&before[4 * q + 3], pre.w);
        }
    } else {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
            int all = 0, pre = 0;
#pragma unroll 8
            for (int b = 0; b < (int)gridDim.x; ++b) {
                const int n = p.hist[(int64_t)b * p.E + e];
                all += n;
                if (b < mine) pre += n;
            }
            total[e] = all, before[e] = pre;
        }
    }
    if (__syncthreads_or(failed)) return;  // (the histograms have not been written)
    scan_totals(total, p.E, off, tmp, p.plan, mine == 0);
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) off[e] += before[e];
    __syncthreads();
    const int first = mine * p.per, end = min(first + p.per, p.rows);
    place_choices<false>(p.ids, first * p.K, max(end - first, 0) * p.K, p.E, wh, off, p.plan.lists);
}

template <int NL>
cudaError_t run(RouteParams p, Carve& ws, cudaStream_t st) {
    constexpr int most = (NL <= 8 ? 1024 : NL == 16 ? 512 : 256) / 32;  // warps
    constexpr size_t limit = 65536;
    static_assert(most * NL * 32 * 8 <= limit, "a CTA's rows in shared memory");
    const int sms = device_info().sms;
    auto bytes = [&](int W) { return (size_t)W * max(p.E, 32) * 8; };
    if (bytes(most) > (48 << 10)) {
        static std::atomic<uint64_t> done;
        const cudaError_t e = allow_smem(route_kernel<NL>, limit, done);
        if (e != cudaSuccess) return e;
    }
    if (!p.plan.counts) {
        const int W = 4;
        const int64_t grid = min((int64_t)(p.rows + W - 1) / W, (int64_t)sms * 8);
        return launch(route_kernel<NL>, dim3((unsigned)grid), dim3(32 * W), bytes(W), st, 1, p);
    }
    // With a plan: up to 1536 choices a row a warp and the grouping by the last CTA, which is one launch; from there on a CTA an
    // SM, and a second launch.  Measured, us: 16 rows of 64 experts, 6 chosen, 5.0 and 8.8; 8 of 256: 128 rows 8.2 and 10.6, 256
    // rows 11.4 and 10.6, 512 rows 16.7 and 11.0.
    const bool few = (int64_t)p.rows * p.K <= 1536;
    const int W = few ? min(most, 8) : most;
    const int grid = few ? (p.rows + W - 1) / W : min(sms, (p.rows + W - 1) / W);
    p.per = (p.rows + grid - 1) / grid;
    p.failed = ws.failed;
    if (few && grid > 1) p.arrived = ws.take_counters(1);
    if (!few) p.hist = ws.take<int32_t>((size_t)grid * p.E);
    if (ws.overflow) return cudaSuccess;
    cudaError_t e = launch(route_kernel<NL>, dim3(grid), dim3(32 * W), bytes(W), st, 1, p);
    if (e != cudaSuccess || few) return e;
    const size_t place = (size_t)p.E * 4 * (3 + kPlaceThreads / 32);
    if (place > (48 << 10)) {
        static std::atomic<uint64_t> done;
        e = allow_smem(place_kernel, 1024 * 4 * (3 + kPlaceThreads / 32), done);
        if (e != cudaSuccess) return e;
    }
    return launch(place_kernel, dim3(grid), dim3(kPlaceThreads), place, st, 1, p);
}

}  // namespace

cudaError_t launch_route_scored(const RouteScoredCall& c, Carve& ws, cudaStream_t st) {
    RouteParams p = {c.logits, c.stride, (int)c.rows, c.E, c.K, c.rule.bias, c.rule.score == Q8_SCORE_SIGMOID,
                     c.rule.groups, c.rule.keep_groups, c.rule.group_top, c.rule.renorm, c.rule.scale, c.ids, c.gates, c.plan,
                     nullptr, nullptr, 0, nullptr};
    if (p.E <= 32) return run<1>(p, ws, st);
    if (p.E <= 64) return run<2>(p, ws, st);
    if (p.E <= 128) return run<4>(p, ws, st);
    if (p.E <= 256) return run<8>(p, ws, st);
    if (p.E <= 512) return run<16>(p, ws, st);
    return run<32>(p, ws, st);
}

}  // namespace q8
