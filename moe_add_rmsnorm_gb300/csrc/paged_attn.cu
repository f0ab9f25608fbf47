// Causal attention of a ragged batch's rows over pages of 8-bit key and value words (q8moe.h, q8_paged_attention): the
// kernel for few query vectors a key/value head (decoding), and the choice between it and paged_attn_tc.cu's.
//
// What it computes: qwen_emit docs, emit_qwen30b_generate (causal attention over a cache, query heads grouped evenly over
// key/value heads) for rows of several sequences over pages; out = sum_t w_t d_t v_t / sum_t w_t with
// w_t = 2^(s_t - m), s_t = log2(e) scale c_t (q . k_t), c and d the cached rows' scales, k and v their words.
//
// How: a position is read once (2 (hd + 4) bytes a key/value head) for all the query vectors of its group, so the words'
// bytes bound it; on the CUDA cores the products of 8 vectors already cost more than the bytes (4 * 8 * 128 flops on 264
// bytes: about 100 TFLOP/s at the memory's rate, above the part's f32 rate), so they run on the tensor cores' warp-wide
// form, m16n8k16: 16 positions (or dimensions) by 8 vectors.  Words are exact in f16.  The f32 operand (query, or weight
// times value scale) is scaled by a power of two and split into two f16 parts, x = hi + lo to 2^-22, both products
// accumulated in f32.
//  - A warp takes 16 positions at a time from a ring of its own: two stages in shared memory, filled by tensor copies of
//    a page's 16 rows that are issued as a stage is read out, waited for by that warp alone.  (Loads straight into
//    registers could be issued only half a step ahead within 128 registers: 64 sequences of up to 4096, 32 heads over 4,
//    took 8% more, one of 100003 5%.)  The order of a contraction's index is free, so each
//    lane reads 32 (hd 128) consecutive bytes of a key row as its share of the scores' dimensions, and 16 of four value
//    rows as its share of the output's; the copies' swizzle keeps those reads apart.
//  - Scores come out as positions by vectors and go back in as the second product's operand after an 8 x 8 transpose of
//    their f16 parts across the warp.
//  - Every warp keeps its own running maximum and sums, rescaled only when one moves.  The tensor cores truncate as they
//    accumulate, so every 8 steps the products are added (rounded) to the warp's f32 totals in shared memory.
//  - 8 warps a CTA, two CTAs an SM (one for more than 8 vectors, whose sums take the registers), each CTA an equal run of
//    128-position units over the whole batch.  The warps' results meet in shared memory; an item that several CTAs share
//    meets in the workspace, folded in order by the last to arrive.
//
// What holds it back: a step's own chain (words, scores, maximum, exponentials, transposes, products), which 16 warps an SM
// do not hide.  A step is 610 warp instructions on 4224 bytes (over a third turn bytes into pairs of f16, the rest are the
// products, the softmax and the splits); 64 sequences of 4096 (66 us, 4.2 TB/s) use 57% of the issue slots and 55% of the
// memory's rate, and the stalls that lead are fixed latencies (wait) and other warps' turns (not selected).  64 ragged
// ones of up to 4096 take 45.2 us (3.4 TB/s), one of 100003 38.6 (2.7 TB/s).
#include <cuda_fp16.h>

#include "paged_attn.cuh"

namespace q8 {

namespace {

constexpr int PR_WARPS = 8, PR_THREADS = PR_WARPS * 32;
constexpr int PR_UNIT = 128;   // positions a unit
// What an item's start and end cost, in units (64 ragged sequences of up to 4096, one row each: 49.3 us with 0, 47.1 with 1,
// 45.0 with 2, 45.4 with 4, 50.8 with 8; 33 of up to 8885, 3 rows of heads of 64: 61.4, 59.2, 57.4, 55.2, 56.5; in the
// present form, with 2, 3 and 4, 45.8, 45.2 and 47.1, and 58.2, 56.8 and 55.4).
constexpr int PR_START = 3;
constexpr int PR_STEP = 16;    // positions a warp takes at a time
constexpr int PR_FLUSH = 8;    // steps between additions to the totals
// Weights times value scales are split as values of up to 65472 (f16 holds 65504): PR_TOP times a scale below 2.
constexpr float PR_TOP = 32736.f;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Two f32 values as two f16 parts each.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack_f16(a, b);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    lo = pack_f16(a - f.x, b - f.y);
}

template <int BYTES>
struct Bytes {
    uint32_t w[BYTES / 4];
};

// NT: 8-vector tiles an item (1 or 2).
template <int HD, int NT>
struct RowsShared {
    static constexpr int CTAS = NT == 1 ? 2 : 1;           // of an SM
    unsigned char ring[PR_WARPS][2][2][PR_STEP * HD];      // each warp's next steps: two stages of keys and values
    uint64_t full[PR_WARPS][2];
    static constexpr int MT = 8 * NT, FR = HD / 16 * NT;   // vectors an item; float4 totals a lane
    uint4 q[NT][HD / 16][32];          // the queries' parts in the scores' operand order: hi (2 registers), lo
    float4 o[PR_WARPS][FR][32];        // the warps' totals, in the accumulators' order
    float m[PR_WARPS][MT], l[PR_WARPS][MT], f[PR_WARPS][MT];
    float qf[MT];                      // what turns a scaled product into a score, without the key's scale
    int lim[MT];                       // the last position a vector attends (-1: none)
    int64_t at[MT];                    // where a vector's output starts (-1: no such vector)
    int64_t lse_at[MT];
    // What the walk over the items keeps between them (in shared memory: the registers are the inner loop's).
    int64_t cur, lo, hi, seq_at, item_at, units, total;
    int seq, ctas, last;
    int dead;                          // a wait gave up: the CTA leaves
};

template <int HD, int WORDS, int NT>
__global__ void __launch_bounds__(PR_THREADS, RowsShared<HD, NT>::CTAS)
    paged_rows_kernel(const PagedParams pk, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v) {
    constexpr int MT = 8 * NT, KB = HD / 4, KS = HD / 16, DPG = HD / 8, FR = HD / 16 * NT;
    constexpr int SLOT = FR * 32 * 4 + 2 * MT;  // floats of a partial result
    extern __shared__ unsigned char raw[];
    RowsShared<HD, NT>& sh = *reinterpret_cast<RowsShared<HD, NT>*>(raw + (1024u - smem_addr(raw) % 1024u) % 1024u);
    const KvView& kv = pk.view;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, t = lane & 3;
    const int G = pk.group;

    auto tiles_of = [&](const KvSeq& s) { return (s.n * G + MT - 1) / MT; };  // (MT is a power of two)
    auto span_of = [&](const KvSeq& s) -> int64_t {  // units of one item
        return s.len_ok ? (s.len + PR_UNIT - 1) / PR_UNIT : 1;
    };
    auto units = [&](const KvSeq& s) -> int64_t {
        return paged_takes(pk, s) ? kv.kv * tiles_of(s) * (PR_START + span_of(s)) : 0;
    };
    {
        const PagedRun run = paged_run<PR_THREADS>(pk, units);
        if ((int)blockIdx.x >= run.ctas) return;
        if (tid == 0) {
            sh.cur = sh.lo = run.lo, sh.hi = run.hi;
            sh.seq = run.seq, sh.seq_at = run.seq_at;
            sh.total = run.total, sh.ctas = run.ctas;
            for (int i = 0; i < 2 * PR_WARPS; ++i) mbar_init(&sh.full[0][i], 1);
            sh.dead = 0;
            fence_barrier_init();
        }
    }
    __syncthreads();

    // Where this lane reads a stage: keys of rows g, g + 8, 32 dimensions from KB t (two 16-byte chunks; hd 64: one);
    // values of rows 2t, 2t + 1, 2t + 8, 2t + 9, dimensions from DPG g; as the tensor copies' swizzle places them (a
    // quarter warp's reads lie in different banks).
    const uint32_t k_lane = HD == 128 ? g * 128 + (((2 * t) ^ g) << 4) : g * 64 + ((t ^ ((g >> 1) & 3)) << 4);
    const uint32_t k_next = g * 128 + (((2 * t + 1) ^ g) << 4);  // (hd 128)
    const uint32_t v_lane = HD == 128 ? 2 * t * 128 + ((g ^ (2 * t)) << 4) : 2 * t * 64 + (((g >> 1) ^ t) << 4) + (g & 1) * 8;
    const uint32_t v_odd = HD == 128 ? (2 * t + 1) * 128 + ((g ^ (2 * t + 1)) << 4) : v_lane + 64;
    unsigned used = 0;  // steps this warp has taken

    for (;;) {
        int b, begin, end, h;
        KvSeq s;
        int64_t m0;
        {
            const int64_t cur = sh.cur, hi = sh.hi;
            if (cur >= hi) break;
            b = sh.seq;
            int64_t at = sh.seq_at, n_units;
            s = kv_seq(kv, b);
            while (cur >= at + (n_units = units(s))) {  // the sequence of unit `cur`
                at += n_units;
                s = kv_seq(kv, ++b);
            }
            const int64_t U = span_of(s), tiles = tiles_of(s), item = div_small(cur - at, PR_START + U);
            h = (int)div_small(item, tiles);
            m0 = (item - h * tiles) * MT;  // the item's first vector
            const int64_t item_at = at + item * (PR_START + U), first = item_at + PR_START;
            const int64_t u0 = max(int64_t(0), cur - first), u1 = min(U, hi - first);
            if (u1 <= u0) break;  // the run ends in the item's start: nothing of it is this CTA's
            begin = (int)(u0 * PR_UNIT);
            end = s.len_ok ? (int)min((int64_t)s.len, u1 * PR_UNIT) : 0;  // positions before which the piece ends
            __syncthreads();  // every thread has read the walk's state
            if (tid == 0) {
                sh.cur = u1 == U ? first + U : hi;
                sh.seq = b, sh.seq_at = at;
                sh.item_at = item_at, sh.units = U;
                sh.last = u0 == 0 && u1 == U ? 1 : 0;  // whether the piece is the whole item
            }
        }

        // ---- this warp's first positions are on their way while the queries are prepared
        const int steps = end > begin ? (end - begin + PR_STEP - 1) / PR_STEP : 0;  // of all warps
        int page_l = -1;  // this lane's: the page of the warp's step (batch of 32 steps)
        auto look_up = [&](int i) {  // the pages of the warp's steps i .. i + 31
            const int step = wid + (i + lane) * PR_WARPS;
            page_l = -1;
            if (step < steps) {
                page_l = kv_page(kv, b, begin + step * PR_STEP);
                if (page_l < 0) kv_flag(kv, Q8_KV_ERR_PAGE);
            }
        };
        auto page_of = [&](int i) { return __shfl_sync(0xffffffffu, page_l, i & 31); };
        auto slot_of_step = [&](int i) {  // the row of step i's first position in its page
            return (h << kv.page_log2) + ((begin + (wid + i * PR_WARPS) * PR_STEP) & ((1 << kv.page_log2) - 1));
        };
        auto issue = [&](int i, int page) {  // step i's words on their way
            if (lane == 0) {
                const unsigned stage = (used + i) & 1;
                mbar_arrive_expect_tx(&sh.full[wid][stage], 2 * PR_STEP * HD + pk.missing);
                tma_box(sh.ring[wid][stage][0], &map_k, slot_of_step(i), page < 0 ? kv.pages : page, &sh.full[wid][stage]);
                tma_box(sh.ring[wid][stage][1], &map_v, slot_of_step(i), page < 0 ? kv.pages : page, &sh.full[wid][stage]);
            }
        };
        const uint32_t page_rows = (uint32_t)kv.kv << kv.page_log2;
        float ks[2], vs[2];
        auto load_scales = [&](int i, int page) {
            const uint64_t row = (uint64_t)(uint32_t)max(page, 0) * page_rows + slot_of_step(i) + g;
#pragma unroll
            for (int j = 0; j < 2; ++j) ks[j] = ld_scale_stream(kv.ks + row + 8 * j), vs[j] = ld_scale_stream(kv.vs + row + 8 * j);
        };
        const int mine = steps > wid ? (steps - wid + PR_WARPS - 1) / PR_WARPS : 0;
        int page_next = -1, page_after = -1;
        if (mine > 0) {
            look_up(0);
            page_next = page_of(0);
            issue(0, page_next);
            load_scales(0, page_next);
            if (mine > 1) {
                page_after = page_of(1);
                issue(1, page_after);
            }
        }
        // ---- the item's queries: a warp a vector, split into two f16 parts after a scaling by a power of two
        for (int vec = wid; vec < MT; vec += PR_WARPS) {
            const int64_t m = m0 + vec;
            const bool valid = m < s.n * G;
            const int token = (int)div_small(m, G);
            const int64_t row = s.first + token;
            const int head = h * G + (int)(m - (int64_t)token * G);
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (valid && lane < HD / 4)
                x = *reinterpret_cast<const float4*>(pk.q + row * pk.q_stride + (int64_t)head * HD + 4 * lane);
            const unsigned big = __reduce_max_sync(
                0xffffffffu, max(max(__float_as_uint(fabsf(x.x)), __float_as_uint(fabsf(x.y))),
                                 max(__float_as_uint(fabsf(x.z)), __float_as_uint(fabsf(x.w)))));
            const int e = big == 0u ? 0 : 14 - exponent_of(big);
            const float f = pow2i(e);
            uint4 r;
            split2(x.x * f, x.y * f, r.x, r.z);
            split2(x.z * f, x.w * f, r.y, r.w);
            if (lane < HD / 4) sh.q[vec / 8][lane % KS][(vec % 8) * 4 + lane / KS] = r;
            if (lane == 0) {
                sh.qf[vec] = pow2i(-e) * pk.scale;
                sh.lim[vec] = valid && s.len_ok ? (int)(s.len - s.n + token) : -1;
                sh.at[vec] = valid ? row * pk.out_stride + (int64_t)head * HD : -1;
                sh.lse_at[vec] = row * pk.heads + head;
            }
        }
        __syncthreads();

        // ---- this warp's positions
        float m_run[NT][2], l_run[NT][2], fac[NT][2], qf[NT][2];
        float acc[NT][HD / 16][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                m_run[n][c] = -INFINITY;
                l_run[n][c] = 0.f;
                fac[n][c] = 1.f;
                qf[n][c] = sh.qf[8 * n + 2 * t + c];
            }
#pragma unroll
            for (int i = 0; i < HD / 16; ++i) {
                sh.o[wid][n * (HD / 16) + i][lane] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[n][i][c] = 0.f;
            }
        }
        int low = INT_MAX;
#pragma unroll
        for (int i = 0; i < MT; ++i) low = min(low, sh.at[i] >= 0 ? sh.lim[i] : INT_MAX);
        int exp_run = -100, exp_top = -100;  // the weights' scaling, and the largest it has been
#pragma unroll 1
        for (int i = 0; i < mine; ++i) {
            const int page = page_next;
            const int p0 = begin + (wid + i * PR_WARPS) * PR_STEP;
            const unsigned stage = (used + i) & 1;
            const float kscale[2] = {ks[0], ks[1]}, vraw[2] = {vs[0], vs[1]};
            if (i + 1 < mine) load_scales(i + 1, page_after);
            bool got = try_wait(&sh.full[wid][stage], ((used + i) >> 1) & 1);
#pragma unroll 1
            for (unsigned poll = 0; !got && poll < pk.polls && !*(volatile int*)&sh.dead; ++poll)
                got = try_wait(&sh.full[wid][stage], ((used + i) >> 1) & 1);
            if (__builtin_expect(!__all_sync(0xffffffffu, got), 0)) {
                // Nothing of what the ring holds is used and nothing more is copied; this step's copies and the next one's
                // may be on their way, and none is in flight when the CTA leaves.
                *(volatile int*)&sh.dead = 1;
#pragma unroll 1
                for (int j = i; j < mine && j < i + 2; ++j) drain(&sh.full[wid][(used + j) & 1], ((used + j) >> 1) & 1);
                break;
            }
            Bytes<KB> kw[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const unsigned char* from = sh.ring[wid][stage][0] + 8 * HD * j;
#pragma unroll
                for (int x = 0; x < KB / 16; ++x) {
                    const uint4 w = *reinterpret_cast<const uint4*>(from + (x ? k_next : k_lane));
                    kw[j].w[4 * x] = w.x, kw[j].w[4 * x + 1] = w.y, kw[j].w[4 * x + 2] = w.z, kw[j].w[4 * x + 3] = w.w;
                }
            }
            // scores: positions g, g + 8 by vectors 2t, 2t + 1 of each tile
            float sh_hi[NT][4], sh_lo[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) sh_hi[n][c] = 0.f, sh_lo[n][c] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const uint32_t w0 = words_flip<WORDS>(kw[0].w[k]), w1 = words_flip<WORDS>(kw[1].w[k]);
                const uint32_t a0 = words2_f16<WORDS, 0>(w0), a1 = words2_f16<WORDS, 0>(w1);
                const uint32_t a2 = words2_f16<WORDS, 1>(w0), a3 = words2_f16<WORDS, 1>(w1);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 q = sh.q[n][k][lane];
                    mma16816(sh_hi[n], a0, a1, a2, a3, q.x, q.y);
                    mma16816(sh_lo[n], a0, a1, a2, a3, q.z, q.w);
                }
            }
            // the softmax's running maximum and sums, and the weights' parts
            const bool here = page >= 0;
            float vscale[2];
            unsigned vtop = 0u;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                vscale[j] = here && p0 + g + 8 * j < end ? vraw[j] : 0.f;
                vtop = max(vtop, finite_bits(vscale[j]));
            }
            vtop = __reduce_max_sync(0xffffffffu, vtop);
            float sc[NT][4];
            bool moved = false;  // whether a maximum or the weights' scaling changes: the sums are rescaled then
            const bool all = here && p0 + PR_STEP <= low + 1;  // (low: the smallest of the vectors' last positions)
            unsigned seen = 0xffffffffu;
            bool apart = false;  // whether some of a masked step's value scales lie far below the weights' scaling
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) sc[n][c] = (sh_hi[n][c] + sh_lo[n][c]) * (kscale[c >> 1] * qf[n][c & 1]);
            if (!all) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (!(here && p0 + g + 8 * (c >> 1) <= sh.lim[8 * n + 2 * t + (c & 1)])) {
                            sc[n][c] = -INFINITY;
                            seen &= ~(1u << (4 * n + c));
                        }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) moved |= fmaxf(sc[n][c], sc[n][c + 2]) > m_run[n][c];
            if (vtop != 0u) {
                const int e = exponent_of(vtop);
                // (kept while the tile's largest scale is within its octave or the one below: fewer rescalings)
                moved |= e > exp_run || e < exp_run - 1;
            }
            if (__any_sync(0xffffffffu, moved)) {
                const int exp_old = exp_run;
                if (vtop != 0u) {
                    const int e = exponent_of(vtop);
                    exp_top = max(exp_top, e);
                    // (not far below what it was, so that rescaling the sums never overflows)
                    if (e > exp_run || e < exp_run - 1) exp_run = max(e, exp_top - 40);
                }
                const float eshift = exp_old - exp_run <= -126 ? 0.f : pow2i(exp_old - exp_run);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float alpha[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mx = fmaxf(sc[n][c], sc[n][c + 2]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        const float mn = fmaxf(m_run[n][c], mx), ms = mn == -INFINITY ? 0.f : mn;
                        alpha[c] = ex2(m_run[n][c] - ms);
                        m_run[n][c] = mn;
                        l_run[n][c] *= alpha[c];
                        alpha[c] *= eshift;
                        fac[n][c] *= alpha[c];
                    }
#pragma unroll
                    for (int j = 0; j < HD / 16; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[n][j][c] *= alpha[c & 1];
                }
            }
            const float wscale = pow2i(14 - exp_run) * (PR_TOP / 16384.f);
            uint32_t ph[NT][2], pl[NT][2];
            float wt[NT][4];
            const float vw0 = vscale[0] * wscale, vw1 = vscale[1] * wscale;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float ms = m_run[n][c] == -INFINITY ? 0.f : m_run[n][c];
                    const float e0 = ex2(sc[n][c] - ms), e1 = ex2(sc[n][c + 2] - ms);
                    l_run[n][c] += e0 + e1;
                    wt[n][c] = e0 * vw0;
                    wt[n][c + 2] = e1 * vw1;
                }
            if (!all) {  // (a value scale that is not a number stays behind the mask)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (!((seen >> (4 * n + c)) & 1u)) wt[n][c] = 0.f;
                const unsigned bits[2] = {finite_bits(vscale[0]), finite_bits(vscale[1])};
#pragma unroll
                for (int j = 0; j < 2; ++j) apart |= bits[j] != 0u && exp_run - exponent_of(bits[j]) > PA_SPREAD;
                apart = __any_sync(0xffffffffu, apart);
                if (__builtin_expect(apart, 0)) {
                    // The weights of a vector that sees only such scales, and its products so far, go up by a power of two
                    // for this step, and down after it.  (The products so far are fewer than 2^7 of values below 2^16 times
                    // words below 2^9, in terms of exp_top: what they go up by keeps them below 2^122.)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            unsigned own = max((seen >> (4 * n + c)) & 1u ? bits[0] : 0u, (seen >> (4 * n + c + 2)) & 1u ? bits[1] : 0u);
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) own = max(own, __shfl_xor_sync(0xffffffffu, own, o));
                            const int d = own == 0u ? 0 : min(max(exp_run - exponent_of(own), 0), 90 - (exp_top - exp_run));
                            wt[n][c] *= pow2i(d), wt[n][c + 2] *= pow2i(d);
#pragma unroll
                            for (int j = 0; j < HD / 16; ++j) acc[n][j][c] *= pow2i(d), acc[n][j][c + 2] *= pow2i(d);
                            if (g == 0) sh.f[wid][8 * n + 2 * t + c] = pow2i(-d);
                        }
                    __syncwarp();
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                split2(wt[n][0], wt[n][1], ph[n][0], pl[n][0]);
                split2(wt[n][2], wt[n][3], ph[n][1], pl[n][1]);
#pragma unroll
                for (int j = 0; j < 2; ++j) ph[n][j] = transpose8x8(ph[n][j]), pl[n][j] = transpose8x8(pl[n][j]);
            }
            Bytes<DPG> vw[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const unsigned char* from = sh.ring[wid][stage][1] + 8 * HD * (j >> 1) + (j & 1 ? v_odd : v_lane);
                if constexpr (DPG == 16) {
                    const uint4 w = *reinterpret_cast<const uint4*>(from);
                    vw[j].w[0] = w.x, vw[j].w[1] = w.y, vw[j].w[2] = w.z, vw[j].w[3] = w.w;
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(from);
                    vw[j].w[0] = w.x, vw[j].w[1] = w.y;
                }
            }
            if (p0 + PR_STEP > end || !here) {  // words past the end are whatever the page holds: left out
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (!here || p0 + 2 * t + (j & 1) + 8 * (j >> 1) >= end)
#pragma unroll
                        for (int x = 0; x < DPG / 4; ++x) vw[j].w[x] = 0u;
            }
            // weighted values: dimensions by vectors
#pragma unroll
            for (int x = 0; x < DPG / 4; ++x) {
                uint32_t a[2][4];  // [positions 2t, 2t+1 | 2t+8, 2t+9][dimension 4x + .]
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t lo = words_flip<WORDS>(__byte_perm(vw[2 * j].w[x], vw[2 * j + 1].w[x], 0x5140));
                    const uint32_t hi = words_flip<WORDS>(__byte_perm(vw[2 * j].w[x], vw[2 * j + 1].w[x], 0x7362));
                    a[j][0] = words2_f16<WORDS, 0>(lo), a[j][1] = words2_f16<WORDS, 1>(lo);
                    a[j][2] = words2_f16<WORDS, 0>(hi), a[j][3] = words2_f16<WORDS, 1>(hi);
                }
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma16816(acc[n][2 * x + y], a[0][2 * y], a[0][2 * y + 1], a[1][2 * y], a[1][2 * y + 1], pl[n][0], pl[n][1]);
                        mma16816(acc[n][2 * x + y], a[0][2 * y], a[0][2 * y + 1], a[1][2 * y], a[1][2 * y + 1], ph[n][0], ph[n][1]);
                    }
            }
            if (__builtin_expect(apart, 0)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float f = sh.f[wid][8 * n + 2 * t + c];
#pragma unroll
                        for (int j = 0; j < HD / 16; ++j) acc[n][j][c] *= f, acc[n][j][c + 2] *= f;
                    }
            }
            __syncwarp();  // every lane has read the stage (and the factors)
            page_next = page_after;
            if (i + 2 < mine) {
                if (((i + 2) & 31) == 0) look_up(i + 2);
                page_after = page_of(i + 2);
                issue(i + 2, page_after);
            }
            if (i % PR_FLUSH == PR_FLUSH - 1 || i + 1 == mine) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int j = 0; j < HD / 16; ++j) {
                        float4& o = sh.o[wid][n * (HD / 16) + j][lane];
                        float4 v = o;
                        v.x = fmaf(v.x, fac[n][0], acc[n][j][0]), v.y = fmaf(v.y, fac[n][1], acc[n][j][1]);
                        v.z = fmaf(v.z, fac[n][0], acc[n][j][2]), v.w = fmaf(v.w, fac[n][1], acc[n][j][3]);
                        o = v;
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[n][j][c] = 0.f;
                    }
                    fac[n][0] = fac[n][1] = 1.f;
                }
            }
        }
        used += mine;
        // ---- the warps meet: every vector's maximum and sum, then the totals with each warp's factor
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = l_run[n][c];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                if (g == 0) {
                    sh.m[wid][8 * n + 2 * t + c] = m_run[n][c];
                    sh.l[wid][8 * n + 2 * t + c] = l;
                    sh.f[wid][8 * n + 2 * t + c] = pow2i(exp_run) * (1.f / PR_TOP);
                }
            }
        __syncthreads();
        if (sh.dead) {  // (every warp's copies have arrived, and no result of this item is written)
            if (tid == 0) wait_gave_up(pk);
            return;
        }
        float M = -INFINITY, L = 0.f;
        if (tid < MT) {
            for (int w = 0; w < PR_WARPS; ++w) M = fmaxf(M, sh.m[w][tid]);
            for (int w = 0; w < PR_WARPS; ++w) {
                const float f = M == -INFINITY ? 0.f : ex2(sh.m[w][tid] - M);
                L = fmaf(sh.l[w][tid], f, L);  // (no number where a warp saw scores that are none, though its maximum is -infinity)
                sh.f[w][tid] *= f;
            }
            // (the totals are divided by the sum as they are added up, so that no sum of large values overflows)
            const float inv = L == 0.f ? 0.f : 1.f / L;
            for (int w = 0; w < PR_WARPS; ++w) sh.f[w][tid] *= inv;
            sh.m[0][tid] = M;
            sh.l[0][tid] = L;
        }
        __syncthreads();
        const bool whole = sh.last != 0;
        const int64_t item_at = sh.item_at;
        float* slot = pk.part + (int64_t)(2 * blockIdx.x + (sh.lo >= item_at ? 0 : 1)) * SLOT;
        auto write_out = [&](int i, int ln, float4 v, const float* m, const float* l) {
            const int n = i / (HD / 16), dim = DPG * (ln >> 2) + 2 * (i % (HD / 16)), c = 8 * n + 2 * (ln & 3);
            if (sh.at[c] >= 0) *reinterpret_cast<float2*>(pk.out + sh.at[c] + dim) = make_float2(v.x, v.z);
            if (sh.at[c + 1] >= 0) *reinterpret_cast<float2*>(pk.out + sh.at[c + 1] + dim) = make_float2(v.y, v.w);
            if (pk.lse && i % (HD / 16) == 0 && (ln >> 2) == 0)
                for (int j = 0; j < 2; ++j)
                    if (sh.at[c + j] >= 0)
                        pk.lse[sh.lse_at[c + j]] = l[c + j] == 0.f ? -INFINITY : (m[c + j] + log2f(l[c + j])) * 0.693147180559945f;
        };
        for (int i = tid; i < FR * 32; i += PR_THREADS) {
            const int fr = i >> 5, ln = i & 31, c = 8 * (fr / (HD / 16)) + 2 * (ln & 3);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = 0; w < PR_WARPS; ++w) {
                const float4 o = sh.o[w][fr][ln];
                const float f0 = sh.f[w][c], f1 = sh.f[w][c + 1];
                v.x = fmaf(o.x, f0, v.x), v.y = fmaf(o.y, f1, v.y), v.z = fmaf(o.z, f0, v.z), v.w = fmaf(o.w, f1, v.w);
            }
            if (whole) write_out(fr, ln, v, sh.m[0], sh.l[0]);
            else __stcg(reinterpret_cast<float4*>(slot) + i, v);
        }
        if (!whole) {
            // ---- the item's pieces meet: the last CTA to arrive folds them in order
            if (tid < MT) {
                __stcg(slot + FR * 128 + tid, M);
                __stcg(slot + FR * 128 + MT + tid, L);
            }
            PagedRun run;
            run.total = sh.total, run.ctas = sh.ctas;
            const int c0 = run.owner(item_at + PR_START), c1 = run.owner(item_at + PR_START + sh.units - 1);
            __syncthreads();
            if (tid == 0) sh.last = atomic_add_acq_rel_gpu(pk.counters + c0, 1) == c1 - c0;
            __syncthreads();
            if (sh.last) {
                if (tid == 0) pk.counters[c0] = 0;
                const bool opens = run.start(c0) >= item_at;
                auto slot_of = [&](int c) { return pk.part + (int64_t)paged_slot(c, c0, opens) * SLOT; };
                // every piece's share of every vector's sum, then the results with many pieces' loads in flight
                const int pieces = c1 - c0 + 1;
                float* wf = reinterpret_cast<float*>(sh.o);  // [pieces][MT]: the warps' totals are used up
                for (int i = tid; i < pieces * MT; i += PR_THREADS) wf[i] = __ldcg(slot_of(c0 + i / MT) + FR * 128 + i % MT);
                __syncthreads();
                if (tid < MT) {
                    float Mx = -INFINITY;
                    for (int p = 0; p < pieces; ++p) Mx = fmaxf(Mx, wf[p * MT + tid]);
                    sh.m[0][tid] = Mx;
                }
                __syncthreads();
                for (int i = tid; i < pieces * MT; i += PR_THREADS) {
                    const float mx = sh.m[0][i % MT], l = __ldcg(slot_of(c0 + i / MT) + FR * 128 + MT + i % MT);
                    wf[i] = ex2(wf[i] - (mx == -INFINITY ? 0.f : mx)) * l;
                }
                __syncthreads();
                if (tid < MT) {
                    float Lx = 0.f;
                    for (int p = 0; p < pieces; ++p) Lx += wf[p * MT + tid];
                    sh.l[0][tid] = Lx;
                    sh.f[0][tid] = Lx == 0.f ? 0.f : 1.f / Lx;
                }
                __syncthreads();
                for (int i = tid; i < FR * 32; i += PR_THREADS) {
                    const int fr = i >> 5, ln = i & 31, c = 8 * (fr / (HD / 16)) + 2 * (ln & 3);
                    const float x0 = sh.f[0][c], x1 = sh.f[0][c + 1];
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int p = 0; p < pieces; ++p) {
                        const float4 o = __ldcg(reinterpret_cast<const float4*>(slot_of(c0 + p)) + i);
                        const float f0 = wf[p * MT + c] * x0, f1 = wf[p * MT + c + 1] * x1;
                        v.x = fmaf(o.x, f0, v.x), v.y = fmaf(o.y, f1, v.y), v.z = fmaf(o.z, f0, v.z), v.w = fmaf(o.w, f1, v.w);
                    }
                    write_out(fr, ln, v, sh.m[0], sh.l[0]);
                }
            }
        }
        __syncthreads();  // the shared arrays are the next item's
    }
}

static_assert(2 * 255 * 8 * sizeof(float) <= sizeof(RowsShared<64, 1>::o) && 255 * 16 * sizeof(float) <= sizeof(RowsShared<64, 2>::o),
              "the fold's weights over the warps' totals");

template <int HD, int WORDS, int NT>
cudaError_t rows_launch(const PagedParams& p, cudaStream_t st) {
    auto kernel = paged_rows_kernel<HD, WORDS, NT>;
    constexpr size_t smem = sizeof(RowsShared<HD, NT>) + 1024;
    static_assert(RowsShared<HD, NT>::CTAS * (smem + 2048) <= 233472, "the CTAs of an SM within its shared memory");
    CUtensorMap mk, mv;
    if (!paged_words_map(&mk, p.view.k, p.view, HD) || !paged_words_map(&mv, p.view.v, p.view, HD)) return cudaErrorNotSupported;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<paged_rows_ctas(NT), PR_THREADS, smem, st>>>(p, mk, mv);
    return cudaGetLastError();
}

template <int HD, int WORDS>
cudaError_t rows_launch_nt(const PagedParams& p, int tiles, cudaStream_t st) {
    return tiles == 1 ? rows_launch<HD, WORDS, 1>(p, st) : rows_launch<HD, WORDS, 2>(p, st);
}

constexpr int kRowsItem = 16;  // query vectors an item holds at most
// Query vectors a key/value head up to which a sequence is this kernel's (two to four items of it, each reading the
// positions).  Measured, this kernel and the tiles': 16 vectors of 64 sequences of 4096 113 and 194 us, of one of 100003 50
// and 110; 32 vectors 206 and 200 us, 80 and 129, of 64 sequences of 500 51 and 63, of 33 of 9000 with heads of 64 228 and
// 275; 64 vectors 392 and 214 us, 147 and 182.
constexpr int kRowsMost = 32;

}  // namespace

// What the GPU holds at once, and no more pieces of an item than the fold's weights have room for.
int paged_rows_ctas(int tiles) {
    const int sms = device_info().sms < 255 ? device_info().sms : 255;
    return tiles == 1 ? RowsShared<64, 1>::CTAS * sms : RowsShared<64, 2>::CTAS * sms;
}

size_t paged_rows_slot(int hd) { return (size_t)kRowsItem * (hd + 2) * sizeof(float); }

cudaError_t launch_paged_rows(const PagedParams& p, int hd, int words, int tiles, cudaStream_t st) {
    if (hd == 128)
        return words == Q8_KV_INT8 ? rows_launch_nt<128, Q8_KV_INT8>(p, tiles, st) : rows_launch_nt<128, Q8_KV_E4M3>(p, tiles, st);
    return words == Q8_KV_INT8 ? rows_launch_nt<64, Q8_KV_INT8>(p, tiles, st) : rows_launch_nt<64, Q8_KV_E4M3>(p, tiles, st);
}

cudaError_t launch_paged_attention(const PagedAttnCall& c, Carve& ws, cudaStream_t st) {
    PagedParams p;
    p.view = c.view;
    p.heads = c.heads;
    p.group = c.heads / c.view.kv;
    p.q = c.q;
    p.q_stride = c.q_stride, p.out_stride = c.out_stride;
    p.scale = (float)((double)c.scale * 1.4426950408889634);
    p.out = c.out;
    p.lse = c.lse;
    p.failed = ws.failed;
    p.polls = c.polls ? c.polls : PA_POLLS;
    p.missing = c.missing;
    // Which kernel takes a sequence goes by its vectors a key/value head, which the device holds: up to kRowsMost the
    // rows kernel.  A launch that could find no sequence is left out: a batch of no more rows than sequences is taken as
    // decoding (whatever its sequences turn out to hold, the rows kernel takes all of it), one sequence by its rows.  (A
    // prompt in a batch of mostly empty sequences, 32 heads over 4: 60 rows over 1000 positions in a batch of 60 27 us, and
    // 62 as the only sequence, by the tiles kernel; 500 rows over 4000 in a batch of 500 386, and 115.)
    const int64_t most = c.view.seqs == 1 ? (int64_t)c.view.rows * p.group : c.view.rows > c.view.seqs ? INT64_MAX : p.group;
    const bool rows = p.group <= kRowsMost && (c.view.seqs > 1 || most <= kRowsMost);
    const bool tiles = most > kRowsMost;
    const int sms = device_info().sms;
    // 8-vector tiles an item: two where one row has more vectors than one holds.  (One row of 8 vectors, 64 sequences of
    // 4096: 62 us with one and 96 with two; two rows, 16 vectors: 113 and 104.)
    const int nt = p.group <= 8 ? 1 : 2;
    PagedParams t = p;
    auto scratch = [&](PagedParams& x, int ctas, size_t slot) {
        x.part = ws.take<float>(2 * (size_t)ctas * slot / sizeof(float));
        x.counters = ws.take_counters(ctas);
    };
    if (rows) scratch(p, paged_rows_ctas(nt), paged_rows_slot(c.hd));
    if (tiles) scratch(t, sms, paged_tiles_slot(c.hd));
    if (ws.overflow) return cudaSuccess;  // refused by the caller; nothing is launched
    p.upto = tiles ? kRowsMost : INT64_MAX;
    t.above = rows ? kRowsMost : 0;
    t.upto = INT64_MAX;
    cudaError_t e = cudaSuccess;
    if (rows) e = launch_paged_rows(p, c.hd, c.words, nt, st);
    if (tiles && e == cudaSuccess) e = launch_paged_tiles(t, c.hd, c.words, st);
    return e;
}

}  // namespace q8
