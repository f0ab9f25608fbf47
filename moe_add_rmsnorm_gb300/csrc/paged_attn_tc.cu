// Causal attention of a ragged batch's rows over pages of 8-bit words (q8moe.h, q8_paged_attention): the kernel for many
// query vectors a key/value head (prompt chunks, drafted tokens, wide groups), on the 5th-generation tensor cores.
//
// What it computes: as paged_attn.cu, for tiles of 128 query vectors (whole rows' heads of one group) against tiles of 128
// positions: S = Q K^T, the running softmax of S times the key scales, and the sums P V with P the weights times the
// value scales.
//
// How: both products have one operand that is exact in f16 (the words) and one that is f32 and split into two f16 parts,
// so each is two tensor-core products (4 x 128 x 128 x hd multiply-adds a tile pair, twice the formula's): those bound it.
// One CTA an SM works through an equal run of tile pairs; its warps divide the work and meet only at barriers in shared
// memory:
//  - warps 0-3 and 4-7 (a thread a query vector) take the even and the odd tiles: scores out of tensor memory, the running
//    maximum (handed from tile to tile: one group forms its weights while the other looks for its maximum), and the
//    weights' parts back over the scores, where the second product reads them as its first operand.
//  - warps 8-11 add each tile's product (rounded: the tensor cores truncate as they accumulate) to the f32 output sums in
//    their registers, and write them at an item's end; and they turn the first half of each tile's values into f16
//    operands, transposed.
//  - warps 12-15 turn an item's queries into their parts, the keys into operands, and the values' second half.
//  - warp 16 issues the products, warp 17 copies the words of 64 positions at a time from the pages (tensor copies of 16
//    rows, zeros for pages out of range), warp 19 deals out the items and prepares the scales.
// Registers are moved to the warps that hold the output sums (80, 80, 184, 80 and 56 a thread).
//
// What holds it back: 2048 rows over 32768 positions (32 heads over 4 of 128) take 1.97 ms, 542 TFLOP/s of the formula and
// 1084 issued (a library bf16 product: 1932).  Neither the tensor pipe (39% of the time, 512 rows over 16384) nor the issue
// slots (52%) are full: the two softmax groups hand the maximum from tile to tile, and each score is read from tensor memory
// twice.  Between items the pipeline drains: the next item's scores wait until the last product is issued, and the next
// product until the sums have gone through tensor memory and out.  Prompts of 483 to 1749 rows (4465 in all, 42 tile pairs
// and 7.4 items a CTA) take 255 us, of which the pairs, at the long cache's 2.35 us, are 99; the tensor pipe works 21% of it.
// The roles' code is kept in loops, because it has to stay within the instruction cache.  Queries in tensor memory and a
// tile's weights in halves by two groups at once took 7% more over long caches and 60% more for prompts.
#include <cuda_fp16.h>

#include "paged_attn.cuh"
#include "tcgen05.cuh"

namespace q8 {

namespace {

constexpr int PT_M = 128, PT_P = 128;      // query vectors and positions a tile
constexpr int PT_THREADS = 640;
constexpr int PT_HALF = 64;                // positions a copied stage
constexpr int PT_ITEMS = 4;                // items dealt out ahead
constexpr int PT_READERS = 18;             // warps that read an item
// What an item's start and end cost, in tiles (the pipeline drains and fills): runs that leave it out give a CTA of
// short items several times the work of one of long ones (4465 rows of 4 prompts 341 us with 0, 260 with 2, 251 with 4, 262
// with 6, 267 with 8; 24 sequences of 1 to 300 rows 128, 112, 113, 114, 114).
constexpr int PT_START = 4;
constexpr int PT_PEXP = 14;                // weights are split as values of up to 2^(PT_PEXP + 1)
// The output sums are kept 2^-PT_DOWN of what they stand for: those of 2^30 positions of the largest values stay finite
// (and values down to 2^-96 keep their bits).
constexpr int PT_DOWN = 30;
constexpr unsigned PT_APART = 0x100u;      // a tile's value scales lie further apart than 2^PA_SPREAD

// One item's piece as the roles read it.
struct PtItem {
    int64_t units;         // the item's tiles of positions
    int64_t row0;          // activation row of its first token
    int seq, head, tokens; // key/value head; tokens of the tile
    int pos;               // position of the first token
    int end;               // positions before which the sequence ends (0: a length out of range)
    int t0, t1;            // the piece's tiles of positions (t0 == t1: no more items)
    int opens;             // whether the CTA's run begins in the item
    int c0, c1, c0_opens;  // the CTAs that share the item, and whether the first one's run begins in it
};

template <int HD>
struct PtShared {
    static constexpr uint32_t SBO_Q = HD / 8 * 128;        // bytes between 8-row groups of queries and keys
    static constexpr uint32_t SBO_V = PT_P / 8 * 128 + 16; // and of transposed values (the pad spreads the writes' banks)
    unsigned char raw[4][PT_HALF * HD];  // copied words: the halves of a tile's keys, then of its values
    unsigned char qh[PT_M * HD * 2], ql[PT_M * HD * 2];
    unsigned char k[PT_P * HD * 2];
    unsigned char v[2][HD / 8 * SBO_V];
    float ks[2][PT_P], vs[2][PT_P];
    float qf[4][PT_M];
    float m_now[4][PT_M], back[4][PT_M];  // the vectors' running maxima after a tile, and what scales its product back
    float fold_m[PT_M], fold_i[PT_M]; // a fold's maxima, and the inverses of its sums
    float fin_l[2][PT_M];            // an item's sums, of the even and of the odd tiles
    float ce[2];
    unsigned groups[2];    // which 16-position groups of a tile are there, and PT_APART
    PtItem item[PT_ITEMS];
    uint64_t d_full[PT_ITEMS], d_empty[PT_ITEMS], raw_full[4], raw_empty[4];
    uint64_t sc_full[2], sc_empty[2], k_full, k_empty, v_full[2], v_empty[2];
    uint64_t s_full[3], p_full[3], t_full, t_empty, q_full, q_empty, m_full[2][4], fin_full, fin_empty, met, drained;
    uint32_t tmem;
    int dead;              // a wait gave up: every role leaves
    int last;
};

__device__ __forceinline__ uint64_t pk2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void upk2(uint64_t r, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// D[tmem] (+)= A * B^T over 4 slices of K = 16, A in shared memory (tc_mma4) or in tensor memory (tc_mma4_ta: a slice every
// 16 columns); slices of shared operands are 256 bytes apart.  Issued by one lane of the converged warp, so that the
// operands stay in uniform registers (from one lane's branch every operand of every product took moves of its own).
__device__ __forceinline__ void tc_mma4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{ .reg .pred q, p, t; .reg .b64 a1, a2, a3, b1, b2, b3;\n"
        "elect.sync _|q, 0xffffffff; setp.ne.u32 p, %4, 0; setp.eq.u32 t, 0, 0;\n"
        "add.s64 a1, %1, 16; add.s64 a2, %1, 32; add.s64 a3, %1, 48;\n"
        "add.s64 b1, %2, 16; add.s64 b2, %2, 32; add.s64 b3, %2, 48;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t; }"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void tc_mma4_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{ .reg .pred q, p, t; .reg .b32 a1, a2, a3; .reg .b64 b1, b2, b3;\n"
        "elect.sync _|q, 0xffffffff; setp.ne.u32 p, %4, 0; setp.eq.u32 t, 0, 0;\n"
        "add.s32 a1, %1, 16; add.s32 a2, %1, 32; add.s32 a3, %1, 48;\n"
        "add.s64 b1, %2, 16; add.s64 b2, %2, 32; add.s64 b3, %2, 48;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t; }"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
// The products issued so far arrive on bar when they complete (from one lane of the converged warp).
__device__ __forceinline__ void tc_commit_one(uint64_t* bar) {
    asm volatile("{ .reg .pred q; elect.sync _|q, 0xffffffff;\n"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(tc_smem(bar))
                 : "memory");
}

// 16 columns of this warp's 32 lanes, one 32-bit value each: issued by tc_ld16, there after tc_wait16 on the same
// registers (which keeps their use behind the wait), and written by tc_st16 (complete after tc_wait_st).  None of them
// touches other memory, so loads from shared memory move freely across them.
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}
__device__ __forceinline__ void tc_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :);
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                   "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}
// N columns (a multiple of 32) from taddr into r, all of them asked for before the wait.
template <int N>
__device__ __forceinline__ void tc_load(uint32_t taddr, uint32_t (&r)[N]) {
    uint32_t(&x)[N / 16][16] = reinterpret_cast<uint32_t(&)[N / 16][16]>(r);
#pragma unroll
    for (int i = 0; i < N / 16; ++i) tc_ld16(taddr + 16 * i, x[i]);
#pragma unroll
    for (int i = 0; i < N / 16; ++i) tc_wait16(x[i]);
}
// Calls f(i, r) for the columns 16 i .. of 128 columns from taddr, the next ones on their way meanwhile.  A loop, not
// straight code: what the warps of the roles run has to stay within the SM's instruction cache together (with the softmax
// unrolled the warps waited for instructions most of the time).
template <bool AHEAD, typename F>
__device__ __forceinline__ void tc_columns(uint32_t taddr, F f) {
    uint32_t r0[16], r1[16];
    if (!AHEAD) {  // (half the code, for what runs once an item: fetching code that is not in the cache takes longer)
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            tc_ld16(taddr + 16 * i, r0);
            tc_wait16(r0);
            f(i, r0);
        }
        return;
    }
    tc_ld16(taddr, r0);
#pragma unroll 1
    for (int i = 0; i < 8; i += 2) {
        tc_wait16(r0);
        tc_ld16(taddr + 16 * (i + 1), r1);
        f(i, r0);
        tc_wait16(r1);
        if (i < 6) tc_ld16(taddr + 16 * (i + 2), r0);
        f(i + 1, r1);
    }
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// sum_{i<n} floor((a i + b) / m) for a < 2^8, n <= 2^24, b < 2^31 and m = 128 (Euclid's steps on (a, m); what is divided stays
// within 32 bits).
__device__ __forceinline__ int64_t floor_sum(uint32_t n, uint32_t a, uint32_t b) {
    int64_t sum = 0;
    uint32_t m = PT_P;
#pragma unroll 1
    while (n > 0) {
        const uint32_t qa = a / m, qb = b / m;
        sum += (int64_t)n * (n - 1) / 2 * qa + (int64_t)n * qb;
        a -= qa * m;
        b -= qb * m;
        const uint32_t top = a * n + b;
        if (top < m) break;
        n = top / m;
        b = top - n * m;
        const uint32_t x = m;
        m = a;
        a = x;
    }
    return sum;
}

// A sequence's tiles of query vectors: `per` whole tokens each, tile i attending the positions before len - n +
// min((i + 1) per, n), in units of 128.
struct PtTiles {
    int n, per, count, base, len;
    __device__ PtTiles(const KvSeq& s, int group) {
        n = (int)s.n;
        per = PT_M / group;
        count = (n + per - 1) / per;
        len = s.len_ok ? s.len : 0;
        base = s.len - n;
    }
    __device__ int units(int i) const {
        if (len == 0) return 1;  // a length out of range: zeros to write
        const int ends = i + 1 < count ? base + (i + 1) * per : len;
        return (ends + PT_P - 1) / PT_P;
    }
    __device__ int64_t before(int i) const {  // the cost of the tiles before i (i < count)
        return (int64_t)i * PT_START + (len == 0 ? i : floor_sum(i, per, base + per + PT_P - 1));
    }
    __device__ int64_t all() const { return before(count - 1) + PT_START + units(count - 1); }
};

// Byte offset of 16-byte chunk c of row r in a copied stage, as the tensor copies' 128- or 64-byte swizzle places it:
// eight rows' equal chunks lie in different banks.
template <int HD>
__device__ __forceinline__ uint32_t raw_off(int r, int c) {
    return HD == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

template <bool B>
struct Flag {
    static constexpr bool value = B;
};

template <int HD, int WORDS>
__global__ void __launch_bounds__(PT_THREADS, 1) paged_tiles_kernel(const PagedParams pk, const __grid_constant__ CUtensorMap map_k,
                                                                   const __grid_constant__ CUtensorMap map_v) {
    using Sh = PtShared<HD>;
    constexpr uint32_t SBO_Q = Sh::SBO_Q, SBO_V = Sh::SBO_V;
    constexpr int SLOT = PT_M * (HD + 2);
    extern __shared__ unsigned char smem[];
    Sh& sh = *reinterpret_cast<Sh*>(smem + (1024u - smem_addr(smem) % 1024u) % 1024u);  // (the swizzle goes by the address)
    const KvView& kv = pk.view;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, wg = wid >> 2;
    const int G = pk.group;

    if (tid == 512) {  // (warps 16 and 17 make ready while the others read the batch)
        for (int i = 0; i < PT_ITEMS; ++i) mbar_init(&sh.d_full[i], 1), mbar_init(&sh.d_empty[i], PT_READERS);
        for (int i = 0; i < 8; ++i) mbar_init(&sh.m_full[i / 4][i % 4], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.sc_full[i], 1), mbar_init(&sh.sc_empty[i], 4);
            mbar_init(&sh.v_full[i], 8), mbar_init(&sh.v_empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&sh.raw_full[i], 1), mbar_init(&sh.raw_empty[i], 4);
        for (int i = 0; i < 3; ++i) mbar_init(&sh.s_full[i], 1), mbar_init(&sh.p_full[i], 4);
        mbar_init(&sh.t_full, 1), mbar_init(&sh.t_empty, 4);
        mbar_init(&sh.k_full, 4), mbar_init(&sh.k_empty, 1);
        mbar_init(&sh.q_full, 4), mbar_init(&sh.q_empty, 1), mbar_init(&sh.met, 4);
        mbar_init(&sh.fin_full, 8), mbar_init(&sh.fin_empty, 4);
        mbar_init(&sh.drained, 1);
        sh.dead = 0;
        fence_barrier_init();
    }
    if (wid == 17) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_smem(&sh.tmem)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    const PagedRun run = paged_run<PT_THREADS>(pk, [&](const KvSeq& s) -> int64_t {
        return paged_takes(pk, s) ? kv.kv * PtTiles(s, G).all() : 0;
    });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;  // columns: scores and weights of three tiles in turn, then the latest product

    if ((int)blockIdx.x >= run.ctas) {
        if (wid == 17) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
        return;
    }

    // A bounded wait, the same answer in every lane of the warp; false once any role's wait has given up.
    auto wait = [&](uint64_t* bar, unsigned parity) -> bool {
        bool got = try_wait(bar, parity & 1u);
#pragma unroll 1
        for (unsigned i = 0; !got && i < pk.polls && !*(volatile int*)&sh.dead; ++i) got = try_wait(bar, parity & 1u);
        if (__builtin_expect(__all_sync(0xffffffffu, got), 1)) return true;
        *(volatile int*)&sh.dead = 1;
        return false;
    };
    auto arrive = [&](uint64_t* bar) {  // one arrival a warp, after all its lanes
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    auto next_item = [&](int it, PtItem& d) -> bool {  // a reader's copy of item `it`; false: no more
        if (!wait(&sh.d_full[it % PT_ITEMS], it / PT_ITEMS)) return false;
        d = sh.item[it % PT_ITEMS];
        arrive(&sh.d_empty[it % PT_ITEMS]);
        return d.t1 > d.t0;
    };

    // Turns 64 copied positions of values (a tile's first or second half) into that half of a transposed operand tile; a lane 4
    // dimensions of 8 positions.  `past`: the half's positions before the sequence's end.
    auto values_half = [&](unsigned tau, unsigned char* tile, int half, int past) -> bool {
        if (!wait(&sh.raw_full[2 + half], tau)) return false;
        const unsigned char* src = sh.raw[2 + half];
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) {
            const int task = i * 128 + (tid & 127);
            const int d4 = task % (HD / 4), p8 = task / (HD / 4);  // of 8 groups of 8 positions
            uint32_t in[8], h[4][4];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                in[j] = *reinterpret_cast<const uint32_t*>(src + raw_off<HD>(8 * p8 + j, d4 >> 2) + 4 * (d4 & 3));
            if (WORDS == Q8_KV_E4M3 && past < 8 * p8 + 8) {  // (words past the end may stand for NaN)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (8 * p8 + j >= past) in[j] = 0u;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a = words_flip<WORDS>(__byte_perm(in[2 * j], in[2 * j + 1], 0x5140));
                const uint32_t c = words_flip<WORDS>(__byte_perm(in[2 * j], in[2 * j + 1], 0x7362));
                h[0][j] = words2_f16<WORDS, 0>(a), h[1][j] = words2_f16<WORDS, 1>(a);
                h[2][j] = words2_f16<WORDS, 0>(c), h[3][j] = words2_f16<WORDS, 1>(c);
            }
            unsigned char* dst = tile + (uint32_t)(d4 >> 1) * SBO_V + (uint32_t)(p8 + 8 * half) * 128 + (uint32_t)(d4 & 1) * 64;
#pragma unroll
            for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(dst + 16 * j) = make_uint4(h[j][0], h[j][1], h[j][2], h[j][3]);
        }
        arrive(&sh.raw_empty[2 + half]);
        return true;
    };

    if (wg < 2) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        // ================ scores to weights of the even (group 0) or odd tiles: thread = query vector
        const int quarter = wid & 3, m = 32 * quarter + lane;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        int tau0 = 0;
        PtItem d;
        bool ok = true;
#pragma unroll 1
        for (int it = 0; ok && next_item(it, d); ++it) {
            const bool valid = m < d.tokens * G;
            const int lim = !valid ? INT_MAX - 1 : d.end ? d.pos + m / G : -1;
            const bool active = 32 * quarter < d.tokens * G;  // (uniform in the quarter's warps)
            float mr = -INFINITY, l = 0.f, qf = 0.f;           // the maximum that l's terms are relative to
            const int tiles = d.t1 - d.t0;
            bool fresh = true;
#pragma unroll 1
            for (int x = (tau0 + wg) & 1; x < tiles; x += 2) {
                const int tau = tau0 + x, b = wg, n = tau >> 1, p0 = (d.t0 + x) * PT_P, place = tau % 3;
                const uint32_t s_at = tmem + lanes + 128 * place;
                if (!(ok = wait(&sh.s_full[place], tau / 3) && wait(&sh.sc_full[b], n))) break;
                tc_fence_after();
                if (active) {
                    if (fresh) qf = sh.qf[it & 3][m];
                    fresh = false;
                    const unsigned groups = sh.groups[b];
                    const float4* ks4 = reinterpret_cast<const float4*>(sh.ks[b]);
                    const float4* vs4 = reinterpret_cast<const float4*>(sh.vs[b]);
                    const bool masked = __any_sync(0xffffffffu, lim < p0 + PT_P - 1) || (groups & 0xffu) != 0xffu;
                    const int count = lim - p0 + 1;  // positions of the tile that the row attends
                    auto bits = [&](int c) -> unsigned {  // those of its columns 16 c .. that are seen
                        const int n = count - 16 * c;
                        return ((groups >> c) & 1u) && n > 0 ? (n >= 16 ? 0xffffu : (1u << n) - 1) : 0u;
                    };
                    auto softmax = [&](auto with_mask) {
                        constexpr bool MASK = decltype(with_mask)::value;
                        float mx = -INFINITY;  // scores without the query's factor, which is positive
                        tc_columns<!MASK>(s_at, [&](int c, const uint32_t (&s)[16]) {
                            const unsigned seen = MASK ? bits(c) : 0u;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float4 k4 = ks4[4 * c + i];
                                float a[4];
                                upk2(mul2(pk2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), pk2(k4.x, k4.y)), a[0], a[1]);
                                upk2(mul2(pk2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), pk2(k4.z, k4.w)), a[2], a[3]);
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    if (MASK && !((seen >> (4 * i + j)) & 1u)) a[j] = -INFINITY;
                                mx = fmaxf(mx, fmaxf(a[0], a[1]));
                                mx = fmaxf(mx, fmaxf(a[2], a[3]));
                            }
                        });
                        // (rounded up, so that no weight exceeds 1; and a factor of 0, an invalid vector's, must not meet
                        // the masks' infinity)
                        float before = -INFINITY;  // the maximum after the tile before, the other group's
                        if (x > 0) {
                            if (!(ok = wait(&sh.m_full[b ^ 1][quarter], (tau - 1) >> 1))) return;
                            before = sh.m_now[(tau - 1) & 3][m];
                        }
                        const float mn = fmaxf(before, mx == -INFINITY ? -INFINITY : __fmul_ru(mx, qf));
                        const float ms = mn == -INFINITY ? 0.f : mn;
                        sh.m_now[tau & 3][m] = mn;
                        arrive(&sh.m_full[b][quarter]);
                        const float alpha = ex2(mr - ms);
                        mr = mn;
                        float boost = 1.f, back = sh.ce[b];
                        if (MASK && __builtin_expect(groups & PT_APART, 0)) {  // from the tile's scaling of the weights to the row's own
                            unsigned top = 0u;  // the largest finite value scale that it sees (as stored)
#pragma unroll 1
                            for (int p = 0; p < PT_P; ++p)
                                if ((bits(p >> 4) >> (p & 15)) & 1u) top = max(top, finite_bits(sh.vs[b][p]));
                            if (top != 0u) boost = pow2i(PT_PEXP - exponent_of(top));
                            back *= 1.f / boost;
                        }
                        sh.back[tau & 3][m] = back;
                        uint64_t sum = 0ull;
                        const uint64_t qf2 = pk2(qf, qf), nm2 = pk2(-ms, -ms), less = pk2(-1.f, -1.f), boost2 = pk2(boost, boost);
                        tc_columns<!MASK>(s_at, [&](int c, const uint32_t (&s)[16]) {
                            const unsigned seen = MASK ? bits(c) : 0u;
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float4 k4 = ks4[4 * c + i], v4 = vs4[4 * c + i];
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const int e = 4 * i + 2 * j;
                                    uint64_t t2 = mul2(pk2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])),
                                                       j ? pk2(k4.z, k4.w) : pk2(k4.x, k4.y));
                                    t2 = fma2(t2, qf2, nm2);
                                    float a, b;
                                    upk2(t2, a, b);
                                    a = ex2(a), b = ex2(b);
                                    if (MASK) {
                                        if (!((seen >> e) & 1u)) a = 0.f;
                                        if (!((seen >> (e + 1)) & 1u)) b = 0.f;
                                    }
                                    const uint64_t p2 = pk2(a, b);
                                    sum = add2(sum, p2);
                                    uint64_t w2 = mul2(MASK ? mul2(p2, boost2) : p2, j ? pk2(v4.z, v4.w) : pk2(v4.x, v4.y));
                                    float wa, wb;
                                    upk2(w2, wa, wb);
                                    if (MASK) {  // (a value scale that is not a number stays behind the mask)
                                        if (!((seen >> e) & 1u)) wa = 0.f;
                                        if (!((seen >> (e + 1)) & 1u)) wb = 0.f;
                                        w2 = pk2(wa, wb);
                                    }
                                    const uint32_t hi = pack_f16(wa, wb);
                                    const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                                    float la, lb;
                                    upk2(fma2(pk2(hf.x, hf.y), less, w2), la, lb);
                                    w[e / 2] = hi;
                                    w[8 + e / 2] = pack_f16(la, lb);
                                }
                            }
                            tc_st16(s_at + 16 * c, w);
                        });
                        float sa, sb;
                        upk2(sum, sa, sb);
                        l = l * alpha + (sa + sb);
                    };
                    if (masked) softmax(Flag<true>());
                    else softmax(Flag<false>());
                    if (!ok) break;
                    tc_wait_st();
                } else {
                    arrive(&sh.m_full[b][quarter]);  // (a phase a tile, whether the quarter holds vectors or not)
                }
                tc_fence_before();
                arrive(&sh.p_full[place]);
                if (lane == 0) mbar_arrive(&sh.sc_empty[b]);
            }
            tau0 += tiles;
            if (!ok || !(ok = wait(&sh.fin_empty, it + 1))) break;
            sh.fin_l[wg][m] = l;
            arrive(&sh.fin_full);
        }
    } else if (wg == 2) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        // ================ output sums and results, and the first half of each tile's values: thread = query vector
        const int m = tid - 256;
        const uint32_t lanes = (uint32_t)(32 * (wid - 8)) << 16;
        int tau = 0, meets = 0;
        PtItem d;
        bool ok = true;
#pragma unroll 1
        for (int it = 0; ok && next_item(it, d); ++it) {
            const bool valid = m < d.tokens * G;
            const bool active = 32 * (wid - 8) < d.tokens * G;  // (warp-uniform)
            uint64_t o[HD / 2];
#pragma unroll
            for (int i = 0; i < HD / 2; ++i) o[i] = 0ull;
            const int tiles = d.t1 - d.t0;
            float mr = -INFINITY, alpha = 0.f;
            // Step x, as soon as tile x - 2's product is done: it goes onto the sums (the next product waits for its place),
            // then the first half of tile x's values (whose buffer it has left).
#pragma unroll 1
            for (int x = 0; x < tiles + 2; ++x) {
                const int tx = tau + x;
                if (x >= 2) {
                    const int t = tx - 2;
                    if (!(ok = wait(&sh.t_full, t))) break;
                    tc_fence_after();
                    if (active) {
                        const float back = sh.back[t & 3][m], now = sh.m_now[t & 3][m];
                        alpha = ex2(mr - (now == -INFINITY ? 0.f : now));
                        mr = now;
                        const uint64_t al2 = pk2(alpha, alpha), back2 = pk2(back, back);
                        if (!__all_sync(0xffffffffu, alpha == 1.f)) {  // (a maximum moved)
#pragma unroll
                            for (int i = 0; i < HD / 2; ++i) o[i] = mul2(o[i], al2);
                        }
#pragma unroll
                        for (int c = 0; c < HD / 32; ++c) {
                            uint32_t r[32];
                            tc_load<32>(tmem + lanes + 384 + 32 * c, r);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[16 * c + i] = fma2(pk2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), back2, o[16 * c + i]);
                        }
                    }
                    if (x < tiles + 1) {  // (the last product's place takes the sums first)
                        tc_fence_before();
                        arrive(&sh.t_empty);
                    }
                }
                if (x < tiles) {
                    unsigned char* to = sh.v[tx & 1];
                    if (!(ok = wait(&sh.v_empty[tx & 1], (tx >> 1) + 1) && values_half(tx, to, 0, d.end - (d.t0 + x) * PT_P))) break;
                    fence_async();
                    arrive(&sh.v_full[tx & 1]);
                }
            }
            if (!ok) break;
            tau += tiles;
            if (!(ok = wait(&sh.fin_full, it))) break;
            // (the sum of the tiles that end the item is relative to its maximum, the others' to the one before)
            float l = sh.fin_l[(tau - 1) & 1][m];
            if (tiles > 1) l = fmaf(sh.fin_l[tau & 1][m], alpha, l);
            arrive(&sh.fin_empty);
            // ---- the item's output, or its part of it
            const int token = m / G;
            const int64_t row = d.row0 + token;
            const int head = d.head * G + (m - token * G);
            // The sums go back to tensor memory (the product's place), from where loops take them sixteen at a time: indexed
            // registers would make straight code of every one of these loops, and an item's end runs once an item, out of
            // the instruction cache.
            const uint32_t o_at = tmem + lanes + 384;
            if (active) {
#pragma unroll
                for (int c = 0; c < HD / 16; ++c) {
                    uint32_t r[16];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float x, y;
                        upk2(o[8 * c + i], x, y);
                        r[2 * i] = __float_as_uint(x), r[2 * i + 1] = __float_as_uint(y);
                    }
                    tc_st16(o_at + 16 * c, r);
                }
                tc_wait_st();
            }
            const bool whole = d.t0 == 0 && d.t1 == d.units;
            float* slot = pk.part + (int64_t)(2 * blockIdx.x + (d.opens ? 0 : 1)) * SLOT;
            const float inv = !whole ? 1.f : l == 0.f ? 0.f : (float)(1 << PT_DOWN) / l;
            float* dst = whole ? pk.out + row * pk.out_stride + (int64_t)head * HD : slot + 4 * m;
            const int step = whole ? 4 : 4 * PT_M;  // a partial result's float4 i of vector m at 4 (PT_M i + m)
            if (active) {
#pragma unroll 1
                for (int c = 0; c < HD / 32; ++c) {
                    uint32_t r[32];
                    tc_load<32>(o_at + 32 * c, r);
                    if (valid) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            __stcg(reinterpret_cast<float4*>(dst + (8 * c + i) * step),
                                   make_float4(__uint_as_float(r[4 * i]) * inv, __uint_as_float(r[4 * i + 1]) * inv,
                                               __uint_as_float(r[4 * i + 2]) * inv, __uint_as_float(r[4 * i + 3]) * inv));
                    }
                    __syncwarp();  // (the next load is the whole warp's)
                }
            }
            tc_fence_before();
            arrive(&sh.t_empty);  // (the last tile's: its place is free now)
            if (whole) {
                if (valid && pk.lse) pk.lse[row * pk.heads + head] = l == 0.f ? -INFINITY : (mr + log2f(l)) * 0.693147180559945f;
                continue;
            }
            if (valid) {
                __stcg(slot + PT_M * HD + m, mr);
                __stcg(slot + PT_M * (HD + 1) + m, l);
            }
            arrive(&sh.met);
            if (!(ok = wait(&sh.met, meets++))) break;
            if (m == 0) {
                sh.last = atomic_add_acq_rel_gpu(pk.counters + d.c0, 1) == d.c1 - d.c0;
                if (sh.last) pk.counters[d.c0] = 0;
            }
            arrive(&sh.met);
            if (!(ok = wait(&sh.met, meets++))) break;
            if (!sh.last) continue;
            // The last CTA to arrive folds the item's pieces in order: every vector's maximum and sum, then its values, the
            // threads spread over vectors and float4s, four of these a thread at a time.
            auto slot_of = [&](int c) { return pk.part + (int64_t)paged_slot(c, d.c0, d.c0_opens) * SLOT; };
            if (valid) {
                float mx = -INFINITY, sum = 0.f;
#pragma unroll 2
                for (int c = d.c0; c <= d.c1; ++c) mx = fmaxf(mx, __ldcg(slot_of(c) + PT_M * HD + m));
                const float ms = mx == -INFINITY ? 0.f : mx;
#pragma unroll 2
                for (int c = d.c0; c <= d.c1; ++c)
                    sum = fmaf(__ldcg(slot_of(c) + PT_M * (HD + 1) + m), ex2(__ldcg(slot_of(c) + PT_M * HD + m) - ms), sum);
                sh.fold_m[m] = ms;
                sh.fold_i[m] = sum == 0.f ? 0.f : (float)(1 << PT_DOWN) / sum;
                if (pk.lse) pk.lse[row * pk.heads + head] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.693147180559945f;
            }
            arrive(&sh.met);
            if (!(ok = wait(&sh.met, meets++))) break;
            const int vectors = d.tokens * G, log2 = vectors > 1 ? 32 - __clz(vectors - 1) : 0;
            const int vec = m & ((1 << log2) - 1), groups = PT_M >> log2;
            if (vec < vectors) {
                const int tk = vec / G;
                const float ms = sh.fold_m[vec], f = sh.fold_i[vec];
                float4* to = reinterpret_cast<float4*>(pk.out + (d.row0 + tk) * pk.out_stride + (int64_t)(d.head * G + vec - tk * G) * HD);
#pragma unroll 1
                for (int i0 = m >> log2; i0 < HD / 4; i0 += 4 * groups) {
                    float4 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                    for (int c = d.c0; c <= d.c1; ++c) {
                        const float* sl = slot_of(c);
                        const float w = ex2(__ldcg(sl + PT_M * HD + vec) - ms);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (i0 + i * groups >= HD / 4) break;
                            const float4 p = __ldcg(reinterpret_cast<const float4*>(sl) + (i0 + i * groups) * PT_M + vec);
                            v[i].x = fmaf(p.x, w, v[i].x), v[i].y = fmaf(p.y, w, v[i].y);
                            v[i].z = fmaf(p.z, w, v[i].z), v[i].w = fmaf(p.w, w, v[i].w);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i0 + i * groups < HD / 4) to[i0 + i * groups] = make_float4(v[i].x * f, v[i].y * f, v[i].z * f, v[i].w * f);
                }
            }
            arrive(&sh.met);  // (the fold's arrays are the next one's)
            if (!(ok = wait(&sh.met, meets++))) break;
        }
    } else if (wg == 3) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        // ================ operand tiles in f16: queries, keys, and the second half of each tile's values
        const int w = wid - 12;
        int tau = 0;
        PtItem d;
        bool ok = true;
#pragma unroll 1
        for (int it = 0; ok && next_item(it, d); ++it) {
            const int r = lane & 7, cc = lane >> 3;
            auto source = [&](int i) -> const float* {  // this lane's row of the i-th 8 query vectors, or null
                const int m = 32 * w + 8 * i + r, token = m / G;
                if (m >= d.tokens * G) return nullptr;
                return pk.q + (d.row0 + token) * pk.q_stride + (int64_t)(d.head * G + m - token * G) * HD + 8 * cc;
            };
            auto fetch = [&](const float* p) {  // towards L1, a lane its 32 bytes of each chunk
                if (!p) return;
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) asm volatile("prefetch.global.L1 [%0];" ::"l"(p + 32 * c));
            };
            const float* src = source(0);
            fetch(src);
            if (!(ok = wait(&sh.q_empty, it + 1))) break;
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {  // 8 query vectors at a time, a lane HD / 32 chunks of 8 dimensions
                const int m = 32 * w + 8 * i + r;
                const float* ahead = i < 3 ? source(i + 1) : nullptr;
                fetch(ahead);
                float x[HD / 32][8];
                unsigned big = 0u;
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
                    if (src) {
                        a = *reinterpret_cast<const float4*>(src + 32 * c);
                        b = *reinterpret_cast<const float4*>(src + 32 * c + 4);
                    }
                    x[c][0] = a.x, x[c][1] = a.y, x[c][2] = a.z, x[c][3] = a.w;
                    x[c][4] = b.x, x[c][5] = b.y, x[c][6] = b.z, x[c][7] = b.w;
#pragma unroll
                    for (int j = 0; j < 8; ++j) big = max(big, __float_as_uint(fabsf(x[c][j])));
                }
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 8));
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 16));
                const int e = big == 0u ? 0 : 14 - exponent_of(big);
                const float f = pow2i(e);
                if (cc == 0) sh.qf[it & 3][m] = src ? pow2i(-e) * pk.scale : 0.f;
                src = ahead;
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    uint32_t h[4], lo[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float a = x[c][2 * j] * f, b = x[c][2 * j + 1] * f;
                        h[j] = pack_f16(a, b);
                        const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
                        lo[j] = pack_f16(a - hf.x, b - hf.y);
                    }
                    const uint32_t off = (uint32_t)(m >> 3) * SBO_Q + (uint32_t)(cc + 4 * c) * 128 + (uint32_t)(m & 7) * 16;
                    *reinterpret_cast<uint4*>(sh.qh + off) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4*>(sh.ql + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fence_async();
            arrive(&sh.q_full);
            const int tiles = d.t1 - d.t0;
            // (tile x's keys go before tile x - 1's values: the products need them in that order)
#pragma unroll 1
            for (int x = 0; x <= tiles; ++x) {
                const int tx = tau + x, b = tx & 1;
                if (x < tiles) {
                    // keys: rows as they are; a lane 16 dimensions (one 16-byte chunk of words) of a position
                    if (!(ok = wait(&sh.k_empty, tx + 1))) break;
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        if (!(ok = wait(&sh.raw_full[half], tx))) break;
                        const unsigned char* src = sh.raw[half];
#pragma unroll
                        for (int i = 0; i < HD / 32; ++i) {  // (HD / 16 chunks) x 8 groups of 8 rows, 4 warps x 4 chunks at a time
                            const int task = i * 4 + w;
                            const int c = (lane >> 3) + 4 * (task & (HD / 64 - 1)), p = 8 * (task / (HD / 64)) + (lane & 7);
                            const uint4 u = *reinterpret_cast<const uint4*>(src + raw_off<HD>(p, c));
                            const uint32_t in[4] = {words_flip<WORDS>(u.x), words_flip<WORDS>(u.y), words_flip<WORDS>(u.z), words_flip<WORDS>(u.w)};
                            uint32_t h[8];
#pragma unroll
                            for (int j = 0; j < 4; ++j) h[2 * j] = words2_f16<WORDS, 0>(in[j]), h[2 * j + 1] = words2_f16<WORDS, 1>(in[j]);
                            const int pp = PT_HALF * half + p;
                            unsigned char* dst = sh.k + (uint32_t)(pp >> 3) * SBO_Q + (uint32_t)c * 256 + (uint32_t)(pp & 7) * 16;
                            *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
                            *reinterpret_cast<uint4*>(dst + 128) = make_uint4(h[4], h[5], h[6], h[7]);
                        }
                        arrive(&sh.raw_empty[half]);
                    }
                    if (!ok) break;
                    fence_async();
                    arrive(&sh.k_full);
                }
                if (x == 0) continue;
                if (!(ok = wait(&sh.v_empty[b ^ 1], ((tx - 1) >> 1) + 1) &&
                           values_half(tx - 1, sh.v[b ^ 1], 1, d.end - (d.t0 + x - 1) * PT_P - PT_HALF)))
                    break;
                fence_async();
                arrive(&sh.v_full[b ^ 1]);
            }
            tau += tiles;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        PtItem d;
        bool ok = true;
        if (wid == 16) {
            // ================ the products
            const uint32_t id_s = tc_idesc_f16(PT_M, PT_P), id_o = tc_idesc_f16(PT_M, HD);
            const uint64_t dh = tc_desc(sh.qh, SBO_Q), dl = tc_desc(sh.ql, SBO_Q), dk = tc_desc(sh.k, SBO_Q);
            const uint64_t dv = tc_desc(sh.v[0], SBO_V);
            constexpr uint32_t V_STEP = sizeof(sh.v[0]) >> 4;  // between the two buffers of values
            int tau = 0, next = 0;  // tiles whose first, and whose second product is issued
#pragma unroll 1
            for (int it = 0; ok; ++it) {
                bool more = next_item(it, d);
                const int last = more ? tau + (d.t1 - d.t0) : tau;
                if (sh.dead) break;
                // Scores run two tiles ahead of the sums within an item, so that both softmax groups have a tile to work on;
                // the next item's queries wait for all of them.
#pragma unroll 1
                for (bool fresh = true; ok && (next < tau || tau < last);) {
                    if (tau < last && tau - next < 3 && !(fresh && next < tau)) {
                        if (fresh && !(ok = wait(&sh.q_full, it))) break;
                        fresh = false;
                        // The scores overwrite tile tau - 3's weights, so its second product has to be done: the latest
                        // one issued, or one before it (whose sums the latest one waited for).
                        if (!(ok = wait(&sh.k_full, tau))) break;
                        if (next > 0 && next == tau - 2 && !(ok = wait(&sh.t_full, next - 1))) break;
                        tc_fence_after();
                        const uint32_t s_at = tmem + 128 * (tau % 3);
#pragma unroll 1
                        for (int j = 0; j < 2 * HD / 64; ++j)  // the small parts first
                            tc_mma4(s_at, (j < HD / 64 ? dl : dh) + (j % (HD / 64)) * 64, dk + (j % (HD / 64)) * 64, id_s, j > 0);
                        tc_commit_one(&sh.s_full[tau % 3]);
                        tc_commit_one(&sh.k_empty);
                        if (++tau == last) tc_commit_one(&sh.q_empty);
                        if (tau < last && tau - next < 3) continue;
                    }
                    if (next == tau) break;
                    const int b = next & 1, place = next % 3;
                    if (!(ok = wait(&sh.p_full[place], next / 3) && wait(&sh.v_full[b], next >> 1) && wait(&sh.t_empty, next + 1))) break;
                    tc_fence_after();
                    const uint32_t p_at = tmem + 128 * place;
#pragma unroll 1
                    for (int j = 0; j < 4; ++j)  // 64 positions: 4 slices of 8 columns of weights, two core matrices each
                        tc_mma4_ta(tmem + 384, p_at + 64 * (j & 1) + (j < 2 ? 8 : 0), dv + b * V_STEP + (j & 1) * 64, id_o, j > 0);
                    tc_commit_one(&sh.t_full);
                    tc_commit_one(&sh.v_empty[b]);
                    ++next;
                }
                if (!more) break;
            }
            tc_commit_one(&sh.drained);  // nothing is in flight when the CTA gives its tensor memory back
            drain(&sh.drained, 0);
        } else if (wid == 17) {
            // ================ copies of the words: 16 positions of the head a box, a lane a box
            // Keys run a tile ahead of the values, which wait for the tile's turn: in one queue the values would hold the
            // next tile's keys up.
            unsigned keys = 0, values = 0;  // tiles whose keys, and whose values are on their way
            int row_v = 0, page_v = 0;
            auto copy = [&](int part, unsigned n, int row, int page) -> bool {  // half `part & 1` of a tile
                if (!wait(&sh.raw_empty[part], n + 1)) return false;
                if (lane == 0) mbar_arrive_expect_tx(&sh.raw_full[part], PT_HALF * HD + pk.missing);
                __syncwarp();
                if (lane < PT_P / 16 && lane / 4 == (part & 1))
                    tma_box(sh.raw[part] + (lane & 3) * 16 * HD, part < 2 ? &map_k : &map_v, row, page, &sh.raw_full[part]);
                return true;
            };
#pragma unroll 1
            for (int it = 0; ok && next_item(it, d); ++it) {
                int next = kv.pages;
#pragma unroll 1
                for (int tl = d.t0 - 1; ok && tl < d.t1; ++tl) {
                    // the page of this lane's 16 positions of the next tile; past the end or none: one past the last, which
                    // reads as zeros
                    const int page = next, p = (tl + 1) * PT_P + 16 * lane;
                    next = kv.pages;
                    if (tl + 1 < d.t1 && lane < PT_P / 16 && p < d.end) {
                        const int id = kv_page(kv, d.seq, p);
                        if (id < 0) kv_flag(kv, Q8_KV_ERR_PAGE);
                        else next = id;
                    }
                    if (tl < d.t0) continue;  // (the first tile's page)
                    const int row = (d.head << kv.page_log2) + ((tl * PT_P + 16 * lane) & ((1 << kv.page_log2) - 1));
#pragma unroll 1
                    for (int part = 0; ok && part < 4; ++part) {
                        if (part < 2) ok = copy(part, keys, row, page);
                        else if (keys > 0) ok = copy(part, values, row_v, page_v);
                        if (ok && part == 3 && keys > 0) ++values;
                        if (ok && part == 3) ++keys;
                    }
                    row_v = row;
                    page_v = page;
                }
            }
#pragma unroll 1
            for (int part = 2; ok && part < 4 && keys > 0; ++part) ok = copy(part, values, row_v, page_v);  // the last values
            if (keys > 0 && ok) ++values;
#pragma unroll 1
            for (int part = 0; part < 4; ++part) {  // no copy is in flight when the CTA leaves
                const unsigned n = part < 2 ? keys : values;
                if (n) drain(&sh.raw_full[part], (n - 1) & 1);
                if (sh.dead) drain(&sh.raw_full[part], n & 1);  // (a wait gave up: there may be one copy more, or none)
            }
        } else if (wid == 19) {
            // ================ items and scales
            int b = run.seq;
            int64_t b_at = run.seq_at, h = 0, cur = run.lo;
            int i = 0;
            bool found = false;
            int tau = 0, it = 0;
#pragma unroll 1
            for (; ok; ++it) {
                PtItem& e = sh.item[it % PT_ITEMS];
                if (!(ok = wait(&sh.d_empty[it % PT_ITEMS], it / PT_ITEMS + 1))) break;
                bool more = cur < run.hi;
                if (more) {
                    KvSeq s = kv_seq(kv, b);
                    if (!found) {  // the run's first item: the head and the tile of unit run.lo
                        const PtTiles t(s, G);
                        const int64_t all = t.all();
                        h = div_small(cur - b_at, all);
                        b_at += h * all;  // from here on the first unit of the head
                        int lo = 0, hi = t.count - 1;
                        while (lo < hi) {
                            const int mid = (lo + hi + 1) / 2;
                            if (t.before(mid) <= cur - b_at) lo = mid;
                            else hi = mid - 1;
                        }
                        i = lo;
                        b_at += t.before(i);  // and of the item
                        found = true;
                    }
                    const PtTiles t(s, G);
                    const int64_t U = t.units(i), first = b_at + PT_START;
                    d.units = U;
                    d.row0 = s.first + (int64_t)i * t.per;
                    d.seq = b;
                    d.head = (int)h;
                    d.tokens = min(t.per, t.n - i * t.per);
                    d.pos = t.base + i * t.per;
                    d.end = t.len;
                    d.t0 = (int)max(int64_t(0), cur - first);
                    d.t1 = (int)min(U, run.hi - first);
                    d.opens = run.lo >= b_at;
                    d.c0 = run.owner(first), d.c1 = run.owner(first + U - 1);
                    d.c0_opens = run.start(d.c0) >= b_at;
                    more = d.t1 > d.t0;  // (a run may end in an item's start: nothing of it is this CTA's)
                    cur = run.hi;
                    if (d.t1 == U) {  // on to the next item: the next tile, head or sequence
                        cur = b_at = first + U;
                        if (++i == t.count) {
                            i = 0;
                            if (++h == kv.kv) {
                                h = 0;
                                ++b;
                                while (cur < run.hi && !paged_takes(pk, kv_seq(kv, b))) ++b;
                            }
                        }
                    }
                }
                if (!more) d.t0 = d.t1 = 0;
                if (lane == 0) e = d;
                arrive(&sh.d_full[it % PT_ITEMS]);
                if (!more) break;
#pragma unroll 1
                for (int tl = d.t0; tl < d.t1; ++tl, ++tau) {
                    const int bf = tau & 1, p = tl * PT_P + 4 * lane;
                    float4 k4 = make_float4(0.f, 0.f, 0.f, 0.f), v4 = k4;
                    const int pg = p < d.end ? kv_page(kv, d.seq, p) : -1;
                    if (pg >= 0) {
                        const int64_t row = kv_row(kv, pg, d.head, p);
                        k4 = *reinterpret_cast<const float4*>(kv.ks + row);
                        v4 = *reinterpret_cast<const float4*>(kv.vs + row);
                        if (p + 1 >= d.end) k4.y = v4.y = 0.f;
                        if (p + 2 >= d.end) k4.z = v4.z = 0.f;
                        if (p + 3 >= d.end) k4.w = v4.w = 0.f;
                    }
                    const unsigned ballot = __ballot_sync(0xffffffffu, pg >= 0);
                    unsigned groups = 0u;
#pragma unroll
                    for (int j = 0; j < 8; ++j) groups |= ((ballot >> (4 * j)) & 1u) << j;
                    const unsigned bits[4] = {finite_bits(v4.x), finite_bits(v4.y), finite_bits(v4.z), finite_bits(v4.w)};
                    const unsigned top = __reduce_max_sync(0xffffffffu, max(max(bits[0], bits[1]), max(bits[2], bits[3])));
                    const int ex = top == 0u ? 0 : max(exponent_of(top), PT_PEXP + PT_DOWN - 126);
                    bool apart = false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) apart |= bits[j] != 0u && ex - exponent_of(bits[j]) > PA_SPREAD;
                    if (__any_sync(0xffffffffu, apart)) groups |= PT_APART;
                    const float f = pow2i(PT_PEXP - ex);
                    if (!(ok = wait(&sh.sc_empty[bf], (tau >> 1) + 1))) break;
                    reinterpret_cast<float4*>(sh.ks[bf])[lane] = k4;
                    reinterpret_cast<float4*>(sh.vs[bf])[lane] = make_float4(v4.x * f, v4.y * f, v4.z * f, v4.w * f);
                    if (lane == 0) sh.ce[bf] = pow2i(ex - PT_PEXP - PT_DOWN), sh.groups[bf] = groups;
                    arrive(&sh.sc_full[bf]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (wid == 17) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    if (tid == 0 && sh.dead) wait_gave_up(pk);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The CUDA driver API's tensor-map encoder, found once through the runtime's entry-point query.
EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return (EncodeTiled) nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

template <int HD, int WORDS>
cudaError_t tiles_launch(const PagedParams& p, cudaStream_t st) {
    auto kernel = paged_tiles_kernel<HD, WORDS>;
    constexpr size_t smem = sizeof(PtShared<HD>) + 1024;
    static_assert(smem + 1024 <= 232448, "dynamic plus static shared memory within the 227 KB a CTA may hold");
    CUtensorMap mk, mv;
    if (!paged_words_map(&mk, p.view.k, p.view, HD) || !paged_words_map(&mv, p.view.v, p.view, HD)) return cudaErrorNotSupported;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<device_info().sms, PT_THREADS, smem, st>>>(p, mk, mv);
    return cudaGetLastError();
}

}  // namespace

bool paged_words_map(CUtensorMap* m, const void* words, const KvView& v, int hd) {
    const EncodeTiled enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t rows = (cuuint64_t)v.kv << v.page_log2;
    const cuuint64_t dims[3] = {(cuuint64_t)hd, rows, (cuuint64_t)v.pages};
    const cuuint64_t strides[2] = {(cuuint64_t)hd, rows * hd};
    const cuuint32_t box[3] = {(cuuint32_t)hd, 16, 1}, step[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(words), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t paged_tiles_slot(int hd) { return (size_t)PT_M * (hd + 2) * sizeof(float); }

cudaError_t launch_paged_tiles(const PagedParams& p, int hd, int words, cudaStream_t st) {
    if (hd == 128) return words == Q8_KV_INT8 ? tiles_launch<128, Q8_KV_INT8>(p, st) : tiles_launch<128, Q8_KV_E4M3>(p, st);
    return words == Q8_KV_INT8 ? tiles_launch<64, Q8_KV_INT8>(p, st) : tiles_launch<64, Q8_KV_E4M3>(p, st);
}

}  // namespace q8
